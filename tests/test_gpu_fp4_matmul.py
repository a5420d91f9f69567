"""gptq_fp4_matmul and gptq_fp4_grouped_matmul against the fp64 product of what
the packed operands stand for.

Two kinds of comparison.  `_exact` inputs: scales that are powers of two close
together and codes drawn so that every partial sum is a multiple of a common
unit below 2^24 of it: fp32 sums are then exact in any order and the output
must equal the rounded exact product.  Drawn inputs: the tensor cores add 64
products a step to an fp32 sum; with the sum cut to 24 bits at each step (at
most 2^-23 of it) and at most S = sum |w x| in it, n / 64 steps are off by at
most (n / 64) 2^-23 S; the two tensor scales and parts that are added in fp32
afterwards are (up to 16) roundings of 2^-24.  The bound is
((n / 64) + 9) 2^-23 S |tw tx|, and for bf16 outputs 2^-8 |y| more for their
rounding (and its second order).
"""
import numpy as np
import pytest
import torch

from oracle import fp4_oracle as fo

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import post_weight_quantization_accum_b200 as gq

FMTS = ["mxfp4", "nvfp4"]


def _matrix(rows, n, fmt, seed, bounds, exact=False):
    """A packed matrix (dict on the GPU) and what it stands for, without the
    tensor scale (fp64), and the tensor scales."""
    rng = np.random.default_rng(seed)
    B = fo.BLOCK[fmt]
    nb = -(-n // B)
    codes = rng.integers(0, 16, size=(rows, nb * B)).astype(np.uint8)
    if exact:
        codes = rng.choice(np.array([0, 2, 4, 10, 12], dtype=np.uint8), size=codes.shape)  # 0, +-1, +-2
    codes[:, n:] = 0
    if fmt == "mxfp4":
        byte = rng.integers(127, 129, size=(rows, nb)) if exact else rng.integers(120, 134, size=(rows, nb))
    else:
        byte = rng.integers(7, 9, size=(rows, nb)) * 8 if exact else rng.integers(1, 127, size=(rows, nb))
    byte = byte.astype(np.uint8)
    groups = len(bounds) - 1
    ragged_bands = sum(-(-(b - a) // 128) for a, b in zip(bounds[:-1], bounds[1:]))
    tiles = fo.scale_tiles(byte, bounds)
    assert tiles.shape[0] == ragged_bands
    room = np.zeros((max(rows // 128 + groups, ragged_bands),) + tiles.shape[1:], dtype=np.uint8)
    room[:ragged_bands] = tiles
    packed = fo.pack(codes, n)
    t = rng.uniform(0.5, 2.0, size=groups).astype(np.float32) if fmt == "nvfp4" else np.ones(groups, dtype=np.float32)
    if exact:
        t[:] = 0.5 if fmt == "nvfp4" else 1.0
    q = {"packed": torch.tensor(packed).cuda(), "scales": torch.tensor(room).cuda(),
         "tensor_scale": torch.tensor(t).cuda() if fmt == "nvfp4" else None, "rows": rows, "n": n, "format": fmt,
         "groups": groups}
    return q, fo.unpack(packed, tiles, n, fmt, bounds), t


def _check(y, ref, mag, n, dtype, exact):
    y = y.double().cpu().numpy()
    if exact:
        want = torch.tensor(ref).to(dtype).double().numpy()
        np.testing.assert_array_equal(y, want)
        return
    bound = (n / 64 + 9) * 2.0 ** -23 * mag
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    worst = np.max(np.abs(y - ref) / np.maximum(bound, 1e-300))
    assert worst <= 1.0, worst


SIZES = [(1, 32, 1), (1, 4096, 128), (1, 1000, 300), (3, 64, 129), (16, 96, 128), (17, 200, 65), (31, 2080, 384),
         (33, 256, 130), (64, 4096, 256), (100, 1056, 1000), (128, 128, 128), (129, 300, 200), (250, 777, 131),
         (256, 512, 256), (257, 640, 129), (511, 100, 640), (1000, 2000, 1111)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,n,rows", SIZES)
@pytest.mark.parametrize("exact", [True, False])
def test_matmul_matches_the_exact_product(fmt, tokens, n, rows, exact):
    w, wv, wt = _matrix(rows, n, fmt, rows + n, [0, rows], exact)
    x, xv, xt = _matrix(tokens, n, fmt, tokens + 1, [0, tokens], exact)
    k = float(wt[0]) * float(xt[0])
    ref, mag = xv @ wv.T * k, np.abs(xv) @ np.abs(wv).T * k
    for dtype in (torch.float32, torch.bfloat16):
        y = gq.gptq_fp4_matmul(w, x, dtype=dtype)
        torch.cuda.synchronize()
        assert y.dtype == dtype and tuple(y.shape) == (tokens, rows)
        _check(y, ref, mag, n, dtype, exact)
    assert gq.gptq_get_device_status() == 0


GROUPS = [([1], 64, 32), ([4, 0, 1, 0], 128, 96), ([0, 0, 7], 300, 1000), ([1] * 9, 257, 64), ([130, 1, 0, 255, 40], 200, 264),
          ([300, 513, 16], 129, 520), ([0, 0], 64, 64), ([17] * 33, 64, 100),
          # few rows a group on average, some with several tiles
          ([100] + [0] * 9, 136, 320), ([0, 65, 3] + [1] * 20, 200, 768), ([300] + [2] * 11, 64, 1030), ([129, 64, 200] + [0] * 30, 130, 264)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,rows,n", GROUPS)
@pytest.mark.parametrize("exact", [True, False])
def test_grouped_matmul_matches_the_exact_products(fmt, counts, rows, n, exact):
    groups, tokens = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)])
    w, wv, wt = _matrix(groups * rows, n, fmt, 5, list(np.arange(groups + 1) * rows), exact)
    x, xv, xt = _matrix(tokens, n, fmt, 6, list(off), exact)
    offsets = torch.tensor(off, dtype=torch.int32).cuda()
    for dtype in (torch.float32, torch.bfloat16):
        y = gq.gptq_fp4_grouped_matmul(w, x, offsets, dtype=dtype)
        torch.cuda.synchronize()
        assert tuple(y.shape) == (tokens, rows)
        for g in range(groups):
            a, b = off[g], off[g + 1]
            if a == b:
                continue
            W, X, k = wv[g * rows:(g + 1) * rows], xv[a:b], float(wt[g]) * float(xt[g])
            _check(y[a:b], X @ W.T * k, np.abs(X) @ np.abs(W).T * k, n, dtype, exact)
    assert gq.gptq_get_device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_of_no_group_and_columns_past_the_rows_are_left_alone(fmt):
    off = np.array([5, 9, 9, 40])
    rows, n = 70, 96
    w, wv, wt = _matrix(3 * rows, n, fmt, 5, list(np.arange(4) * rows), True)
    x, xv, xt = _matrix(35, n, fmt, 6, [0, 4, 4, 35], True)
    packed = torch.zeros((50, x["packed"].shape[1]), dtype=torch.uint8, device="cuda")
    packed[5:40] = x["packed"]
    x = dict(x, packed=packed, rows=50, scales=x["scales"].clone())
    wide = torch.full((50, 100), 7.0, device="cuda")
    y = gq.gptq_fp4_grouped_matmul(w, x, torch.tensor(off, dtype=torch.int32).cuda(), y=wide[:, :rows])
    torch.cuda.synchronize()
    assert (wide[:5] == 7).all() and (wide[40:] == 7).all() and (wide[:, rows:] == 7).all()
    k = float(wt[0]) * float(xt[0])
    np.testing.assert_array_equal(y[5:9].double().cpu().numpy(), xv[:4] @ wv[:rows].T * k)
    np.testing.assert_array_equal(y[9:40].double().cpu().numpy(), xv[4:] @ wv[2 * rows:].T * k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,pitch", [(70, 72), (70, 71), (264, 512), (300, 301)])
def test_many_rows_stay_in_their_groups_and_columns(dtype, rows, pitch):
    """The same of the kernel for many tokens, with outputs that TMA can
    address and others."""
    fmt, n, off = "mxfp4", 160, np.array([3, 400, 400, 817])
    w, wv, wt = _matrix(3 * rows, n, fmt, 5, list(np.arange(4) * rows), True)
    x, xv, xt = _matrix(814, n, fmt, 6, [0, 397, 397, 814], True)
    packed = torch.zeros((830, x["packed"].shape[1]), dtype=torch.uint8, device="cuda")
    packed[3:817] = x["packed"]
    x = dict(x, packed=packed, rows=830)
    wide = torch.full((830, pitch), 7.0, dtype=dtype, device="cuda")
    y = gq.gptq_fp4_grouped_matmul(w, x, torch.tensor(off, dtype=torch.int32).cuda(), y=wide[:, :rows])
    torch.cuda.synchronize()
    assert (wide[:3] == 7).all() and (wide[817:] == 7).all() and (wide[:, rows:] == 7).all()
    _check(y[3:400], xv[:397] @ wv[:rows].T, None, n, dtype, True)
    _check(y[400:817], xv[397:] @ wv[2 * rows:].T, None, n, dtype, True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,n,rows,pitch", [(2100, 96, 2310, 2312), (2100, 96, 2304, 2304), (2305, 300, 2329, 2400),
                                                 (2100, 96, 2310, 2311), (20000, 64, 33, 40), (20001, 64, 24, 24)])
def test_many_tiles_of_one_matrix(fmt, dtype, tokens, n, rows, pitch):
    """More tiles than pairs of CTAs, the last of them part full both ways;
    rows of y that TMA can address and others, and what is beside them."""
    w, wv, wt = _matrix(rows, n, fmt, 7, [0, rows], True)
    x, xv, xt = _matrix(tokens, n, fmt, 8, [0, tokens], True)
    wide = torch.full((tokens + 1, pitch), 7.0, dtype=dtype, device="cuda")
    y = gq.gptq_fp4_matmul(w, x, y=wide[:tokens, :rows])
    torch.cuda.synchronize()
    assert (wide[tokens:] == 7).all() and (wide[:, rows:] == 7).all()
    _check(y, xv @ wv.T * (float(wt[0]) * float(xt[0])), None, n, dtype, True)
    assert gq.gptq_get_device_status() == 0


@pytest.mark.parametrize("off", [[0, 9, 5, 20], [0, 5, 21, 20], [-1, 5, 9, 20], [0, 5, 9, 21]])
@pytest.mark.parametrize("times", [1, 30])
def test_bad_offsets_touch_nothing_and_are_reported(off, times):
    """Of the kernels for few tokens and for many."""
    w, _, _ = _matrix(3 * 32, 64, "mxfp4", 5, [0, 32, 64, 96])
    x, _, _ = _matrix(20 * times, 64, "mxfp4", 6, [0, 5 * times, 9 * times, 20 * times])
    gq.gptq_get_device_status()
    y = torch.full((20 * times, 32), 7.0, device="cuda")
    gq.gptq_fp4_grouped_matmul(w, x, torch.tensor(off, dtype=torch.int32).cuda() * times, y=y)
    assert gq.gptq_get_device_status() == 1
    assert (y == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_a_nan_scale_reaches_its_row_and_no_other(fmt):
    w, wv, wt = _matrix(200, 320, fmt, 5, [0, 200], True)
    x, xv, xt = _matrix(40, 320, fmt, 6, [0, 40], True)
    x["scales"][0, 0, 16 * (35 % 32) + 4 + 1] = 255 if fmt == "mxfp4" else 127   # row 35, block 1
    y = gq.gptq_fp4_matmul(w, x)
    torch.cuda.synchronize()
    k = float(wt[0]) * float(xt[0])
    y = y.double().cpu().numpy()
    assert np.isnan(y[35]).all()
    keep = np.arange(40) != 35
    np.testing.assert_array_equal(y[keep], (xv @ wv.T * k)[keep])


def test_the_same_bits_every_time():
    w, _, _ = _matrix(1000, 4096, "nvfp4", 5, [0, 1000])
    for tokens in (1, 20, 300):
        x, _, _ = _matrix(tokens, 4096, "nvfp4", 6, [0, tokens])
        first = gq.gptq_fp4_matmul(w, x)
        for _ in range(3):
            assert torch.equal(first, gq.gptq_fp4_matmul(w, x))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [1, 40, 600])
def test_a_layer_from_weights_to_outputs(fmt, tokens):
    """Weights and activations quantised by the library and multiplied, as a
    layer is used: against the oracle's quantisation and an fp64 product."""
    gen = torch.Generator().manual_seed(tokens)
    W = torch.randn((520, 1032), generator=gen) * 0.02
    X = torch.randn((tokens, 1032), generator=gen).to(torch.bfloat16)
    w = gq.gptq_fp4_quantize(W.cuda(), fmt)
    y = gq.fp4_linear(w, X.cuda(), dtype=torch.float32)
    torch.cuda.synchronize()
    wv = fo.quantize(W.double().numpy(), fmt)[3].astype(np.float64)
    xv = fo.quantize(X.double().numpy(), fmt)[3].astype(np.float64)
    _check(y, xv @ wv.T, np.abs(xv) @ np.abs(wv).T, 1032 + 64, torch.float32, False)  # (a step more: the values' own rounding)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,top,experts", [(1, 4, 8), (50, 2, 5), (300, 3, 4)])
def test_a_layer_of_experts(fmt, tokens, top, experts):
    """Dispatch (gather, quantise), the experts' products, and back to the
    tokens: against plain fp64 arithmetic on the oracle's quantised values."""
    rng = np.random.default_rng(tokens)
    rows, n = 136, 544
    W = torch.tensor(rng.standard_normal((experts, rows, n)) * 0.02, dtype=torch.float32).to(torch.bfloat16)
    X = torch.tensor(rng.standard_normal((tokens, n)), dtype=torch.float32).to(torch.bfloat16)
    expert = np.stack([rng.choice(experts, size=top, replace=False) for _ in range(tokens)]).reshape(-1)
    order = np.argsort(expert, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(expert, minlength=experts))])
    index = order // top
    w = gq.gptq_fp4_quantize(W.cuda(), fmt)
    y = gq.fp4_linear(w, X.cuda(), dtype=torch.bfloat16, row_index=torch.tensor(index, dtype=torch.int32).cuda(),
                      offsets=torch.tensor(off, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    xv = fo.quantize(X.double().numpy()[index], fmt, off)[3].astype(np.float64)
    wv = fo.quantize(W.double().numpy().reshape(-1, n), fmt, np.arange(experts + 1) * rows)[3].astype(np.float64)
    for g in range(experts):
        a, b = off[g], off[g + 1]
        if a < b:
            w_g = wv[g * rows:(g + 1) * rows]
            _check(y[a:b], xv[a:b] @ w_g.T, np.abs(xv[a:b]) @ np.abs(w_g).T, n + 64, torch.bfloat16, False)


LINEAR = [(1, 32, 40), (1, 4096, 4096), (1, 4100, 300), (2, 2048, 129), (3, 777, 1000), (4, 4096, 700), (5, 1000, 64),
          (16, 1024, 256), (16, 96, 130), (1, 16384, 128), (1, 16384, 20000), (17, 512, 128), (2, 9000, 64), (40, 1032, 300)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,n,rows", LINEAR)
def test_linear_equals_quantise_and_product(fmt, dtype, tokens, n, rows):
    """One call or two: the same bits, where the product quantises its few
    tokens itself and where it does not; rows of X with a pitch, values that
    are zero and not finite, given tensor scales."""
    gen = torch.Generator("cuda").manual_seed(tokens + n)
    w = gq.gptq_fp4_quantize(torch.randn((rows, n), device="cuda", generator=gen) * 0.02, fmt)
    base = torch.randn((tokens, n + 24), device="cuda", generator=gen)
    base[:, 3] = 0
    if tokens > 1:
        base[1] = 0
    for off in (0, 1, 8, 24):
        X = base.to(dtype)[:, off:off + n]
        want = gq.gptq_fp4_matmul(w, gq.gptq_fp4_quantize(X, fmt))
        assert torch.equal(gq.fp4_linear(w, X, dtype=torch.float32), want)
    if fmt == "nvfp4":
        t = torch.tensor([0.0173], device="cuda")
        want = gq.gptq_fp4_matmul(w, gq.gptq_fp4_quantize(X, fmt, tensor_scale=t))
        assert torch.equal(gq.fp4_linear(w, X, dtype=torch.float32, tensor_scale=t), want)
    X = X.clone()
    X[tokens - 1, n - 1] = float("nan")
    want = gq.gptq_fp4_matmul(w, gq.gptq_fp4_quantize(X, fmt), dtype=torch.bfloat16)
    got = gq.fp4_linear(w, X, dtype=torch.bfloat16)
    assert torch.isnan(got[tokens - 1]).all()
    assert torch.equal(got[: tokens - 1], want[: tokens - 1]) and not torch.isnan(got[: tokens - 1]).any()
    assert gq.gptq_get_device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,rows,n", [([1], 64, 32), ([0, 4, 0], 200, 4096), ([1, 1, 1, 1], 256, 4096), ([0, 0, 16, 0], 130, 1000),
                                           ([3, 0, 5, 8], 129, 1024), ([1] * 16, 96, 96), ([0] * 30 + [2, 1], 512, 2056)])
def test_linear_of_experts_equals_quantise_and_product(fmt, counts, rows, n):
    """Few tokens through experts, gathered; the first rows belong to none."""
    groups, tokens = len(counts), sum(counts)
    gen = torch.Generator("cuda").manual_seed(groups + n)
    w = gq.gptq_fp4_quantize(torch.randn((groups, rows, n), device="cuda", generator=gen) * 0.02, fmt)
    X = torch.randn((7, n), device="cuda", generator=gen).to(torch.bfloat16)
    idx = torch.randint(0, 7, (tokens,), device="cuda", generator=gen).int()
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
    want = gq.gptq_fp4_grouped_matmul(w, gq.gptq_fp4_quantize(X, fmt, row_index=idx, offsets=off), off)
    assert torch.equal(gq.fp4_linear(w, X, dtype=torch.float32, row_index=idx, offsets=off), want)
    assert gq.gptq_get_device_status() == 0
    if tokens >= 2:  # rows of no group are left alone; a bad index is a row of zeros and reported
        off2 = off.clone()
        off2.clamp_(min=1)
        y = torch.full((tokens, rows), 7.0, device="cuda")
        gq.fp4_linear(w, X, row_index=idx, offsets=off2, y=y)
        assert (y[0] == 7).all() and not (y[1:] == 7).any()
        idx[1] = 7
        y = gq.fp4_linear(w, X, row_index=idx, offsets=off)
        assert gq.gptq_get_device_status() == 1
        assert (y[1] == 0).all()
    off[-1] += 1
    y = torch.full((tokens, rows), 7.0, device="cuda")
    gq.fp4_linear(w, X, row_index=torch.zeros_like(idx), offsets=off, y=y)
    assert gq.gptq_get_device_status() == 1 and (y == 7).all()


def test_captured_and_replayed():
    """A quantise and product pair in a CUDA graph, replayed on new inputs."""
    w = gq.gptq_fp4_quantize((torch.randn((512, 2048), device="cuda") * 0.02), "nvfp4")
    X = torch.randn((24, 2048), device="cuda").to(torch.bfloat16)
    gq.fp4_linear(w, X)  # first call outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = gq.fp4_linear(w, X)
    for seed in range(3):
        X.copy_(torch.randn((24, 2048), device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
        g.replay()
        got = y.clone()
        assert torch.equal(got, gq.fp4_linear(w, X))


def test_two_graphs_of_one_layer():
    """Captured apart, replayed in turn and both at once on two streams."""
    w = gq.gptq_fp4_quantize((torch.randn((1024, 2048), device="cuda") * 0.02), "nvfp4")
    Xs = [torch.randn((t, 2048), device="cuda").to(torch.bfloat16) for t in (1, 200)]
    want = [gq.fp4_linear(w, X) for X in Xs]
    graphs, ys = [], []
    for X in Xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys.append(gq.fp4_linear(w, X))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, want))


def test_outputs_past_32_bits():
    """Over 2^31 outputs: the last tokens like the same tokens alone."""
    tokens, rows, n = 270000, 8192, 64
    w = gq.gptq_fp4_quantize(torch.randn((rows, n), device="cuda"), "mxfp4")
    X = torch.zeros((tokens, n), dtype=torch.bfloat16, device="cuda")
    X[-400:] = torch.randn((400, n), device="cuda").to(torch.bfloat16)
    y = gq.fp4_linear(w, X)
    assert y.numel() > 2 ** 31
    assert torch.equal(y[-400:], gq.fp4_linear(w, X[-400:].contiguous()))
    assert not y[: tokens - 400: 1000].any()


@pytest.mark.parametrize("fmt", FMTS)
def test_tensor_scales_whose_product_leaves_the_normal_numbers(fmt):
    """Weights of 1e-30 and activations of 1e-18 or 1e30: each scale is used in
    turn where their product is no normal number."""
    gen = torch.Generator("cuda").manual_seed(3)
    W = torch.randn((130, 96), device="cuda", generator=gen)
    X = torch.randn((300, 96), device="cuda", generator=gen)
    for tokens in (5, 300):
        want = gq.fp4_linear(gq.gptq_fp4_quantize(W, fmt), X[:tokens]).double()
        for a, b in ((2.0 ** -100, 2.0 ** -20), (2.0 ** -60, 2.0 ** 100), (2.0 ** 50, 2.0 ** 60)):
            y = gq.fp4_linear(gq.gptq_fp4_quantize(W * a, fmt), X[:tokens] * b).double() / (a * b)
            # powers of two move no code; each product with a scale rounds, at most half of the least subnormal
            bound = want.abs() * 2.0 ** -22 + 2.0 ** -149 / (a * b)
            assert ((y - want).abs() <= bound).all()


def test_on_another_stream():
    w = gq.gptq_fp4_quantize(torch.randn((300, 1024), device="cuda"), "nvfp4")
    X = torch.randn((70, 1024), device="cuda").to(torch.bfloat16)
    want = gq.fp4_linear(w, X)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [gq.fp4_linear(w, X, stream=side) for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(want, y) for y in got)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,rows", [(1, 300), (3, 9000), (12, 300), (70, 300), (128, 20000), (600, 300), (900, 4096)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(fmt, tokens, rows):
    """Each kind of product (that quantises its tokens, cut along K or not, of
    CTA pairs): every wait is bounded, and the GPU is as before afterwards."""
    w = gq.gptq_fp4_quantize(torch.randn((rows, 2048), device="cuda"), fmt)
    X = torch.randn((tokens, 2048), device="cuda")
    x = gq.gptq_fp4_quantize(X, fmt)
    want = gq.gptq_fp4_matmul(w, x)
    for call in (lambda: gq.gptq_fp4_matmul(w, x), lambda: gq.fp4_linear(w, X)):
        torch.cuda.synchronize()
        gq.gptq_set_wait_limit_ns(0)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            gq.gptq_set_wait_limit_ns(2 ** 64 - 1)
        assert gq.gptq_get_device_status() == 6
        assert torch.equal(want, call())
        assert gq.gptq_get_device_status() == 0
