"""gptq_fp4_quantize against the fp64 oracle: codes, scales, tensor scales and
dequantised values are decided on exact numbers on both sides, so all of them
must be equal (the dequantised value is one rounding of an exact product)."""
import numpy as np
import pytest
import torch

from oracle import fp4_oracle as fo

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import post_weight_quantization_accum_b200 as gq

FMTS = ["mxfp4", "nvfp4"]
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _x(rows, n, seed, dtype, kind="normal"):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, n))
    if kind == "outliers":
        x[:, rng.random(n) < 0.02] *= 30
    if kind == "zeros":
        x[rng.random((rows, n)) < 0.4] = 0.0
        x[:: 3] = 0.0
        x[:, :5] = -0.0
    if kind == "wide":
        x *= 2.0 ** rng.integers(-60, 60, size=(rows, n))
    return torch.tensor(x, dtype=torch.float32).to(DTYPES[dtype])


def _compare(q, X, fmt, bounds=None, tensor_scale=None):
    """q (with deq) against the oracle on X (host tensor, rows in result order)."""
    rows, n = X.shape
    bounds = [0, rows] if bounds is None else list(bounds)
    codes, byte, t, values = fo.quantize(X.double().numpy(), fmt, bounds, tensor_scale)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(q["packed"].cpu().numpy(), fo.pack(codes, n))
    tiles = fo.scale_tiles(byte, bounds)
    np.testing.assert_array_equal(q["scales"].cpu().numpy()[: tiles.shape[0]], tiles)
    if fmt == "nvfp4":
        np.testing.assert_array_equal(q["tensor_scale"].cpu().numpy(), t if tensor_scale is None else tensor_scale)
    else:
        assert q["tensor_scale"] is None
    if "deq" in q:
        np.testing.assert_array_equal(q["deq"].cpu().numpy(), values)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", [(1, 1), (1, 16), (1, 4096), (2, 31), (3, 33), (5, 100), (128, 256), (129, 264),
                                    (257, 1000), (40, 4097), (300, 2056)])
def test_quantize_matches_oracle(fmt, dtype, rows, n):
    X = _x(rows, n, rows + n, dtype, "outliers")
    _compare(gq.gptq_fp4_quantize(X.cuda(), fmt, want_deq=True), X, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["zeros", "wide"])
def test_quantize_zeros_and_wide_ranges(fmt, dtype, kind):
    X = _x(70, 520, 7, dtype, kind)
    _compare(gq.gptq_fp4_quantize(X.cuda(), fmt, want_deq=True), X, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("value", [0.0, 1e-45, 2.0 ** -126, 3.0e38])
def test_quantize_one_value_everywhere(fmt, value):
    """All zeros, the smallest fp32, the smallest normal one, near the largest."""
    X = torch.full((4, 64), value, dtype=torch.float32)
    X[1] *= -1
    X[2, ::2] = 0
    _compare(gq.gptq_fp4_quantize(X.cuda(), fmt, want_deq=True), X, fmt)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** 118])
@pytest.mark.parametrize("n", [1, 17, 33, 300])
def test_tensor_scales_at_the_ends_of_the_range(dtype, scale, n):
    """Values whose tensor scale, or 1 / (s t), is near the ends of fp32: the
    decisions are then taken in 64 bits, at the rows' ends too."""
    X = (_x(40, n, 3, "f32") * scale).to(DTYPES[dtype])
    _compare(gq.gptq_fp4_quantize(X.cuda(), "nvfp4", want_deq=True), X, "nvfp4")
    ts = torch.tensor([scale / 100])
    _compare(gq.gptq_fp4_quantize(X.cuda(), "nvfp4", tensor_scale=ts.cuda(), want_deq=True), X, "nvfp4",
             tensor_scale=ts.numpy())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_that_are_not_finite_make_their_block_nan(fmt, dtype):
    X = _x(200, 300, 3, dtype)
    X[0, 0], X[3, 40], X[150, 299], X[7, 100:120] = float("nan"), float("inf"), -float("inf"), float("nan")
    q = gq.gptq_fp4_quantize(X.cuda(), fmt, want_deq=True)
    _compare(q, X, fmt)
    B = fo.BLOCK[fmt]
    d = q["deq"].cpu()
    assert torch.isnan(d[0, :B]).all() and not torch.isnan(d[1]).any() and torch.isnan(d[150, 299])


@pytest.mark.parametrize("scale", [1.0, 0.75, 0.0123456, 3.1e-5, 2.0 ** -126, 1e36])
def test_decisions_next_to_every_border(scale):
    """nvfp4 with given tensor scales: values a float below, on and above each
    border of the code, for every E4M3 scale (a block's first value fixes it)."""
    t = np.float32(scale)
    rows = []
    for s in fo.E4M3[1:]:
        top = np.float64(s) * np.float64(t) * 6
        if not top < 3e38:
            continue
        v = [np.float32(top)]
        borders = (fo.E2M1[1:] + fo.E2M1[:-1]) / 2 * s * np.float64(t)
        for b in borders:
            c = np.float32(b)
            v += [c, np.nextafter(c, np.float32(0)), -np.nextafter(c, np.float32(np.inf))]
        for at in range(0, len(v) - 1, 15):
            rows.append([v[0]] + (v[1:] + v[1:])[at:at + 15])
    X = torch.tensor(np.array(rows, dtype=np.float32))
    ts = torch.tensor([scale], dtype=torch.float32)
    q = gq.gptq_fp4_quantize(X.cuda(), "nvfp4", tensor_scale=ts.cuda(), want_deq=True)
    _compare(q, X, "nvfp4", tensor_scale=ts.numpy())


def test_scale_decisions_next_to_every_border():
    """The block's maximum a float below, on and above each border between two
    E4M3 scales."""
    t = np.float32(0.0371)
    borders = (fo.E4M3[1:] + fo.E4M3[:-1]) / 2 * 6 * np.float64(t)
    X = np.zeros((3 * len(borders), 16), dtype=np.float32)
    for i, b in enumerate(borders):
        c = np.float32(b)
        X[3 * i, 3], X[3 * i + 1, 3], X[3 * i + 2, 3] = c, np.nextafter(c, np.float32(0)), np.nextafter(c, np.float32(9e9))
        X[3 * i:3 * i + 3, 5] = -c / 3
    X = torch.tensor(X)
    q = gq.gptq_fp4_quantize(X.cuda(), "nvfp4", tensor_scale=torch.tensor([t]).cuda(), want_deq=True)
    _compare(q, X, "nvfp4", tensor_scale=np.array([t]))


def test_tensor_scale_given_too_small_saturates():
    X = _x(9, 48, 5, "f32") * 1e6
    ts = torch.tensor([0.5])
    _compare(gq.gptq_fp4_quantize(X.cuda(), "nvfp4", tensor_scale=ts.cuda(), want_deq=True), X, "nvfp4",
             tensor_scale=ts.numpy())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("pad", [0, 1, 8, 16, 24])
def test_rows_with_a_pitch(fmt, pad):
    """Views whose rows start on 32, 16 and fewer bytes."""
    base = _x(37, 256 + pad, 11, "bf16")
    for off in (0, 1, 8):
        if off > pad:
            continue
        X = base[:, off:off + 256]
        _compare(gq.gptq_fp4_quantize(base.cuda()[:, off:off + 256], fmt, want_deq=True), X, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype,pitch", [("f32", 516), ("bf16", 520)])
@pytest.mark.parametrize("want_deq", [False, True])
def test_rows_on_16_bytes(fmt, dtype, pitch, want_deq):
    """Every other row starts between two 32-byte places; whole chunks of
    columns and one that ends early, one matrix and groups with an empty one."""
    X = _x(700, pitch, 12, dtype, "outliers")
    for n in (512, 300):
        _compare(gq.gptq_fp4_quantize(X.cuda()[:, :n], fmt, want_deq=want_deq), X[:, :n], fmt)
        off = np.array([0, 130, 130, 700])
        q = gq.gptq_fp4_quantize(X.cuda()[:, :n], fmt, offsets=torch.tensor(off, dtype=torch.int32).cuda(), want_deq=want_deq)
        _compare(q, X[:, :n], fmt, off)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [20, 300])
@pytest.mark.parametrize("n", [1, 5, 257, 513, 735, 1021])
def test_the_maximum_is_found_anywhere(dtype, rows, n):
    """One value larger than all others: in a first, last or middle column, of
    rows on every place, dense, with a pitch and gathered; a larger one beside
    the rows, infinities and NaN do not count."""
    base = torch.ones(rows * (n + 3) + 16, dtype=dtype, device="cuda")
    back = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda")
    places = sorted({c for c in (0, 1, 6, 7, 8, 254, 255, 256, 511, 512, n // 2, n - 2, n - 1) if 0 <= c < n})
    want = torch.tensor([max(np.float32(5.0) / np.float32(2688.0), 2.0 ** -126)])
    for off, pitch, index in ((0, n, None), (1, n, None), (3, n + 3, None), (5, n + 1, back), (0, n, back)):
        base.fill_(4096.0)
        X = base[off:off + rows * pitch].as_strided((rows, n), (pitch, 1))
        X.fill_(1.0)
        if n > 1:
            X[rows // 2, n // 2] = float("inf")
            X[0, n - 1] = float("nan")
        for i, c in enumerate(places):
            r = (7 * i) % rows
            old = X[r, c].clone()
            X[r, c] = -5.0
            q = gq.gptq_fp4_quantize(X, "nvfp4", row_index=index)
            assert torch.equal(q["tensor_scale"].cpu(), want), (off, pitch, index is not None, c)
            X[r, c] = old


def test_maxima_and_codes_of_calls_in_a_row():
    """Calls that follow one another with one workspace, each other's inputs
    being different, give what each gives alone."""
    Xs = [(_x(700, 512, 20 + i, "bf16") * 10.0 ** i).to(torch.bfloat16).cuda() for i in range(3)]
    alone = []
    for X in Xs:
        alone.append(gq.gptq_fp4_quantize(X, "nvfp4"))
        torch.cuda.synchronize()
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    out = {k: torch.empty_like(alone[0][k]) for k in ("packed", "scales", "tensor_scale")}
    seen = []
    for _ in range(20):
        for X in Xs:
            q = gq.gptq_fp4_quantize(X, "nvfp4", out=out, ws=ws)
            seen.append({k: q[k].clone() for k in out})
    for i, q in enumerate(seen):
        for k in out:
            assert torch.equal(q[k], alone[i % 3][k]), (i, k)


@pytest.mark.parametrize("counts_off", [[0, 400, 300, 700], [0, 100, 701], [-1, 700]])
def test_bad_offsets_of_many_rows_touch_nothing(counts_off):
    X = _x(700, 512, 5, "bf16").cuda()
    out = {"packed": torch.full((700, 256), 0xA5, dtype=torch.uint8, device="cuda")}
    q = gq.gptq_fp4_quantize(X, "nvfp4", offsets=torch.tensor(counts_off, dtype=torch.int32).cuda(), out=out)
    torch.cuda.synchronize()
    assert (q["packed"] == 0xA5).all()
    assert gq.gptq_get_device_status() != 0
    assert gq.gptq_get_device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[5], [0, 3, 0, 0, 130, 1, 0], [128, 128], [1] * 40, [300, 0, 257]])
def test_ragged_groups(fmt, counts):
    rows, n = sum(counts), 272
    X = _x(rows, n, len(counts), "bf16", "outliers")
    scale = torch.rand(rows, 1) * 3 + 0.1
    X = (X.float() * scale).to(torch.bfloat16)
    off = np.concatenate([[0], np.cumsum(counts)])
    q = gq.gptq_fp4_quantize(X.cuda(), fmt, offsets=torch.tensor(off, dtype=torch.int32).cuda(), want_deq=True)
    _compare(q, X, fmt, off)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("groups,size,n", [(1, 200, 96), (3, 130, 64), (8, 1, 4096), (5, 256, 40)])
def test_stacks(fmt, groups, size, n):
    X = _x(groups * size, n, groups, "f32")
    X *= (torch.arange(groups * size) // max(size, 1) + 1)[:, None]
    q = gq.gptq_fp4_quantize(X.reshape(groups, size, n).cuda(), fmt, want_deq=True)
    assert q["groups"] == groups and q["rows"] == groups * size
    _compare(q, X, fmt, np.arange(groups + 1) * size)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,n", [(10, 64), (90, 1032)])
def test_gathered_rows(fmt, tokens, n):
    """The same source row in several places and groups, others in none."""
    X = _x(tokens, n, 2, "bf16")
    idx = torch.randint(0, tokens, (3 * tokens,), generator=torch.Generator().manual_seed(1))
    off = np.array([0, tokens, tokens, 3 * tokens])
    q = gq.gptq_fp4_quantize(X.cuda(), fmt, row_index=idx.int().cuda(),
                             offsets=torch.tensor(off, dtype=torch.int32).cuda(), want_deq=True)
    _compare(q, X[idx], fmt, off)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [64, 9000])
def test_rows_of_no_group_are_left_alone(fmt, n):
    X = _x(20, n, 4, "bf16")
    off = np.array([4, 9, 15])
    out = {"packed": torch.full((20, 16 * ((n + 31) // 32)), 0xA5, dtype=torch.uint8, device="cuda"),
           "deq": torch.full((20, n), 77.0, device="cuda")}
    q = gq.gptq_fp4_quantize(X.cuda(), fmt, offsets=torch.tensor(off, dtype=torch.int32).cuda(), want_deq=True, out=out)
    torch.cuda.synchronize()
    for a, b in ((0, 4), (15, 20)):
        assert (q["packed"][a:b] == 0xA5).all() and (q["deq"][a:b] == 77.0).all()
    codes, byte, t, values = fo.quantize(X[4:15].double().numpy(), fmt, off - 4)
    np.testing.assert_array_equal(q["packed"][4:15].cpu().numpy(), fo.pack(codes, n))
    np.testing.assert_array_equal(q["deq"][4:15].cpu().numpy(), values)


def test_no_rows():
    q = gq.gptq_fp4_quantize(torch.empty((0, 64), device="cuda"), "nvfp4")
    torch.cuda.synchronize()
    assert q["tensor_scale"].item() == 2.0 ** -126
    q = gq.gptq_fp4_quantize(torch.empty((0, 64), device="cuda"), "mxfp4",
                             offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert q["packed"].shape == (0, 32)


@pytest.mark.parametrize("off", [[0, 9, 5, 20], [0, 5, 21, 20], [-1, 5, 9, 20], [0, 5, 9, 21]])
def test_bad_offsets_touch_nothing_and_are_reported(off):
    X = _x(20, 64, 4, "bf16").cuda()
    gq.gptq_get_device_status()
    packed = torch.full((20, 32), 0xA5, dtype=torch.uint8, device="cuda")
    q = gq.gptq_fp4_quantize(X, "nvfp4", offsets=torch.tensor(off, dtype=torch.int32).cuda(), out={"packed": packed})
    assert gq.gptq_get_device_status() == 1
    assert (q["packed"] == 0xA5).all()


def test_bad_row_index_gives_zeros_and_is_reported():
    X = _x(20, 64, 4, "bf16")
    gq.gptq_get_device_status()
    idx = torch.tensor([3, -1, 19, 20, 2 ** 31 - 1], dtype=torch.int32)
    q = gq.gptq_fp4_quantize(X.cuda(), "mxfp4", row_index=idx.cuda(), want_deq=True)
    assert gq.gptq_get_device_status() == 1
    want = torch.zeros((5, 64), dtype=torch.bfloat16)
    want[0], want[2] = X[3], X[19]
    _compare(q, want, "mxfp4")


def test_codes_are_the_same_every_time_and_on_another_stream():
    X = _x(700, 1032, 9, "bf16", "outliers").cuda()
    first = gq.gptq_fp4_quantize(X, "nvfp4", want_deq=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = gq.gptq_fp4_quantize(X, "nvfp4", want_deq=True, stream=side)
    side.synchronize()
    for k in ("packed", "scales", "tensor_scale", "deq"):
        assert torch.equal(first[k], again[k]), k


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(fmt):
    """Over 2^31 values: the last rows like the same rows alone."""
    rows, n = 530000, 4096
    X = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
    X[:-300] = 0.5
    X[-300:] = torch.randn((300, n), device="cuda").to(torch.bfloat16)
    ts = torch.tensor([0.01], device="cuda") if fmt == "nvfp4" else None
    q = gq.gptq_fp4_quantize(X, fmt, tensor_scale=ts)
    tail = gq.gptq_fp4_quantize(X[-(rows % 128 + 128):], fmt, tensor_scale=ts)
    assert torch.equal(q["packed"][-(rows % 128 + 128):], tail["packed"])
    assert torch.equal(q["scales"][-2:], tail["scales"])
    if fmt == "nvfp4":  # and the maximum over all of them
        full = gq.gptq_fp4_quantize(X, fmt)
        assert full["tensor_scale"].item() == (X[-300:].abs().max().float() / torch.tensor(2688.0, device="cuda")).item()


def test_two_streams_at_once():
    Xs = [torch.randn((2000, 1024), device="cuda") * (i + 1) for i in range(2)]
    want = [gq.gptq_fp4_quantize(X, "nvfp4", want_deq=True) for X in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    got = [[gq.gptq_fp4_quantize(X, "nvfp4", want_deq=True, stream=s) for X, s in zip(Xs, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for run in got:
        for a, b in zip(run, want):
            assert all(torch.equal(a[k], b[k]) for k in ("packed", "scales", "tensor_scale", "deq"))


def test_workspace_and_outputs_of_the_caller():
    X = torch.randn((700, 520), device="cuda")
    want = gq.gptq_fp4_quantize(X, "nvfp4", want_deq=True)
    need = gq.LIB.gptq_fp4_quantize_workspace_size(700, 520, 1, 1, 0)
    assert need > 0
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")[3:]
    out = {k: torch.empty_like(want[k]) for k in ("packed", "scales", "tensor_scale", "deq")}
    got = gq.gptq_fp4_quantize(X, "nvfp4", want_deq=True, out=out, ws=ws[:need + 253])
    assert all(got[k].data_ptr() == out[k].data_ptr() and torch.equal(out[k], want[k]) for k in out)
    with pytest.raises(gq.GptqError, match="INVALID_ARG"):
        gq.gptq_fp4_quantize(X, "nvfp4", ws=ws[:need - 1])
    with pytest.raises(ValueError):
        gq.gptq_fp4_quantize(X, "nvfp4", out={"packed": out["packed"][:-1]})
