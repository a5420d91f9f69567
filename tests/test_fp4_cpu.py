"""The 4-bit floating-point operators without a GPU: the oracle's pins (by hand
and by exact fractions), sizes, and the refusals of the C entry points and of
the binding."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import post_weight_quantization_accum_b200 as gq
from oracle import fp4_oracle as fo

P = ctypes.c_void_p
LIB = gq.LIB
MX, NV, F32, BF16 = 0, 1, 0, 1


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------


def test_mxfp4_by_hand():
    """amax 5.0: floor(log2) = 2, scale 2^0.  Ties: 0.25 -> 0, 0.75 -> 1, 1.25 ->
    1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5.0 -> 4.  amax 7.5: scale 1, 7.5 -> 6."""
    x = np.zeros((3, 32))
    x[0, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0]
    x[1, :4] = [7.5, -0.2, 6.0, 4.999]
    x[2, 0] = 0.0625  # scale 2^-6: 4 in units of it
    codes, byte, t, v = fo.quantize(x, "mxfp4")
    assert codes[0, :8].tolist() == [0, 2, 2, 4, 4, 6, 6, 14]
    assert codes[1, :4].tolist() == [7, 8, 7, 6] and v[1, :4].tolist() == [6.0, -0.0, 6.0, 4.0]
    assert byte[:, 0].tolist() == [127, 127, 121] and t is None
    assert codes[2, 0] == 6 and v[2, 0] == 0.0625
    assert fo.quantize(np.zeros((1, 32)), "mxfp4")[1][0, 0] == 0


def test_nvfp4_by_hand():
    """Largest magnitude 2688: t = 1.  Block 0 has it: s = 448, 2688 -> 6.
    Block 1 with amax 12: s = 2, values in units of 2."""
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1] = 2688.0, -1120.0          # -2.5 in units of 448: the tie goes to 2
    x[0, 16], x[0, 17], x[0, 18] = 12.0, 3.4, -0.4
    codes, byte, t, v = fo.quantize(x, "nvfp4")
    assert t.tolist() == [1.0]
    assert byte.tolist() == [[126, 64]]         # 448, 2
    assert codes[0, :2].tolist() == [7, 12] and codes[0, 16:19].tolist() == [7, 3, 8]
    assert v[0, 16:19].tolist() == [12.0, 3.0, -0.0]
    # all zeros: the least tensor scale, zero codes
    codes, byte, t, v = fo.quantize(np.zeros((2, 16)), "nvfp4")
    assert t[0] == 2.0 ** -126 and not codes.any() and not byte.any()


def _nearest_fraction(a, table, unit):
    """Index nearest to a in multiples of unit, ties to even, in exact fractions."""
    best = min(range(len(table)), key=lambda i: (abs(a - table[i] * unit), i % 2))
    return best


@pytest.mark.parametrize("seed", range(4))
def test_oracle_decides_like_exact_fractions(seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((3, 32)).astype(np.float32)
    x = (x.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32) if seed % 2 else x  # bf16 values tie often
    e2m1 = [Fraction(v) for v in fo.E2M1]
    e4m3 = [Fraction(v) for v in fo.E4M3]
    codes, byte, t, _ = fo.quantize(x, "nvfp4")
    ft = Fraction(float(t[0]))
    assert float(t[0]) == np.float32(np.abs(x).max()) / np.float32(2688)
    for r in range(3):
        for b in range(2):
            blk = [Fraction(float(v)) for v in x[r, 16 * b:16 * b + 16]]
            s = _nearest_fraction(max(abs(v) for v in blk), e4m3, 6 * ft)
            assert byte[r, b] == s
            for j, v in enumerate(blk):
                k = _nearest_fraction(abs(v), e2m1, e4m3[s] * ft)
                assert codes[r, 16 * b + j] == k + 8 * (v < 0)


def test_layout_by_hand():
    codes = np.arange(64, dtype=np.uint8).reshape(1, 64) % 16
    p = fo.pack(codes, 33)
    assert p.shape == (1, 32) and p[0, 0] == 0x10 and p[0, 1] == 0x32
    byte = np.zeros((200, 6), dtype=np.uint8)
    byte[0, 0], byte[37, 3], byte[127, 5], byte[130, 4] = 1, 2, 3, 4
    t = fo.scale_tiles(byte, [0, 200])
    assert t.shape == (2, 2, 512)
    assert t[0, 0, 0] == 1
    assert t[0, 0, 16 * 5 + 4 * 1 + 3] == 2     # row 37: row 5 of the second 32
    assert t[0, 1, 16 * 31 + 4 * 3 + 1] == 3    # row 127, block 5
    assert t[1, 1, 16 * 2 + 0] == 4             # row 130: row 2 of the second band
    # a group starts a band: rows 3.. of group 1 are band 1
    t = fo.scale_tiles(byte[:5], [0, 3, 3, 5])
    assert t.shape == (2, 2, 512)


def test_unpack_inverts_quantise():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((150, 75))
    bounds = [0, 20, 20, 150]
    for fmt in ("mxfp4", "nvfp4"):
        codes, byte, t, v = fo.quantize(x, fmt, bounds)
        u = fo.unpack(fo.pack(codes, 75), fo.scale_tiles(byte, bounds), 75, fmt, bounds)
        tt = np.ones(150) if t is None else np.repeat(t.astype(np.float64), np.diff(bounds))
        np.testing.assert_allclose(u * tt[:, None], v, rtol=2.0 ** -24)


# ---------------------------------------------------------------------------
# sizes and refusals of the C entry points
# ---------------------------------------------------------------------------


def test_sizes():
    assert [LIB.gptq_fp4_row_bytes(n) for n in (0, 1, 32, 33, 4096, 65535, 65536)] == [0, 16, 16, 32, 2048, 32768, 0]
    size = LIB.gptq_fp4_scale_bytes
    assert size(1, 4096, NV, 1, 0) == 64 * 512 and size(1, 4096, MX, 1, 0) == 32 * 512
    assert size(129, 64, NV, 1, 0) == 2 * 512 and size(6, 65, NV, 3, 0) == 3 * 2 * 512
    assert size(100, 64, NV, 5, 1) == 5 * 512 and size(300, 64, NV, 5, 1) == 7 * 512
    assert size(7, 64, NV, 2, 0) == 0 and size(7, 64, 2, 1, 0) == 0 and size(-1, 64, NV, 1, 0) == 0
    assert size(7, 64, NV, 513, 1) == 0 and size(7, 0, NV, 1, 0) == 0
    ws = LIB.gptq_fp4_quantize_workspace_size
    assert ws(8192, 4096, MX, 1, 0) == 0 and ws(16, 4096, NV, 1, 0) == 0
    assert ws(8192, 4096, NV, 1, 0) == 64 * 16 * 4   # a maximum a band and chunk of 256 columns
    assert ws(8192, 4096, NV, 24, 1) > 0 and ws(8192, 4096, NV, 600, 1) == 0
    lin = LIB.gptq_fp4_linear_workspace_size
    assert lin(64, 128, 4096, MX, 1, 0) == 64 * 2048 + 32 * 512 + 256
    assert lin(64, 128, 4096, NV, 2, 0) == 0 and lin(0, 128, 4096, NV, 1, 0) == 0


def _quantize(**kw):
    a = dict(X=P(256), xdt=F32, x_rows=8, n=64, ldx=64, index=None, rows=8, offsets=None, groups=1, format=NV, given=0,
             t=P(256), packed=P(256), scales=P(256), deq=None, ws=P(256), ws_bytes=1 << 30)
    a.update(kw)
    return LIB.gptq_fp4_quantize(a["X"], a["xdt"], a["x_rows"], a["n"], a["ldx"], a["index"], a["rows"], a["offsets"],
                                 a["groups"], a["format"], a["given"], a["t"], a["packed"], a["scales"], a["deq"],
                                 a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(xdt=2), dict(format=2), dict(format=-1), dict(n=0), dict(n=65536), dict(ldx=63), dict(rows=-1), dict(x_rows=-1),
    dict(x_rows=7), dict(rows=2 ** 31 - 256, x_rows=2 ** 31 - 256), dict(groups=0), dict(groups=3),
    dict(offsets=P(256), groups=513), dict(offsets=P(258), groups=2), dict(given=2), dict(t=None), dict(t=P(258)),
    dict(format=MX), dict(format=MX, t=None, given=1), dict(X=None), dict(X=P(258)), dict(X=P(257), xdt=BF16),
    dict(packed=None), dict(packed=P(264)), dict(scales=None), dict(scales=P(264)), dict(deq=P(258)), dict(index=P(258)),
    dict(rows=2048, x_rows=2048, ws=None), dict(rows=2048, x_rows=2048, ws=P(128 + 16)),
    dict(rows=2048, x_rows=2048, ws_bytes=4)])
def test_quantize_refuses(bad):
    assert _quantize(**bad) == 1


def test_quantize_of_nothing_and_too_much():
    assert _quantize(rows=0, x_rows=0, X=None, format=MX, t=None, packed=None, scales=None) == 0
    assert _quantize(rows=0, x_rows=0, X=None, given=1, packed=None, scales=None) == 0
    assert _quantize(rows=2 ** 31 - 257, x_rows=2 ** 31 - 257, n=65535, ldx=65535) == 5


def _matmul(grouped=False, **kw):
    a = dict(format=NV, wq=P(256), ws=P(256), wt=P(256), groups=1, rows=64, n=64, xq=P(256), xs=P(256), xt=P(256),
             tokens=8, offsets=P(256), y=P(256), ydt=F32, ldy=64)
    a.update(kw)
    if grouped:
        return LIB.gptq_fp4_grouped_matmul(a["format"], a["wq"], a["ws"], a["wt"], a["groups"], a["rows"], a["n"], a["xq"],
                                           a["xs"], a["xt"], a["tokens"], a["offsets"], a["y"], a["ydt"], a["ldy"], None)
    return LIB.gptq_fp4_matmul(a["format"], a["wq"], a["ws"], a["wt"], a["rows"], a["n"], a["xq"], a["xs"], a["xt"],
                               a["tokens"], a["y"], a["ydt"], a["ldy"], None)


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("bad", [
    dict(format=2), dict(rows=-1), dict(n=0), dict(n=65536), dict(tokens=-1), dict(tokens=2 ** 31 - 256), dict(ydt=2),
    dict(ldy=63), dict(wq=None), dict(wq=P(264)), dict(ws=None), dict(ws=P(264)), dict(xq=None), dict(xq=P(264)),
    dict(xs=None), dict(xs=P(264)), dict(y=None), dict(y=P(258)), dict(y=P(257), ydt=BF16), dict(wt=None), dict(xt=None),
    dict(wt=P(258)), dict(format=MX), dict(rows=2 ** 31, ldy=2 ** 31)])
def test_products_refuse(grouped, bad):
    assert _matmul(grouped, **bad) == 1


def test_grouped_product_refuses_groups():
    for bad in (dict(offsets=None), dict(offsets=P(258)), dict(groups=0), dict(groups=513), dict(groups=512, rows=2 ** 23, ldy=2 ** 23)):
        assert _matmul(True, **bad) == 1, bad
    assert _matmul(False, n=65535, rows=2 ** 31 - 257, ldy=2 ** 31 - 257) == 5  # more scale tiles than TMA has rows


@pytest.mark.parametrize("grouped", [False, True])
def test_products_of_nothing(grouped):
    none = dict(wq=None, ws=None, wt=None, xq=None, xs=None, xt=None, y=None)
    assert _matmul(grouped, tokens=0, **none) == 0
    assert _matmul(grouped, rows=0, **none) == 0


def _linear(**kw):
    a = dict(format=NV, wq=P(256), ws=P(256), wt=P(256), groups=1, rows=64, n=64, X=P(256), xdt=F32, x_rows=300, ldx=64,
             index=None, tokens=300, offsets=None, xt=None, y=P(256), ydt=F32, ldy=64, wsp=P(256), ws_bytes=1 << 30)
    a.update(kw)
    return LIB.gptq_fp4_linear(a["format"], a["wq"], a["ws"], a["wt"], a["groups"], a["rows"], a["n"], a["X"], a["xdt"],
                               a["x_rows"], a["ldx"], a["index"], a["tokens"], a["offsets"], a["xt"], a["y"], a["ydt"],
                               a["ldy"], a["wsp"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(format=2), dict(wq=None), dict(ws=P(264)), dict(wt=None), dict(groups=2), dict(groups=0), dict(rows=-1), dict(n=0),
    dict(X=None), dict(X=P(258)), dict(xdt=3), dict(x_rows=299), dict(ldx=63), dict(index=P(257)), dict(tokens=-1),
    dict(offsets=P(258)), dict(offsets=P(256), groups=600), dict(xt=P(258)), dict(format=MX, wt=None, xt=P(256)),
    dict(y=None), dict(ydt=4), dict(ldy=63), dict(wsp=None), dict(wsp=P(264)), dict(ws_bytes=100)])
def test_linear_refuses(bad):
    assert _linear(**bad) == 1


def test_linear_of_nothing():
    assert _linear(tokens=0, x_rows=0, X=None, y=None, wsp=None) == 0
    assert _linear(rows=0, wq=None, ws=None, y=None, wsp=None) == 0


# ---------------------------------------------------------------------------
# refusals of the binding (host tensors)
# ---------------------------------------------------------------------------


def test_binding_refuses_what_it_cannot_quantise():
    X = torch.zeros((6, 40))
    for err, kw in ((ValueError, dict(format="fp4")), (ValueError, dict(tensor_scale=torch.ones(2))),
                    (TypeError, dict(tensor_scale=torch.ones(1, dtype=torch.float64))),
                    (ValueError, dict(format="mxfp4", tensor_scale=torch.ones(1))),
                    (TypeError, dict(row_index=torch.zeros(3, dtype=torch.int64))),
                    (TypeError, dict(offsets=torch.zeros(3))), (ValueError, dict(offsets=torch.zeros(1, dtype=torch.int32))),
                    (ValueError, dict(offsets=torch.zeros(600, dtype=torch.int32))),
                    (ValueError, dict(offsets=torch.zeros((2, 2), dtype=torch.int32)))):
        with pytest.raises(err):
            gq.gptq_fp4_quantize(X, **kw)
    for bad in (torch.zeros(4), torch.zeros((2, 2, 2, 2)), torch.zeros((4, 0)), torch.zeros((1, 65536)), X.T,
                torch.zeros((3, 4, 8)).transpose(0, 1), torch.zeros(5).expand(4, 5)):
        with pytest.raises(ValueError):
            gq.gptq_fp4_quantize(bad)
    with pytest.raises(TypeError):
        gq.gptq_fp4_quantize(X.half())
    with pytest.raises(ValueError):
        gq.gptq_fp4_quantize(torch.zeros((2, 4, 8)), offsets=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        gq.gptq_fp4_quantize(X)


def _host(rows, n, format="nvfp4", groups=1, bands=None):
    block = 4 * gq.FP4_BLOCK[format]
    bands = groups * -(-(rows // groups) // 128) if bands is None else bands
    return {"packed": torch.zeros((rows, 16 * -(-n // 32)), dtype=torch.uint8),
            "scales": torch.zeros((bands, -(-n // block), 512), dtype=torch.uint8),
            "tensor_scale": torch.ones(groups) if format == "nvfp4" else None, "rows": rows, "n": n, "format": format,
            "groups": groups}


def test_binding_refuses_what_it_cannot_multiply():
    w, x = _host(40, 100), _host(7, 100)
    off = torch.tensor([0, 7], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gq.gptq_fp4_matmul(w, x)
    for bad in (_host(7, 96), _host(7, 100, "mxfp4"), dict(x, rows=8), dict(x, packed=x["packed"][:, ::2]),
                dict(x, packed=x["packed"][:, 1:]), dict(x, scales=x["scales"][:, :1]), dict(x, scales=x["scales"][0]),
                dict(x, tensor_scale=None), dict(x, tensor_scale=torch.ones(2)), dict(x, format="mxfp4"),
                {k: v for k, v in x.items() if k != "groups"}, _host(8, 100, groups=2)):
        with pytest.raises(ValueError):
            gq.gptq_fp4_matmul(w, bad)
    for bad in (dict(x, packed=x["packed"].int()), dict(x, tensor_scale=torch.ones(1, dtype=torch.float64))):
        with pytest.raises(TypeError):
            gq.gptq_fp4_matmul(w, bad)
    with pytest.raises(TypeError):
        gq.gptq_fp4_matmul(w, x, dtype=torch.float16)
    for bad in (torch.zeros((7, 41)), torch.zeros((40, 7)).T, torch.zeros(40).expand(7, 40)):
        with pytest.raises(ValueError):
            gq.gptq_fp4_matmul(w, x, y=bad)
    with pytest.raises(TypeError):
        gq.gptq_fp4_matmul(w, x, y=torch.zeros((7, 40), dtype=torch.float64))
    stack = _host(80, 100, groups=2)
    with pytest.raises(ValueError):
        gq.gptq_fp4_matmul(stack, x)
    with pytest.raises(ValueError):
        gq.gptq_fp4_grouped_matmul(stack, x, off)
    with pytest.raises(TypeError):
        gq.gptq_fp4_grouped_matmul(w, x, off.long())
    with pytest.raises(ValueError):
        gq.gptq_fp4_grouped_matmul(w, _host(300, 100, bands=2), off)  # fewer bands than any offsets may need
    X = torch.zeros((7, 100))
    with pytest.raises(ValueError):
        gq.fp4_linear(w, X[:, :99])
    with pytest.raises(ValueError):
        gq.fp4_linear(stack, X)
    with pytest.raises(ValueError):
        gq.fp4_linear(stack, X, offsets=off)
    with pytest.raises(TypeError):
        gq.fp4_linear(w, X.double())
    with pytest.raises(ValueError, match="CUDA"):
        gq.fp4_linear(w, X)
