"""Matrices used in another way than they were grouped: right where the groups
are even, refused elsewhere (test_fp4_grouping_cpu.py has the rules)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import post_weight_quantization_accum_b200 as gq


def _offsets(*bounds):
    return torch.tensor(bounds, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_weights_by_offsets_as_a_stack(fmt):
    gen = torch.Generator("cuda").manual_seed(1)
    W = torch.randn((300, 96), device="cuda", generator=gen)
    X = torch.randn((20, 96), device="cuda", generator=gen)
    off = _offsets(0, 7, 7, 20)
    want = gq.fp4_linear(gq.gptq_fp4_quantize(W.reshape(3, 100, 96), fmt), X, offsets=off)
    even = gq.gptq_fp4_quantize(W, fmt, offsets=_offsets(0, 100, 200, 300))
    assert torch.equal(gq.fp4_linear(even, X, offsets=off), want)
    x = gq.gptq_fp4_quantize(X, fmt, offsets=off)
    assert torch.equal(gq.gptq_fp4_grouped_matmul(even, x, off), want)
    for bad in (_offsets(0, 99, 200, 300), _offsets(0, 100, 200, 299)):
        w = gq.gptq_fp4_quantize(W, fmt, offsets=bad)
        with pytest.raises(ValueError, match="grouped by offsets"):
            gq.fp4_linear(w, X, offsets=off)
        with pytest.raises(ValueError, match="grouped by offsets"):
            gq.gptq_fp4_grouped_matmul(w, x, off)
    assert gq.gptq_get_device_status() == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("tokens", [20, 128, 300])
def test_rows_by_offsets_as_all_rows_and_the_other_way(fmt, tokens):
    gen = torch.Generator("cuda").manual_seed(2)
    W = torch.randn((140, 96), device="cuda", generator=gen)
    X = torch.randn((tokens, 96), device="cuda", generator=gen)
    w, all_rows, part = gq.gptq_fp4_quantize(W, fmt), _offsets(0, tokens), _offsets(5, tokens)
    plain = gq.gptq_fp4_quantize(X, fmt)
    want = gq.gptq_fp4_matmul(w, plain)
    assert torch.equal(gq.gptq_fp4_matmul(w, gq.gptq_fp4_quantize(X, fmt, offsets=all_rows)), want)
    with pytest.raises(ValueError, match="grouped by offsets"):
        gq.gptq_fp4_matmul(w, gq.gptq_fp4_quantize(X, fmt, offsets=part))
    if tokens % 128:  # (else the scales have too few bands for any offsets)
        grouped = gq.gptq_fp4_quantize(X, fmt, offsets=all_rows)
        assert torch.equal(gq.gptq_fp4_grouped_matmul(w, plain, all_rows), gq.gptq_fp4_grouped_matmul(w, grouped, all_rows))
        with pytest.raises(ValueError, match="without the product's offsets"):
            gq.gptq_fp4_grouped_matmul(w, plain, part)
    assert gq.gptq_get_device_status() == 0


def test_offsets_are_read_on_the_call_s_stream_and_not_in_a_capture():
    X = torch.randn((20, 96), device="cuda")
    w = gq.gptq_fp4_quantize(torch.randn((140, 96), device="cuda"), "nvfp4")
    x = gq.gptq_fp4_quantize(X, "nvfp4", offsets=_offsets(0, 20))
    want = gq.gptq_fp4_matmul(w, x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = gq.gptq_fp4_matmul(w, x, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    refused = []
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        try:
            gq.gptq_fp4_matmul(w, x)
        except ValueError as e:
            refused.append(str(e))
        y = gq.gptq_fp4_matmul(w, dict(x, offsets=None))  # (the capture goes on)
    assert len(refused) == 1 and "capture" in refused[0]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
