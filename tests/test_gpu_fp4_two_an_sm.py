"""A layer on few tokens whose CTAs hold eight stages of them and share an SM:
the bits of quantising and multiplying in two calls, in a graph too."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import post_weight_quantization_accum_b200 as gq


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,n,rows", [(1, 4096, 14336), (4, 4096, 14300), (1, 14336, 5120), (1, 14001, 5100), (3, 4000, 16385)])
def test_linear_equals_quantise_and_product(fmt, dtype, tokens, n, rows):
    gen = torch.Generator("cuda").manual_seed(n)
    w = gq.gptq_fp4_quantize(torch.randn((rows, n), device="cuda", generator=gen) * 0.02, fmt)
    X = torch.randn((tokens, n), device="cuda", generator=gen).to(dtype)
    want = gq.gptq_fp4_matmul(w, gq.gptq_fp4_quantize(X, fmt))
    for _ in range(3):
        assert torch.equal(gq.fp4_linear(w, X, dtype=torch.float32), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = gq.fp4_linear(w, X, dtype=torch.float32)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert gq.gptq_get_device_status() == 0


def test_waits_that_run_out():
    w = gq.gptq_fp4_quantize(torch.randn((14336, 4096), device="cuda") * 0.02, "nvfp4")
    X = torch.randn((2, 4096), device="cuda")
    want = gq.fp4_linear(w, X)
    gq.gptq_get_device_status()
    try:
        gq.gptq_set_wait_limit_ns(0)
        gq.fp4_linear(w, X)
        torch.cuda.synchronize()
    finally:
        gq.gptq_set_wait_limit_ns(2 ** 64 - 1)
    assert gq.gptq_get_device_status() == 6
    assert torch.equal(gq.fp4_linear(w, X), want)
    assert gq.gptq_get_device_status() == 0
