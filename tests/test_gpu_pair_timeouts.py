"""Waits that run out at many places of the kernels of CTA pairs: reported, and
the next call is right (the two CTAs give up apart, see test_pair_drain_cpu.py)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import post_weight_quantization_accum_b200 as gq

LIMITS = [0, 200, 1000, 3000, 10000, 30000]


def _cut_short(call, times=4):
    """Runs `call` with short limits; whether one of the runs was cut short."""
    cut = 0
    try:
        for limit in LIMITS * times:
            gq.gptq_set_wait_limit_ns(limit)
            call()
            torch.cuda.synchronize()
            status = gq.gptq_get_device_status()
            assert status in (0, 6)
            cut += status == 6
    finally:
        gq.gptq_set_wait_limit_ns(2 ** 64 - 1)
    return cut


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,rows,n", [(300, 520, 4096), (2100, 9000, 1500), (4096, 8192, 4096)])
def test_product_of_many_tokens(fmt, dtype, tokens, rows, n):
    gen = torch.Generator("cuda").manual_seed(tokens)
    w = gq.gptq_fp4_quantize(torch.randn((rows, n), device="cuda", generator=gen), fmt)
    x = gq.gptq_fp4_quantize(torch.randn((tokens, n), device="cuda", generator=gen), fmt)
    want = gq.gptq_fp4_matmul(w, x, dtype=dtype)
    assert gq.gptq_get_device_status() == 0
    assert _cut_short(lambda: gq.gptq_fp4_matmul(w, x, dtype=dtype)) > 0
    assert torch.equal(want, gq.gptq_fp4_matmul(w, x, dtype=dtype))
    assert gq.gptq_get_device_status() == 0


@pytest.mark.parametrize("tokens,n", [(4096, 1024), (20000, 2048)])
def test_hessian(tokens, n):
    X = torch.randn((tokens, n), device="cuda", generator=torch.Generator("cuda").manual_seed(n)).to(torch.bfloat16)

    def call():
        return gq.gptq_hessian_accum(torch.zeros((n, n), device="cuda"), X, 2.0 / tokens)

    want = call()
    assert gq.gptq_get_device_status() == 0
    assert _cut_short(call) > 0
    assert torch.equal(want, call())
    assert gq.gptq_get_device_status() == 0
