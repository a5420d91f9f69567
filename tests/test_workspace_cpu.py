"""Workspaces that a caller gives, without a GPU: what a call's kernels could
not write, or would write past the end of, is refused before the device is
touched (host tensors stand for the call's, "meta" for another device)."""
import pytest
import torch

import post_weight_quantization_accum_b200 as gq
from post_weight_quantization_accum_b200._lib import aligned_workspace

ELSEWHERE = torch.empty(1 << 20, dtype=torch.uint8, device="meta")
STRIDED = torch.zeros(1 << 20, dtype=torch.uint8)[::2]
EXPANDED = torch.zeros(1, dtype=torch.uint8).expand(1 << 20)


def _calls():
    """name -> (call with a workspace, the LIB entry that must not be reached)"""
    H = torch.eye(64)
    X = torch.zeros((128, 64), dtype=torch.bfloat16)
    W = torch.zeros((8, 64))
    packed = torch.zeros((8, 8), dtype=torch.int32)
    w = {"packed": torch.zeros((8, 32), dtype=torch.uint8), "scales": torch.zeros((1, 1, 512), dtype=torch.uint8),
         "tensor_scale": torch.ones(1), "rows": 8, "n": 64, "format": "nvfp4", "groups": 1}
    return {
        "gptq_hessian_accum": lambda ws: gq.gptq_hessian_accum(H, X, 1.0, ws=ws),
        "gptq_prepare_hinv": lambda ws: gq.gptq_prepare_hinv(H, 0.01, False, ws=ws),
        "gptq_quantize_layer": lambda ws: gq.gptq_quantize_layer(W, H, 4, 32, ws=ws),
        "gptq_dequant_matvec": lambda ws: gq.gptq_dequant_matvec(packed, torch.ones((8, 2)), torch.zeros((8, 2), dtype=torch.uint8),
                                                                 64, 4, 32, torch.zeros((8, 64), dtype=torch.bfloat16), ws=ws),
        "gptq2d_round": lambda ws: gq.gptq2d_round(W, torch.eye(8), H, ws=ws),
        "gptq_fp4_quantize": lambda ws: gq.gptq_fp4_quantize(W, "nvfp4", ws=ws),
        "gptq_fp4_linear": lambda ws: gq.fp4_linear(w, X, ws=ws),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
@pytest.mark.parametrize("ws", [ELSEWHERE, STRIDED, EXPANDED], ids=["elsewhere", "strided", "expanded"])
def test_a_workspace_that_cannot_be_one_is_refused(name, ws, monkeypatch):
    call = _calls()[name]
    monkeypatch.setattr(gq.LIB, "gptq_matvec_workspace_size", lambda *a: 256)
    for entry in _calls():
        monkeypatch.setattr(gq.LIB, entry, lambda *a, entry=entry: pytest.fail(f"{entry} was called"))
    with pytest.raises(ValueError, match="ws must be"):
        call(ws)


def test_a_workspace_counts_its_bytes_from_the_aligned_address():
    base = torch.zeros(4096, dtype=torch.uint8)
    start = -base.data_ptr() % 256
    for off, size in ((0, 1024), (1, 1024), (255, 300), (1, 100), (1, 255), (0, 0), (17, 0)):
        p, n = aligned_workspace(base[start + off:start + off + size])
        assert p % 256 == 0 and n == max(0, size - (-off % 256))
    assert aligned_workspace(torch.zeros(64, dtype=torch.float32)[:64])[1] >= 0
    f = base[start:start + 1024].view(torch.float32)
    assert aligned_workspace(f) == (f.data_ptr(), 1024)


def test_a_matrix_has_groups():
    w = {"packed": torch.zeros((8, 32), dtype=torch.uint8), "scales": torch.zeros((1, 1, 512), dtype=torch.uint8),
         "tensor_scale": torch.ones(1), "rows": 8, "n": 64, "format": "nvfp4", "groups": 1}
    gq.fp4_check_matrix(w, "w")
    for groups in (0, -1):
        for ragged in (False, True):
            with pytest.raises(ValueError, match="group"):
                gq.fp4_check_matrix(dict(w, groups=groups), "w", ragged)
    off = torch.tensor([0, 8], dtype=torch.int32)
    with pytest.raises(ValueError, match="lacks 'groups'"):
        gq.gptq_fp4_grouped_matmul({k: v for k, v in w.items() if k != "groups"}, w, off)
    with pytest.raises(ValueError, match="offsets"):
        gq.gptq_fp4_grouped_matmul(w, w, None)
