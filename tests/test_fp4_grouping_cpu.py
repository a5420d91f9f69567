"""How a quantised matrix's rows were grouped, without a GPU: a product takes it
only where its scales lie as the product reads them."""
import numpy as np
import pytest
import torch

import post_weight_quantization_accum_b200 as gq
from oracle import fp4_oracle as fo


def _matrix(bounds, n=64, bands=None, **more):
    rows, groups = bounds[-1], len(bounds) - 1
    bands = rows // 128 + groups if bands is None else bands
    return dict({"packed": torch.zeros((rows, 16 * -(-n // 32)), dtype=torch.uint8),
                 "scales": torch.zeros((bands, -(-n // 64), 512), dtype=torch.uint8), "tensor_scale": torch.ones(groups),
                 "rows": rows, "n": n, "format": "nvfp4", "groups": groups}, **more)


def _offsets(*bounds):
    return torch.tensor(bounds, dtype=torch.int32)


def test_groups_that_are_not_even_are_laid_out_in_another_way():
    """Why: the same bytes in groups of 100 and 156 rows, or from row 5 on, lie
    elsewhere than in two groups of 128, or from row 0 on."""
    byte = np.arange(256 * 4, dtype=np.int64).reshape(256, 4).astype(np.uint8)
    even, uneven = fo.scale_tiles(byte, [0, 128, 256]), fo.scale_tiles(byte, [0, 100, 256])
    assert uneven.shape[0] == 3 and not np.array_equal(uneven[:2], even)
    assert np.array_equal(even, fo.scale_tiles(byte, [0, 256]))
    assert not np.array_equal(fo.scale_tiles(byte[5:20], [0, 15]), fo.scale_tiles(byte[:20], [0, 20]))


@pytest.mark.parametrize("call", ["matmul", "grouped", "linear"])
def test_weights_in_uneven_groups_are_no_stack(call):
    def run(w):
        if call == "linear":
            return gq.fp4_linear(w, torch.zeros((12, 64)), offsets=None if w["groups"] == 1 else off)
        if call == "matmul":
            return gq.gptq_fp4_matmul(w, x)
        return gq.gptq_fp4_grouped_matmul(w, x, off)

    one = call == "matmul"
    off = _offsets(0, 4, 12)
    x = _matrix([0, 12]) if one else _matrix([0, 4, 12], offsets=off)
    bounds = [0, 256] if one else [0, 128, 256]
    for bad in ([_offsets(0, 200), _offsets(5, 256)] if one else [_offsets(0, 100, 256), _offsets(0, 128, 255), _offsets(1, 128, 256)]):
        with pytest.raises(ValueError, match="w's rows were grouped by offsets"):
            run(_matrix(bounds, offsets=bad))
    for good in (dict(), dict(offsets=None), dict(offsets=torch.tensor(bounds, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):  # nothing else is wrong with it
            run(_matrix(bounds, **good))


def test_rows_in_a_group_of_their_own_are_not_all_rows():
    w = _matrix([0, 40])
    for bad in (_offsets(5, 20), _offsets(0, 19), _offsets(1, 20)):
        with pytest.raises(ValueError, match="x's rows were grouped by offsets"):
            gq.gptq_fp4_matmul(w, _matrix([0, 20], offsets=bad))
    for good in (dict(), dict(offsets=None), dict(offsets=_offsets(0, 20))):
        with pytest.raises(ValueError, match="CUDA"):
            gq.gptq_fp4_matmul(w, _matrix([0, 20], **good))


def test_rows_without_offsets_are_in_no_other_groups():
    w, w2 = _matrix([0, 40]), _matrix([0, 20, 40])
    x, x2 = _matrix([0, 20], offsets=None), _matrix([0, 10, 20], offsets=None)
    for a, b, off in ((w, x, _offsets(5, 20)), (w, x, _offsets(0, 19)), (w2, x2, _offsets(0, 9, 20)), (w2, x2, _offsets(0, 10, 19))):
        with pytest.raises(ValueError, match="without the product's offsets"):
            gq.gptq_fp4_grouped_matmul(a, b, off)
    for a, b, off in ((w, x, _offsets(0, 20)), (w2, x2, _offsets(0, 10, 20)), (w, _matrix([0, 20]), _offsets(5, 20)),
                      (w, _matrix([0, 20], offsets=_offsets(5, 20)), _offsets(5, 20))):
        with pytest.raises(ValueError, match="CUDA"):
            gq.gptq_fp4_grouped_matmul(a, b, off)
