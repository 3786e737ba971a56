"""Sizes that would wrap around in the C ABI's int32 are refused by the binding of the product by
expert (CPU: nothing reaches the library)."""
import pytest
import torch

import skinny_gemm_projection_amd as sg


@pytest.mark.parametrize("topk", [0, -1, 2 ** 31, 2 ** 32 + 1])
def test_topk_past_int32(topk):
    u8, w = torch.zeros((8, 64), dtype=torch.uint8), torch.zeros((8, 2))
    ids = torch.zeros((8,), dtype=torch.int32)
    with pytest.raises(ValueError, match="topk"):
        sg.grouped_skinny_gemm_fp8(u8, w, u8[None], w, ids, sorted_pairs=ids, topk=topk)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")
def test_pairs_past_int32():
    f = dict(device="cuda")
    u8 = torch.zeros((2, 16), dtype=torch.uint8, **f)
    pairs = torch.zeros((1,), dtype=torch.int32, **f).expand(2 ** 32 + 8)  # a view of one element
    with pytest.raises(ValueError, match="pairs are past"):
        sg.grouped_skinny_gemm_fp8(u8, torch.ones((1, 2), **f), torch.zeros((1, 1, 16), dtype=torch.uint8, **f),
                                   torch.ones((1, 1, 1), **f), torch.zeros((2,), dtype=torch.int32, **f),
                                   sorted_pairs=pairs, y_f32=torch.empty((8, 1), **f))
