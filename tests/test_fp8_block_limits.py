"""The documented limits of the block-scaled FP8 operators, without a GPU: what the size queries
accept the calls accept too."""
import ctypes

import pytest
import torch

import skinny_gemm_projection_amd as sg
from skinny_gemm_projection_amd import _lib

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake device pointers are only passed on a host without a GPU")
A = 0x10000  # aligned, never dereferenced
WORKSPACE, HIP = 5, 7

# (T, topk, E, H, F): the largest of each limit, alone and together
STEPS = [(1 << 17, 32, 8, 16368, 65536), (1 << 17, 32, 4096, 16368, 65536), (1 << 22, 1, 1, 496, 65536),
         (1 << 15, 32, 4096, 65520, 65536), (4096, 6, 4096, 16, 65536), (1, 1, 1, 65536, 16)]


@pytest.mark.parametrize("T,topk,E,H,F", STEPS)
def test_step_takes_what_its_workspace_query_takes(T, topk, E, H, F):
    need = sg.skinny_moe_fp8_step_workspace(T, topk, E, H, F)
    assert need > 0
    s = _lib.SgMoeFp8Step(x=A, topk_ids=A, topk_weights=A, W_gate_up=A, gate_up_scales=A, W_down=A,
                          down_scales=A, out=A, T=T, topk=topk, E=E, H=H, F=F)
    c = _lib.load()
    assert c.skinny_moe_fp8_step(ctypes.byref(s), A, need - 1, None) == WORKSPACE
    assert c.skinny_moe_fp8_step(ctypes.byref(s), None, 0, None) == WORKSPACE


@pytest.mark.parametrize("rows,E,N,K", [(24576, 4096, 1 << 20, 16), (1 << 22, 4096, 1 << 20, 16),
                                        (1 << 22, 1, 1 << 20, 16), (1 << 22, 4096, 1 << 20, 65536)])
@pytest.mark.parametrize("f32", [False, True])
def test_product_by_expert_takes_its_documented_sizes(rows, E, N, K, f32):
    """Nothing is refused: the call gets as far as a launch, which needs a GPU."""
    out = (A, None) if f32 else (None, A)
    assert _lib.load().grouped_skinny_gemm_fp8(rows, rows, E, N, K, A, A, A, A, A, None, 1, *out, None) == HIP
