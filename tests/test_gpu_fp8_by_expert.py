"""GPU tests of the block-scaled FP8 operators by expert: forms of the step that depend on F."""
import pytest
import torch

import skinny_gemm_projection_amd as sg
from gpu_common import DEV, announce
from test_gpu_fp8_block import step_inputs, step_reference, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

# (T, topk, E, H, F, experts drawn from): many rows an expert, gated products stored in fp32
STORED = [(400, 1, 2, 144, 272, 2), (340, 2, 3, 272, 144, 4)]


@pytest.mark.parametrize("T,topk,E,H,F,total", STORED)
def test_step_whose_gated_products_are_stored(T, topk, E, H, F, total):
    announce(f"moe_fp8_step stored T={T} topk={topk} E={E} H={H} F={F}")
    x, ids, w, wgu, sgu, wd, sd, r = step_inputs(T, topk, E, H, F, total)
    want, bound = step_reference(x, ids, w, wgu, sgu, wd, sd, r, E)
    d = [t.to(DEV) for t in (x, ids, w, wgu, sgu, wd, sd)]
    out = sg.skinny_moe_fp8_step(*d, r=r.to(DEV))
    within(out, want, bound, "stored")
    assert torch.equal(sg.skinny_moe_fp8_step(*d, r=r.to(DEV)), out), "repeated calls give identical bits"
