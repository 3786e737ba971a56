"""GPU test of the experts' step: expert outputs keep fp32 up to the weighted sum."""
import pytest
import torch

import fp8_block_ref as ref
import skinny_gemm_projection_amd as sg
from gpu_common import DEV, announce

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

BF16, F64, I32, U8 = torch.bfloat16, torch.float64, torch.int32, torch.uint8


def nearly_equal_experts(T, F, seed):
    """Two experts whose outputs of some thousands differ by a few, and weights 1 and -1.  Every stage
    is exact: x has one value, a power of two; gates of 32 times it, whose sigmoid is 1; up values
    and W_down's in [1, 2), so that no product lies far below another."""
    H, E = 272, 2
    g = ref.gen(seed)
    x = torch.zeros((T, H))
    x[:, 0] = 2.0 ** torch.randint(0, 3, (T,), generator=g)
    wgu = torch.zeros((E, 2 * F, H), dtype=U8)
    wgu[:, :F, 0] = 0x60  # 32
    wgu[:, F:, 0] = torch.randint(0x38, 0x40, (F,), generator=g).to(U8)  # one up projection for both
    wd = torch.randint(0x38, 0x40, (H, F), generator=g).to(U8).repeat(E, 1, 1)
    at = torch.randint(0, F, (H,), generator=g)
    wd[1, torch.arange(H), at] ^= 1  # an eighth more or less
    one = [torch.ones((E, ref.ceil(2 * F), ref.ceil(H))), torch.ones((E, ref.ceil(H), ref.ceil(F)))]
    ids = torch.tensor([[0, 1]], dtype=I32).repeat(T, 1)
    w = torch.tensor([[1.0, -1.0]]).repeat(T, 1)
    v = 32 * x[:, :1].to(F64) ** 2 * ref.value(wgu[0, F:, 0])
    out = v @ (ref.value(wd[0]) - ref.value(wd[1])).t().contiguous()
    return x.to(BF16), ids, w, wgu, one[0], wd, one[1], out, float((v @ ref.value(wd[0]).t().contiguous()).min())


@pytest.mark.parametrize("F", [128, 144])
@pytest.mark.parametrize("T", [3, 40, 100, 300])
def test_expert_outputs_are_not_rounded_before_their_sum(T, F):
    announce(f"moe_fp8_step of nearly equal experts T={T} F={F}")
    *args, want, least = nearly_equal_experts(T, F, T + F)
    assert float(want.abs().max()) < 2.0 ** -5 * least and float(want.abs().min()) > 0
    for residual in (False, True):
        r = (torch.randint(-8, 9, want.shape, generator=ref.gen(1)).to(BF16)) if residual else None
        out = sg.skinny_moe_fp8_step(*[t.to(DEV) for t in args], r=None if r is None else r.to(DEV))
        y = want if r is None else want + r.to(F64)
        # exact but for the output's own rounding
        assert ((out.cpu().to(F64) - y).abs() <= 2.0 ** -8 * y.abs()).all(), f"residual {residual}"
