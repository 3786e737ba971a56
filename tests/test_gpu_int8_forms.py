"""GPU tests of the 8-bit integer operators at the places their other tests leave out: the
accuracy of the gated product, the kernel forms that long prompts use, every form of a product
that takes two launches or splits K, and sizes on both sides of the borders between them."""
import pytest
import torch

import int8_ref as ref
import skinny_gemm_projection_amd as sg
from gpu_common import DEV, announce, counters_delta
from int8_forms import BLOCKS, PRODUCTS, SPLITS, form
from test_gpu_int8 import (check_norm, check_quant, mlp_inputs, norm_inputs, parts, product_inputs,
                           same)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

BF16 = torch.bfloat16
EPS = 1e-6


# ------------------------------------------------------------------ gated product


@pytest.mark.parametrize("lo,hi", [(-87, -80), (-80, -40), (-40, -20), (-20, -10), (-10, -3), (-3, 0),
                                   (0, 3), (3, 10), (10, 90), (90, 300)])
def test_gated_product_error_does_not_grow_with_the_gate(lo, hi):
    """Rows of one gate and one up value: the scale is the gated product / 127.  exp(-|gate|) is
    off by 3 u (one step of the hardware's exponential, 2 u, and one rounding), the sum, product,
    quotient and product with up round once each (4 u), the scale once more."""
    announce(f"gated product {lo}..{hi}")
    g = torch.rand(20000, generator=torch.Generator().manual_seed(lo + 100)) * (hi - lo) + lo
    for u in (1.0, -0.7, 1.0e4):
        x = torch.cat([g[:, None].expand(-1, 8), torch.full((g.numel(), 8), u)], dim=1).contiguous()
        codes, scales = sg.skinny_quant_int8(x.to(DEV), gated=True)
        want = (g.double() * torch.sigmoid(g.double()) * x[:, 8].double()).abs()
        err = (scales.cpu().double() * 127.0 - want).abs()
        worst = (err / want.clamp_min(1e-300)).max().item() / ref.U
        assert (err <= 8 * ref.U * want).all(), f"u = {u}: {worst:.1f} u"
        assert (codes.abs() == 127).all()


def test_gated_product_at_the_ends():
    """Gates of both zeros, the smallest and largest numbers, below -87 and of both infinities."""
    tiny, top = 2.0 ** -149, torch.finfo(torch.float32).max
    g = torch.tensor([0.0, -0.0, tiny, -tiny, top, -top, -104.0, -300.0, float("inf"), float("-inf"),
                      float("nan")])
    x = torch.cat([g[:, None].expand(-1, 8), torch.ones(g.numel(), 8)], dim=1).contiguous()
    codes, scales = [t.cpu() for t in sg.skinny_quant_int8(x.to(DEV), gated=True)]
    assert (codes[:2] == 0).all() and (scales[:2] == 0).all()
    assert (scales[2:4] == 0).all()  # 2^-150 and its 127th are below half of the smallest number
    # (top / 127 is one rounding)
    assert (codes[4] == 127).all() and abs(scales[4].item() * 127.0 / top - 1) <= 2 * ref.U
    assert (codes[5:8] == 0).all() and (scales[5:8] == 0).all()
    assert (codes[8:] == 0).all() and torch.isnan(scales[8:]).all()


# ------------------------------------------------------------------ norm


def test_norm_with_the_smallest_eps():
    """eps = 2^-126 and rows whose squares are below the normal range: adding a square is off by
    at most 2^-150 there, so the mean by that and by as much again in its own rounding: 2 u of
    eps, u after the root."""
    K, eps = 1032, 2.0 ** -126
    x = torch.randn((60, K), generator=torch.Generator().manual_seed(3))
    x = (x * 10.0 ** -(17 + torch.arange(60)[:, None] / 6.0)).to(BF16)
    g = torch.ones(K, dtype=BF16)
    y = torch.empty((60, K), dtype=BF16, device=DEV)
    _, _, codes, scales = sg.skinny_rmsnorm(x.to(DEV), g.to(DEV), eps, y_bf16=y,
                                            codes=torch.empty((60, K), dtype=torch.int8, device=DEV))
    inv, y64 = ref.norm64(x, None, g, eps)
    rel = ref.norm_rel(K) + ref.U
    bound = (2.0 ** -8 + rel + 3 * ref.U) * y64.abs() + 2.0 ** -133
    assert ((y.cpu().double() - y64).abs() <= bound).all()
    want, amax, _ = ref.codes_of(x.float())
    assert torch.equal(codes.cpu(), want)
    s64 = amax.double() * inv / 127.0
    assert ((scales.cpu().double() - s64).abs() <= (rel + 3 * ref.U) * s64).all()


# ------------------------------------------------------------------ row kernels of long prompts

# rows of 2056..8192 values take 1024 threads each below 256 rows and 256 threads from there on
LONG_K = [2056, 4096, 4104, 7168, 8192]


@pytest.mark.parametrize("K", LONG_K)
def test_norm_on_both_sides_of_256_rows(K):
    announce(f"rmsnorm 255..257 x {K}")
    x, r, g = norm_inputs(257, K, 20 + K)
    dx, dr, dg = x.to(DEV), r.to(DEV), g.to(DEV)
    got = {}
    for M in (255, 256, 257):
        h, y = torch.empty_like(dx[:M]), torch.empty_like(dx[:M])
        codes = torch.full((M + 1, K), 99, dtype=torch.int8, device=DEV)
        scales = torch.full((M + 1,), -7.0, device=DEV)
        sg.skinny_rmsnorm(dx[:M], dg, EPS, r=dr[:M], h=h, y_bf16=y, codes=codes[:M], scales=scales[:M])
        check_norm(x[:M], r[:M], g, EPS, h, y, codes[:M], scales[:M], f"M={M} K={K}")
        assert (codes[M] == 99).all() and scales[M] == -7.0
        got[M] = h, codes[:M]
        hr, yx = dr[:M].clone(), dx[:M].clone()  # h over r, y over x
        sg.skinny_rmsnorm(yx, dg, EPS, r=hr, h=hr, y_bf16=yx)
        same(hr, h, "h in place"), same(yx, y, "y in place")
        y2 = torch.empty_like(y)  # bf16 alone, no residual
        sg.skinny_rmsnorm(dx[:M], dg, EPS, y_bf16=y2)
        check_norm(x[:M], None, g, EPS, None, y2, None, None, "bf16 alone")
    for M in (255, 256):  # a row's h and codes do not depend on the batch
        same(got[M][0], got[257][0][:M], "h"), same(got[M][1], got[257][1][:M], "codes")


@pytest.mark.parametrize("K", LONG_K)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_quant_on_both_sides_of_256_rows(K, f32, gated):
    announce(f"quant_int8 255..257 x {K} f32={f32} gated={gated}")
    x = torch.randn((257, 2 * K if gated else K), generator=torch.Generator().manual_seed(K)) * 2
    x[3, 5], x[256, K - 1] = float("nan"), float("inf")
    x[7] = 0
    x = x if f32 else x.to(BF16)
    got = {}
    for M in (255, 256, 257):
        codes = torch.full((M + 1, K), 99, dtype=torch.int8, device=DEV)
        scales = torch.full((M + 1,), -7.0, device=DEV)
        sg.skinny_quant_int8(x[:M].to(DEV), gated, codes[:M], scales[:M])
        check_quant(x[:M], gated, codes[:M], scales[:M], f"M={M} K={K}")
        assert (codes[M] == 99).all() and scales[M] == -7.0
        got[M] = codes[:M], scales[:M]
    for M in (255, 256):
        same(got[M][0], got[257][0][:M], "codes"), same(got[M][1], got[257][1][:M], "scales")


# ------------------------------------------------------------------ forms of the product


def check_product(M, N, K, launches):
    cpu, d = product_inputs(M, N, K, 5)
    r = torch.randn((M, N), generator=torch.Generator().manual_seed(9)).to(BF16)
    flat32 = torch.full((M * N + 16,), -7.0, device=DEV)
    flat16 = torch.full((M * N + 16,), -7.0, device=DEV, dtype=BF16)
    before = sg.skinny_gemm_get_counters()
    sg.skinny_gemm_int8(*d, r=r.to(DEV), y_f32=flat32[:M * N].view(M, N), y_bf16=flat16[:M * N].view(M, N))
    torch.cuda.synchronize()
    ran = counters_delta(before, sg.skinny_gemm_get_counters())
    assert (ran[sg.SG_KERNEL_INT8], ran[sg.SG_KERNEL_REDUCE]) == launches
    want = ref.linear(*cpu, r)
    for flat, t in ((flat32, torch.float32), (flat16, BF16)):
        same(flat[:M * N].view(M, N), want.to(t), str(t))
        assert (flat[M * N:] == -7.0).all(), f"{t}: behind the last element"
    y, _ = sg.skinny_gemm_int8(*d)
    same(y, ref.linear(*cpu), "no residual")
    return cpu, d


@pytest.mark.parametrize("M,N,K,kind", PRODUCTS)
def test_products_of_two_launches(M, N, K, kind):
    """Whole rounds of the largest tiles, then the other columns in tiles of each smaller size."""
    announce(f"int8 M={M} N={N} K={K}: {kind}")
    assert form(M, N, K) == kind
    check_product(M, N, K, (2, 0))


@pytest.mark.parametrize("M,N,K,kind", SPLITS)
def test_products_split_between_workgroups(M, N, K, kind):
    """Every tile size with its K split: the workspace is needed, long enough, and not overrun."""
    announce(f"int8 M={M} N={N} K={K}: {kind}")
    need = sg.skinny_gemm_int8_workspace(M, N, K)
    assert form(M, N, K) == kind and need > 0
    cpu, d = check_product(M, N, K, (1, 1))
    want = ref.linear(*cpu)
    for fill in (0, 255):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
        y, _ = sg.skinny_gemm_int8(*d, workspace=ws)
        same(y, want, f"workspace of {fill}")
        assert (ws[need:] == fill).all()
    before = sg.skinny_gemm_get_counters()
    with pytest.raises(sg.SkinnyGemmError) as e:
        sg.skinny_gemm_int8(*d, workspace=torch.empty(need - 16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5
    assert counters_delta(before, sg.skinny_gemm_get_counters()) == [0] * sg.SG_NUM_COUNTERS


@pytest.mark.parametrize("M,H,F,kind", BLOCKS)
def test_gated_products_of_two_launches(M, H, F, kind):
    """The MLP block with the gated product in the epilogues of two launches gives the bits of the
    public calls one after the other, and those are the references'."""
    announce(f"mlp M={M} H={H} F={F}: {kind}")
    assert form(M, 2 * F, H) == kind
    cpu = mlp_inputs(M, H, F, 40 + M)
    x, r, g, wgu, sgu, wd, sd = [t.to(DEV) for t in cpu]
    q, sq, u, p, sp, h, want = parts(x, r, g, wgu, sgu, wd, sd)
    same(sg.skinny_mlp_int8_step(x, g, EPS, wgu, sgu, wd, sd, r=r), want, "step")
    same(u, ref.linear(q.cpu(), sq.cpu(), cpu[3], cpu[4]), "gate and up")
    check_quant(u.cpu(), True, p, sp, "gated codes")
    same(want, ref.linear(p.cpu(), sp.cpu(), cpu[5], cpu[6], h.cpu()).to(BF16), "down")
