"""GPU tests of the block-scaled FP8 operators by expert: forms of the step that depend on F, and
launches of more tiles than one grid dimension takes."""
import pytest
import torch

import fp8_block_ref as ref
import skinny_gemm_projection_amd as sg
from gpu_common import DEV, announce
from test_gpu_fp8_block import step_inputs, step_reference, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

BF16, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8

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


# ------------------------------------------------------------------ more than 65536 tiles of a launch


def on_device(rows, cols, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = torch.randint(0, 256, (rows, cols), generator=g, device=DEV, dtype=U8)
    c &= 0xbf  # no code past 1.875, no NaN
    return c


VALUE = ref.value(torch.arange(256, dtype=U8))


def close(got, x, w, f, K, wide, what):
    """Every output against 64 bits, on the GPU; f: the scales' product, [rows, channels]."""
    table = VALUE.to(DEV)
    xv, wv = table[x.long()], table[w.long()].t().contiguous()
    y, A = xv @ wv * f, xv.abs() @ wv.abs() * f
    bound = (ref.wide_rel(K) if wide else ref.fp8_rel(K)) * A
    if got.dtype is BF16:
        bound = bound + 2.0 ** -8 * (y.abs() + bound)
    assert bool(((got.to(F64) - y).abs() <= bound).all()), what


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_product_of_many_tiles(dtype):
    M, N, K = 20011, 250007, 16
    announce(f"product {M} x {N} x {K} {dtype}")
    xq, wq = on_device(M, K, 1), on_device(N, K, 2)
    xs, ws = ref.rand_scales((1, M), 3).to(DEV), ref.rand_scales((ref.ceil(N), 1), 4).to(DEV)
    out = torch.full((M, N), float("nan"), dtype=dtype, device=DEV)
    sg.skinny_gemm_fp8_block(xq, xs, wq, ws, **{"y_f32" if dtype is F32 else "y_bf16": out})
    wf = ws.double().repeat_interleave(128, 0)[:N, 0]
    for m in range(0, M, 1000):
        s = slice(m, m + 1000)
        close(out[s], xq[s], wq, xs[0, s].double()[:, None] * wf, K, dtype is F32, f"rows {m}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_product_by_expert_of_many_tiles(dtype):
    rows, E, N, K = 2100, 300, 65501, 16
    announce(f"grouped {rows} x {E} x {N} x {K} {dtype}")
    assert (rows // 64 + E) * ref.ceil(N, 256) > 65536
    sizes = torch.randint(0, 13, (E,), generator=ref.gen(1))
    sizes[7], sizes[8] = 0, 70
    ends = sizes.cumsum(0).clamp(max=rows - 5)
    offsets = torch.cat([torch.zeros(1), ends]).to(I32)
    xq, wq = on_device(rows, K, 1), on_device(E * N, K, 2).view(E, N, K)
    xs, ws = ref.rand_scales((1, rows), 3).to(DEV), ref.rand_scales((E, ref.ceil(N), 1), 4).to(DEV)
    out = torch.full((rows, N), -7.0, dtype=dtype, device=DEV)
    sg.grouped_skinny_gemm_fp8(xq, xs, wq, ws, offsets.to(DEV),
                               **{"y_f32" if dtype is F32 else "y_bf16": out})
    for e in range(E):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        f = xs[0, s].double()[:, None] * ws[e].double().repeat_interleave(128, 0)[:N, 0]
        close(out[s], xq[s], wq[e], f, K, dtype is F32, f"expert {e}")
    assert bool((out[int(offsets[E]):] == -7.0).all())


def test_step_of_many_tiles():
    """Against the same tokens a quarter of the experts at a time, whose tiles fit 65536."""
    T, E, H, F = 2100, 300, 16, 65536
    announce(f"moe_fp8_step T={T} E={E} H={H} F={F}")
    assert (T // 64 + E) * ref.ceil(2 * F, 256) > 65536 > (T // 4 // 64 + E // 4) * ref.ceil(2 * F, 256)
    part = E // 4
    ids = torch.randint(0, part, (T, 1), generator=ref.gen(1), dtype=I32)
    ids += part * (torch.arange(T) // (T // 4))[:, None].to(I32)
    x = torch.randn((T, H), generator=ref.gen(2)).to(BF16).to(DEV)
    w = torch.rand((T, 1), generator=ref.gen(3)).to(DEV)
    wgu, wd = on_device(E * 2 * F, H, 4).view(E, 2 * F, H), on_device(E * H, F, 5).view(E, H, F)
    sgu, sd = ref.rand_scales((E, 2 * F // 128, 1), 6).to(DEV), ref.rand_scales((E, 1, F // 128), 7).to(DEV)
    out = sg.skinny_moe_fp8_step(x, ids.to(DEV), w, wgu, sgu, wd, sd)
    for q in range(4):
        t, e = slice(q * T // 4, (q + 1) * T // 4), slice(q * part, (q + 1) * part)
        want = sg.skinny_moe_fp8_step(x[t], (ids[t] - q * part).to(DEV), w[t], wgu[e], sgu[e], wd[e], sd[e])
        assert torch.equal(out[t], want), f"quarter {q}"
    assert bool((out.float().abs().amax(1) > 0).all())
