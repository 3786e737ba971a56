"""GPU tests of the block-scaled FP8 operators through the public binding: skinny_quant_fp8,
skinny_gemm_fp8_block, grouped_skinny_gemm_fp8 and skinny_moe_fp8_step, against the references of
fp8_block_ref.py in 64 bits."""
import pytest
import torch

import fp8_block_ref as ref
import skinny_gemm_projection_amd as sg
from fp8_block_forms import FORMS
from gpu_common import DEV, announce, counters_delta

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def normal(shape, seed, sigma=1.0, dtype=BF16):
    return (torch.randn(shape, generator=ref.gen(seed)) * sigma).to(dtype)


def within(got, want, bound, what):
    g, want = got.detach().cpu().to(F64), want.to(F64)
    assert g.shape == want.shape, what
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN in other places"
    err = torch.where(nan, 0.0, (g - want).abs())
    bad = ~(err <= torch.where(nan, 0.0, bound))
    if bad.any():
        i = int(torch.argmax(torch.where(bad, err / bound.clamp_min(1e-300), torch.zeros_like(err))))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, worst at "
                             f"{i}: {err.flatten()[i]:.3e} > {bound.flatten()[i]:.3e}")


# ------------------------------------------------------------------ quantiser

QUANT = [(1, 8), (1, 128), (1, 136), (3, 120), (2, 7168), (5, 512), (5, 520), (7, 1000), (64, 18432),
         (61, 2048), (257, 264), (511, 136), (512, 1032), (513, 128), (1030, 520), (2051, 2056), (4, 65536)]


def check_quant(codes, scales, q, s, what):
    got = ref.value(codes.cpu())
    assert torch.equal(got, q), f"{what}: {int((got != q).sum())} codes of {q.numel()} differ"
    want = s.to(F32)
    same = (scales.cpu() == want) | (torch.isnan(scales.cpu()) & torch.isnan(want))
    assert same.all(), f"{what}: scales"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K", QUANT)
def test_quant_codes(M, K, dtype):
    announce(f"quant_fp8 {M} x {K} {dtype}")
    x = normal((M, K), M + K, dtype=F32)
    x[:, 3::97] *= 30
    x[0, ::5] *= 2.0 ** -12  # codes below the normal range
    x = x.to(dtype)
    guard = torch.full((M + 2, K), 9, dtype=torch.uint8, device=DEV)
    before = sg.skinny_gemm_get_counters()
    codes, scales = sg.skinny_quant_fp8(x.to(DEV), codes=guard[:M])
    ran = counters_delta(before, sg.skinny_gemm_get_counters())
    assert ran[sg.SG_KERNEL_QUANT_FP8] == 1 and sum(ran) == 1
    assert scales.shape == (ref.ceil(K), M)
    check_quant(codes, scales, *ref.quant(x), f"{M} x {K}")
    assert (guard[M:] == 9).all(), "rows behind the last are left as they were"


@pytest.mark.parametrize("M,K", [(2, 16), (9, 392), (600, 256)])
def test_quant_borders(M, K):
    """Zero blocks, blocks at the edges of fp32, every halfway case of the codes, values that are
    not finite, and maxima on both sides of 448 times a power of two."""
    x = torch.zeros((M, K))
    v = ref.value(torch.arange(0, 127, dtype=torch.uint8))  # and halfway between neighbours:
    mid = ((v[1:] + v[:-1]) / 2).to(F32)
    x[0, :min(K, 126)] = mid[:min(K, 126)]
    x[0, 0] = 448.0
    x[1, :8] = torch.tensor([2.0 ** -149, -2.0 ** -140, 2.0 ** -133, 0.0, -0.0, 2.0 ** -149, 0, 0])
    if M > 2 and K > 256:
        x[2, 5], x[2, 130], x[2, 260] = float("nan"), float("inf"), -float("inf")
        x[3] = torch.finfo(F32).max
        x[4, :128], x[4, 128:256] = 448.0, 448.00003
        x[5, :128], x[5, 128:256] = -0.4375, 0.43750003
        x[6] = 2.0 ** -126 * 448
        x[7] = 2.0 ** -127 * 448
        x[8] = -3e38
    codes, scales = sg.skinny_quant_fp8(x.to(DEV))
    check_quant(codes, scales, *ref.quant(x), "borders")
    if M > 2 and K > 256:
        assert torch.isnan(scales[:3, 2]).all() and not torch.isnan(scales[:3, 1]).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K", [(1, 8), (3, 136), (61, 2048), (64, 18432), (700, 520), (1029, 128)])
def test_quant_gated(M, K, dtype):
    """The gated product is off by at most 7 * 2^-24, so a code is one of those that the ends of
    that interval round to."""
    announce(f"quant_fp8 gated {M} x {K} {dtype}")
    x = normal((M, 2 * K), M + K, 2.0, dtype)
    codes, scales = sg.skinny_quant_fp8(x.to(DEV), gated=True)
    v, s = ref.gated(x), scales.cpu().to(F64)
    t = ref.blocks(v).abs().amax(dim=2).t()
    lo, hi = ref.unit_of(t * (1 - ref.GATED_REL)), ref.unit_of(t * (1 + ref.GATED_REL))
    assert ((s == lo) | (s == hi)).all()
    unit = s.t().repeat_interleave(ref.B, 1)[:, :K]
    got, a = ref.value(codes.cpu()), v / unit
    e = a.abs() * ref.GATED_REL
    low, high = ref.nearest((a - e).clamp(-448, 448)), ref.nearest((a + e).clamp(-448, 448))
    assert ((got >= low) & (got <= high)).all()
    assert ((got != ref.nearest(a.clamp(-448, 448))).double().mean() < 1e-3)


# ------------------------------------------------------------------ product

GEMM = [(1, 1, 16), (1, 40, 16), (1, 129, 112), (1, 1024, 1024), (2, 300, 4128), (3, 70, 2064),
        (4, 257, 8192), (5, 17, 48), (7, 1000, 80), (8, 16, 128), (11, 300, 7168), (15, 31, 144),
        (16, 129, 2064), (16, 2048, 1040), (17, 200, 1040), (31, 130, 272), (32, 300, 4112),
        (33, 64, 16), (47, 257, 2064), (48, 1000, 2048), (61, 333, 7168), (64, 33, 16384), (64, 1, 144),
        (65, 130, 192), (96, 500, 1008), (100, 1000, 4096), (128, 128, 128), (129, 255, 160),
        (200, 37, 9008), (255, 257, 640), (256, 256, 2048), (257, 513, 144), (300, 1001, 2064),
        (511, 1030, 528), (513, 5, 272), (700, 777, 1040), (1025, 1281, 256), (2049, 300, 528),
        (1000, 2051, 1040), (65, 8195, 400), (129, 6147, 1040), (400, 16390, 144)]


@pytest.mark.parametrize("M,N,K", GEMM + list(dict.fromkeys(f[:3] for f in FORMS)))
def test_gemm(M, N, K):
    announce(f"fp8_block M={M} N={N} K={K}")
    make = ref.any_codes if (M + N) % 3 == 0 else ref.rand_codes
    xq, wq = make(M, K, 1 + M), make(N, K, 2 + N)
    kb = ref.ceil(K)
    xs, ws = ref.rand_scales((kb, M), 3), ref.rand_scales((ref.ceil(N), kb), 4)
    r = normal((M, N), 5)
    d = [t.to(DEV) for t in (xq, xs, wq, ws, r)]
    y, A = ref.product(xq, xs, wq, ws)
    guard = torch.full((M + 3, N), -7.0, device=DEV)
    y32, y16 = guard[:M], torch.full((M, N), -7.0, device=DEV, dtype=BF16)
    before = sg.skinny_gemm_get_counters()
    sg.skinny_gemm_fp8_block(*d[:4], y_f32=y32, y_bf16=y16)
    torch.cuda.synchronize()
    ran = counters_delta(before, sg.skinny_gemm_get_counters())
    assert ran[sg.SG_KERNEL_FP8_BLOCK] in (1, 2)
    assert ran[sg.SG_KERNEL_REDUCE] == (1 if sg.skinny_gemm_fp8_block_workspace(M, N, K, True) else 0)
    assert sum(ran) == ran[sg.SG_KERNEL_FP8_BLOCK] + ran[sg.SG_KERNEL_REDUCE]
    wide = ref.wide_rel(K) * A
    within(y32, y, wide, "fp32")
    within(y16, y, wide + 2.0 ** -8 * (y.abs() + wide), "bf16 with fp32")
    assert torch.equal(y16.cpu(), y32.cpu().to(BF16)), "both outputs are roundings of one sum"
    assert (guard[M:] == -7.0).all(), "rows behind the last one are left as they were"
    only = torch.empty_like(y16)
    sg.skinny_gemm_fp8_block(*d[:4], y_bf16=only)
    loose = (ref.wide_rel(K) if M <= 32 else ref.fp8_rel(K)) * A
    within(only, y, loose + 2.0 ** -8 * (y.abs() + loose), "bf16 alone")
    out = d[4].clone()
    sg.skinny_gemm_fp8_block(*d[:4], r=out, y_bf16=out)  # in place
    yr = y + r.to(F64)
    loose = loose + 2 * ref.U * (yr.abs() + loose)
    within(out, yr, loose + 2.0 ** -8 * (yr.abs() + loose), "residual, in place")
    z32, z16 = sg.skinny_gemm_fp8_block(*d[:4], r=d[4])
    assert z16 is None
    within(z32, yr, wide + 2 * ref.U * (yr.abs() + wide), "residual fp32")
    again, _ = sg.skinny_gemm_fp8_block(*d[:4], r=d[4])
    assert torch.equal(z32, again), "repeated calls give identical bits"


@pytest.mark.parametrize("M", [1, 16, 40, 130, 600])
def test_gemm_values_that_are_not_finite(M):
    """A NaN code or scale makes its outputs NaN and no others; scales follow fp32's rules."""
    N, K = 300, 400
    xq, wq = ref.rand_codes(M, K, 1), ref.rand_codes(N, K, 2)
    xs, ws = ref.rand_scales((4, M), 3), ref.rand_scales((3, 4), 4)
    wq[5, 399], wq[290, 0] = 0x7f, 0xff
    if M > 1:
        xq[M - 1, 130] = 0x7f
        xs[3, 0] = float("nan")
    ws[1, 2] = float("nan")
    y, A = ref.product(xq, xs, wq, ws)
    assert torch.isnan(y[0, 5]) and not torch.isnan(y[min(M - 1, 1)]).all() or M == 1
    d = [t.to(DEV) for t in (xq, xs, wq, ws)]
    y32, _ = sg.skinny_gemm_fp8_block(*d)
    within(y32, y, ref.wide_rel(K) * A, "fp32")
    y16 = torch.empty((M, N), device=DEV, dtype=BF16)
    sg.skinny_gemm_fp8_block(*d, y_bf16=y16)
    loose = ref.fp8_rel(K) * A
    within(y16, y, loose + 2.0 ** -8 * (y.abs() + loose), "bf16")


@pytest.mark.parametrize("M,N,K", [(1, 5, 16), (3, 8193, 144), (20, 131, 272), (60, 257, 1040),
                                   (200, 6, 144), (333, 1001, 272), (700, 2051, 272)])
def test_gemm_rows_of_any_alignment(M, N, K):
    announce(f"fp8_block odd rows M={M} N={N} K={K}")
    xq, wq = ref.rand_codes(M, K, 6), ref.rand_codes(N, K, 7)
    xs, ws = ref.rand_scales((ref.ceil(K), M), 8), ref.rand_scales((ref.ceil(N), ref.ceil(K)), 9)
    flat32, flat16 = torch.full((M * N + 16,), -7.0, device=DEV), torch.full((M * N + 16,), -7.0,
                                                                             device=DEV, dtype=BF16)
    d = [t.to(DEV) for t in (xq, xs, wq, ws)]
    sg.skinny_gemm_fp8_block(*d, y_f32=flat32[:M * N].view(M, N), y_bf16=flat16[:M * N].view(M, N))
    y, A = ref.product(xq, xs, wq, ws)
    within(flat32[:M * N].view(M, N), y, ref.wide_rel(K) * A, "fp32")
    for flat in (flat32, flat16):
        assert (flat[M * N:] == -7.0).all(), "behind the last element"


def test_gemm_empty_sizes():
    f = dict(device=DEV)
    u8 = dict(dtype=torch.uint8, **f)
    for M, N, K in [(0, 5, 32), (5, 0, 32), (0, 0, 0)]:
        y, _ = sg.skinny_gemm_fp8_block(torch.empty((M, K), **u8), torch.empty((ref.ceil(K), M), **f),
                                        torch.empty((N, K), **u8),
                                        torch.empty((ref.ceil(N), ref.ceil(K)), **f))
        assert y.shape == (M, N)
    for M in (1, 20, 200):  # K = 0: the empty sum
        r = normal((M, 9), 1).to(DEV)
        for out in (dict(), dict(y_bf16=torch.empty((M, 9), dtype=BF16, **f))):
            y = sg.skinny_gemm_fp8_block(torch.empty((M, 0), **u8), torch.empty((0, M), **f),
                                         torch.empty((9, 0), **u8), torch.empty((1, 0), **f), r=r, **out)
            assert torch.equal((y[0] if y[1] is None else y[1]).float(), r.float()), "K = 0"


def test_gemm_random_sizes():
    rng = ref.gen(77)
    for i in range(40):
        e = torch.rand(3, generator=rng).tolist()
        M, N, K = int(2 ** (e[0] * 9.5)), int(2 ** (e[1] * 10)), 16 * int(2 ** (e[2] * 7))
        announce(f"fp8_block random {i} M={M} N={N} K={K}")
        xq, wq = ref.rand_codes(M, K, 100 + i), ref.rand_codes(N, K, 200 + i)
        xs, ws = ref.rand_scales((ref.ceil(K), M), 3), ref.rand_scales((ref.ceil(N), ref.ceil(K)), 4)
        d = [t.to(DEV) for t in (xq, xs, wq, ws)]
        y, A = ref.product(xq, xs, wq, ws)
        within(sg.skinny_gemm_fp8_block(*d)[0], y, ref.wide_rel(K) * A, f"M={M} N={N} K={K}")
        y16 = torch.empty((M, N), device=DEV, dtype=BF16)
        sg.skinny_gemm_fp8_block(*d, y_bf16=y16)
        loose = ref.fp8_rel(K) * A
        within(y16, y, loose + 2.0 ** -8 * (y.abs() + loose), f"bf16 M={M} N={N} K={K}")


# ------------------------------------------------------------------ routed experts

GROUPED = [(1, 1, 1, 16, 16), (1, 8, 40, 64, 144), (4, 8, 16, 300, 272), (3, 2, 300, 17, 400),
           (50, 4, 7, 129, 1040), (64, 8, 130, 48, 528), (300, 1, 3, 256, 272), (257, 6, 40, 200, 144),
           (1000, 2, 5, 513, 160), (700, 8, 600, 40, 144), (2000, 3, 4, 70, 272), (40, 32, 32, 64, 128),
           (515, 8, 48, 260, 400), (130, 8, 9, 384, 2064)]


@pytest.mark.parametrize("T,topk,E,N,K", GROUPED)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(T, topk, E, N, K, gather):
    announce(f"grouped fp8 T={T} topk={topk} E={E} N={N} K={K} gather={gather}")
    total = E + E // 3  # some pairs are another rank's
    ids, _ = ref.routing(T, topk, E, max(total, 1), 11)
    offsets, order, positions = ref.table(ids, E)
    P = T * topk
    X = T if gather else P
    xq, wq = ref.rand_codes(X, K, 1), ref.rand_codes(E * N, K, 2).view(E, N, K)
    xs = ref.rand_scales((ref.ceil(K), X), 3)
    ws = ref.rand_scales((E, ref.ceil(N), ref.ceil(K)), 4)
    valid = int(offsets[E])
    y, A = torch.full((P, N), -7.0, dtype=F64), torch.zeros((P, N), dtype=F64)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            rows = order[lo:hi].long() // topk if gather else torch.arange(lo, hi)
            y[lo:hi], A[lo:hi] = ref.product(xq[rows], xs[:, rows], wq[e], ws[e])
    d = [t.to(DEV) for t in (xq, xs, wq, ws, offsets)]
    kw = dict(sorted_pairs=order.to(DEV), topk=topk) if gather else {}
    guard = torch.full((P + 3, N), -7.0, device=DEV)
    sg.grouped_skinny_gemm_fp8(*d, y_f32=guard[:P], **kw)
    within(guard[:P], y, ref.wide_rel(K) * A, "fp32")
    assert (guard[valid:] == -7.0).all(), "rows behind the last segment"
    y16 = torch.full((P + 3, N), -7.0, device=DEV, dtype=BF16)
    sg.grouped_skinny_gemm_fp8(*d, y_bf16=y16[:P], **kw)
    loose = ref.fp8_rel(K) * A
    within(y16[:P], y, loose + 2.0 ** -8 * (y.abs() + loose), "bf16")
    assert (y16[valid:] == -7.0).all(), "rows behind the last segment"
    new, none = sg.grouped_skinny_gemm_fp8(*d, **kw)
    assert none is None and torch.equal(new[:valid], guard[:valid]) and (new[valid:] == 0).all()


@pytest.mark.parametrize("sizes", [[0, 0, 0, 700], [700, 0, 0, 0], [1, 0, 698, 1], [64, 64, 64, 508],
                                   [255, 257, 0, 188], [0, 0, 0, 0]])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_grouped_segments(sizes, dtype):
    """Segments that are empty, one row, and just past whole tiles; rows behind the last."""
    E, P, N, K = 4, 700, 260, 400
    offsets = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32)
    xq, wq = ref.rand_codes(P, K, 1), ref.rand_codes(E * N, K, 2).view(E, N, K)
    xs, ws = ref.rand_scales((ref.ceil(K), P), 3), ref.rand_scales((E, ref.ceil(N), ref.ceil(K)), 4)
    out = torch.full((P, N), -7.0, device=DEV, dtype=dtype)
    kind = "y_f32" if dtype is F32 else "y_bf16"
    sg.grouped_skinny_gemm_fp8(*[t.to(DEV) for t in (xq, xs, wq, ws, offsets)], **{kind: out})
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi == lo:
            continue
        y, A = ref.product(xq[lo:hi], xs[:, lo:hi], wq[e], ws[e])
        loose = ref.wide_rel(K) * A if dtype is F32 else ref.fp8_rel(K) * A
        if dtype is BF16:
            loose = loose + 2.0 ** -8 * (y.abs() + loose)
        within(out[lo:hi], y, loose, f"expert {e}")
    assert (out[int(offsets[E]):] == -7.0).all()


@pytest.mark.parametrize("P,E", [(24, 6), (700, 3)])
def test_grouped_table_out_of_range(P, E):
    """Offsets past the rows and pairs past the tokens stay inside the buffers: rows outside read
    as zeros, offsets are clamped."""
    N, K, T = 48, 272, 8
    xq, wq = ref.rand_codes(T, K, 1), ref.rand_codes(E * N, K, 2).view(E, N, K)
    xs, ws = ref.rand_scales((3, T), 3), ref.rand_scales((E, 1, 3), 4)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = 1 << 30
    offsets[0] = -5
    pairs = torch.arange(P, dtype=torch.int32) % T
    pairs[1], pairs[2], pairs[3] = -1, T, 2 ** 31 - 1
    guard = torch.full((P + 2, N), -7.0, device=DEV)
    sg.grouped_skinny_gemm_fp8(*[t.to(DEV) for t in (xq, xs, wq, ws, offsets)],
                               sorted_pairs=pairs.to(DEV), topk=1, y_f32=guard[:P])
    ok = (pairs >= 0) & (pairs < T)
    rows = pairs.clamp(0, T - 1).long()
    y, A = ref.product(xq[rows], xs[:, rows], wq[0], ws[0])
    y[~ok], A[~ok] = 0, 0
    within(guard[:P], y, ref.wide_rel(K) * A, "clamped")
    assert (guard[P:] == -7.0).all()


# ------------------------------------------------------------------ the experts' step


def step_reference(x, ids, w, wgu, sgu, wd, sd, r, E):
    """(out, bound): every stage in 64 bits from the values the stage before may have; the second
    quantisation sees sums that are off by a little, so a code may be the neighbouring one."""
    T, H = x.shape
    F = wd.shape[2]
    q, s = ref.quant(x.to(F64))
    xf = q * s.t().repeat_interleave(ref.B, 1)[:, :H]
    out = torch.zeros((T, H), dtype=F64) if r is None else r.to(F64).clone()
    bound = torch.zeros_like(out)
    mag = out.abs()
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            W, D = ref.weight64(wgu[e], sgu[e]), ref.weight64(wd[e], sd[e])
            u = W @ xf[t]
            du = ref.fp8_rel(H) * (W.abs() @ xf[t].abs())
            g, up = u[:F], u[F:]
            v = g * torch.sigmoid(g) * up
            # |silu'| <= 1.1
            dv = 1.1 * du[:F] * (up.abs() + du[F:]) + (g * torch.sigmoid(g)).abs() * du[F:]
            dv = dv + ref.GATED_REL * (v.abs() + dv)
            p, ps = ref.quant(v[None])
            unit = ps.t().repeat_interleave(ref.B, 1)[0, :F]
            pf = p[0] * unit
            # off by dv before and by half a step (2^-4, or half of 2^-9 units) on either side
            dp = torch.where(dv > 0, dv + 2 * (2.0 ** -4 * (v.abs() + dv) + unit * 2.0 ** -9), 0.0)
            # ... but only where dv reaches a border between codes (of a unit up to twice as large)
            near = (ref.nearest(((v - dv) / unit).clamp(-448, 448)) !=
                    ref.nearest(((v + dv) / unit).clamp(-448, 448)))
            lo = ref.unit_of((ref.blocks(v[None]).abs().amax(2)
                              - ref.blocks(dv[None]).amax(2)).clamp_min(0))
            hi = ref.unit_of(ref.blocks(v[None]).abs().amax(2) + ref.blocks(dv[None]).amax(2))
            moved = (lo != hi)[0].repeat_interleave(ref.B)[:F]
            dp = torch.where(near | moved, dp, torch.zeros_like(dp))
            y = D @ pf
            dy = D.abs() @ dp + ref.fp8_rel(F) * (D.abs() @ (pf.abs() + dp))
            dy = dy + 2.0 ** -8 * (y.abs() + dy)
            f = float(w[t, j])
            out[t] += f * y
            bound[t] += abs(f) * dy
            mag[t] += abs(f) * (y.abs() + dy)
    bound = bound + (ids.shape[1] + 2) * ref.U * mag
    return out, bound + 2.0 ** -8 * (out.abs() + bound)


STEP = [(1, 1, 1, 16, 16, 1), (1, 8, 16, 144, 128, 16), (4, 8, 40, 272, 144, 53), (9, 2, 3, 128, 272, 4),
        (33, 4, 8, 528, 256, 8), (130, 2, 3, 256, 128, 3), (70, 6, 12, 400, 144, 12),
        (300, 1, 2, 144, 272, 3), (260, 3, 2, 256, 256, 4), (515, 2, 3, 128, 384, 3),
        (100, 4, 10, 272, 256, 12)]


def step_inputs(T, topk, E, H, F, total, seed=1):
    ids, w = ref.routing(T, topk, E, total, seed)
    wgu, wd = ref.rand_codes(E * 2 * F, H, 2).view(E, 2 * F, H), ref.rand_codes(E * H, F, 3).view(E, H, F)
    sgu = ref.rand_scales((E, ref.ceil(2 * F), ref.ceil(H)), 4) * 0.2
    sd = ref.rand_scales((E, ref.ceil(H), ref.ceil(F)), 5) * 0.2
    return normal((T, H), 6), ids, w, wgu, sgu, wd, sd, normal((T, H), 7, 3.0)


@pytest.mark.parametrize("T,topk,E,H,F,total", STEP)
def test_step(T, topk, E, H, F, total):
    announce(f"moe_fp8_step T={T} topk={topk} E={E} H={H} F={F}")
    x, ids, w, wgu, sgu, wd, sd, r = step_inputs(T, topk, E, H, F, total)
    d = [t.to(DEV) for t in (x, ids, w, wgu, sgu, wd, sd)]
    for res in (None, r):
        want, bound = step_reference(x, ids, w, wgu, sgu, wd, sd, res, E)
        out = sg.skinny_moe_fp8_step(*d, r=None if res is None else res.to(DEV))
        within(out, want, bound, f"residual {res is not None}")
    inplace = r.to(DEV)
    sg.skinny_moe_fp8_step(*d, r=inplace, out=inplace)
    assert torch.equal(inplace, out), "out may be r"
    again = sg.skinny_moe_fp8_step(*d, r=r.to(DEV))
    assert torch.equal(again, out), "repeated calls give identical bits"
    xin = d[0].clone()
    sg.skinny_moe_fp8_step(xin, *d[1:], r=r.to(DEV), out=xin)
    assert torch.equal(xin, out), "out may be x"


def test_step_is_its_parts():
    """The step against the public calls that it is made of, as a user would chain them after the
    router (a few rows and a prompt): the same numbers up to the roundings of the product."""
    for T in (5, 300):
        topk, E, H, F = 4, 8, 272, 256
        x, ids, w, wgu, sgu, wd, sd, r = [t.to(DEV) for t in step_inputs(T, topk, E, H, F, E)]
        scores = torch.randn((T, E), device=DEV)
        ids = sg.skinny_gemm_router_topk(scores, topk)
        w = torch.softmax(scores.gather(1, ids.long()), dim=1).contiguous()
        q, s = sg.skinny_quant_fp8(x)
        offsets, order, positions = sg.skinny_moe_sort(ids, E)
        u, _ = sg.grouped_skinny_gemm_fp8(q, s, wgu, sgu, offsets, sorted_pairs=order, topk=topk)
        p, ps = sg.skinny_quant_fp8(u, gated=True)
        y = torch.zeros((T * topk, H), device=DEV, dtype=BF16)
        sg.grouped_skinny_gemm_fp8(p, ps, wd, sd, offsets, y_bf16=y)
        out = sg.skinny_moe_combine(y, positions, w, r=r)
        step = sg.skinny_moe_fp8_step(x, ids, w, wgu, sgu, wd, sd, r=r)
        want, bound = step_reference(*[t.cpu() for t in (x, ids, w, wgu, sgu, wd, sd, r)], E)
        within(out, want, bound, "parts")
        within(step, want, bound, "step")
        # the gathered rows give what the gather operator and the plain segments give
        rows = sg.skinny_moe_gather(x, positions)
        q2, s2 = sg.skinny_quant_fp8(rows)
        u2, _ = sg.grouped_skinny_gemm_fp8(q2, s2, wgu, sgu, offsets)
        assert torch.equal(u, u2), "gathered in the product or before it"


@pytest.mark.parametrize("M,N,K", [(33, 129, 144), (131, 1001, 272), (300, 2051, 272), (513, 8229, 144),
                                   (1030, 8192, 528)])
def test_bf16_rows_of_any_alignment(M, N, K):
    """bf16 outputs alone, which leave large products 64 bytes of a row at a time: with a residual,
    at odd widths, in place, and nothing behind the last element."""
    announce(f"fp8_block bf16 rows M={M} N={N} K={K}")
    xq, wq = ref.rand_codes(M, K, 6), ref.rand_codes(N, K, 7)
    xs, ws = ref.rand_scales((ref.ceil(K), M), 8), ref.rand_scales((ref.ceil(N), ref.ceil(K)), 9)
    r = normal((M, N), 10)
    d = [t.to(DEV) for t in (xq, xs, wq, ws)]
    y, A = ref.product(xq, xs, wq, ws)
    loose = ref.fp8_rel(K) * A
    flat = torch.full((M * N + 64,), -7.0, device=DEV, dtype=BF16)
    out = flat[:M * N].view(M, N)
    sg.skinny_gemm_fp8_block(*d, y_bf16=out)
    within(out, y, loose + 2.0 ** -8 * (y.abs() + loose), "plain")
    out.copy_(r)
    sg.skinny_gemm_fp8_block(*d, r=out, y_bf16=out)
    yr = y + r.to(F64)
    loose = loose + 2 * ref.U * (yr.abs() + loose)
    within(out, yr, loose + 2.0 ** -8 * (yr.abs() + loose), "residual, in place")
    assert (flat[M * N:] == -7.0).all(), "behind the last element"
