"""GPU tests of the 8-bit integer operators through the public binding: skinny_gemm_int8,
skinny_rmsnorm, skinny_quant_int8 and skinny_mlp_int8_step, against the plain references of
int8_ref.py.  Codes and scaled products are compared bit for bit."""
import pytest
import torch

import int8_ref as ref
import skinny_gemm_projection_amd as sg
from gpu_common import DEV, announce, counters_delta

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

BF16 = torch.bfloat16
EPS = 1e-6


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rand_codes(rows, cols, seed, lo=-128, hi=127):
    return torch.randint(lo, hi + 1, (rows, cols), generator=gen(seed), dtype=torch.int32).to(torch.int8)


def rand_scales(n, seed):
    return torch.rand(n, generator=gen(seed)) * 1e-3 + 1e-4


def normal(shape, seed, sigma=1.0):
    return (torch.randn(shape, generator=gen(seed)) * sigma).to(BF16)


def same(got, want, what):
    """Equal values, NaN in the same places."""
    got, want = got.cpu(), want.cpu()
    assert got.shape == want.shape and got.dtype == want.dtype, what
    bad = ~((got == want) | (torch.isnan(got.float()) & torch.isnan(want.float())))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ"


# ------------------------------------------------------------------ product

GEMM = [(1, 1, 16), (1, 40, 16), (1, 129, 112), (1, 1024, 1024), (1, 200, 8208), (2, 300, 4128),
        (3, 70, 2064), (4, 257, 8192), (5, 17, 48), (7, 1000, 80), (8, 16, 64), (11, 300, 7168),
        (15, 31, 144), (16, 129, 2064), (16, 2048, 1040), (16, 33, 20000), (17, 200, 1040),
        (20, 129, 7168), (31, 130, 272), (32, 300, 4112), (33, 64, 16), (47, 257, 2064),
        (48, 1000, 8192), (61, 333, 7168), (64, 33, 30000), (64, 1, 144), (64, 4099, 1040),
        (65, 130, 192), (96, 500, 1008), (100, 1000, 4096), (128, 128, 128), (129, 255, 160),
        (200, 37, 9008), (255, 257, 640), (256, 256, 2048), (257, 513, 144), (300, 1001, 2064),
        (511, 1030, 528), (513, 5, 272), (700, 777, 1040), (1025, 1281, 256), (2049, 300, 528),
        (1000, 2051, 2064),
        # wide W: two row tiles a workgroup, x in registers, every tile size (the last two
        # sizes' rows unaligned and aligned), K split with each
        (9, 8195, 1040), (1, 8196, 4112), (17, 8195, 1040), (33, 7170, 1040), (33, 8200, 1296),
        (9, 8195, 16), (1, 6147, 1040), (8, 20003, 528), (5, 6148, 2064), (400, 16390, 144),
        (513, 16392, 272), (129, 16390, 272), (140, 16384, 528), (65, 16390, 400), (70, 16400, 144),
        (65, 8195, 400), (77, 8192, 272), (129, 6147, 8208), (129, 16390, 6160), (129, 16388, 6160),
        (4097, 17, 3088), (3000, 64, 4112),
        # row pitches of a multiple of 4 KB: every workgroup starts elsewhere in K
        (1, 300, 4096), (16, 1000, 8192), (3, 8200, 4096), (20, 8195, 4096), (5, 20001, 4096),
        (40, 500, 12288), (50, 100, 4096), (2, 17, 16384),
        # two launches: whole rounds of the largest tiles, smaller ones for the other columns
        (1281, 12290, 528), (1281, 12292, 528)]


@pytest.mark.parametrize("M,N,K", GEMM)
def test_gemm_bits(M, N, K):
    announce(f"int8 M={M} N={N} K={K}")
    xq, wq = rand_codes(M, K, 1 + M), rand_codes(N, K, 2 + N)
    xs, ws = rand_scales(M, 3), rand_scales(N, 4)
    r = normal((M, N), 5)
    d = [t.to(DEV) for t in (xq, xs, wq, ws, r)]
    guard = torch.full((M + 3, N), -7.0, device=DEV)
    y32, y16 = guard[:M], torch.full((M, N), -7.0, device=DEV, dtype=BF16)
    before = sg.skinny_gemm_get_counters()
    sg.skinny_gemm_int8(*d[:4], y_f32=y32, y_bf16=y16)
    torch.cuda.synchronize()
    ran = counters_delta(before, sg.skinny_gemm_get_counters())
    assert ran[sg.SG_KERNEL_INT8] in (1, 2)  # two: whole rounds of tiles, then the other columns
    assert ran[sg.SG_KERNEL_REDUCE] == (1 if sg.skinny_gemm_int8_workspace(M, N, K) else 0)
    assert sum(ran) == ran[sg.SG_KERNEL_INT8] + ran[sg.SG_KERNEL_REDUCE]
    want = ref.linear(xq, xs, wq, ws)
    same(y32, want, "fp32")
    same(y16, want.to(BF16), "bf16")
    assert (guard[M:] == -7.0).all(), "rows behind the last one are left as they were"
    only16 = torch.empty_like(y16)
    sg.skinny_gemm_int8(*d[:4], y_bf16=only16)
    same(only16, want.to(BF16), "bf16 alone")
    wr = ref.linear(xq, xs, wq, ws, r)
    out = d[4].clone()
    sg.skinny_gemm_int8(*d[:4], r=out, y_bf16=out)  # in place
    same(out, wr.to(BF16), "residual, in place")
    z32, z16 = sg.skinny_gemm_int8(*d[:4], r=d[4])
    assert z16 is None
    same(z32, wr, "residual fp32")


@pytest.mark.parametrize("M,N", [(1, 20), (16, 33), (40, 130), (130, 70), (300, 260)])
def test_gemm_extreme_codes_longest_k(M, N):
    """Every code -128 over the longest K: the largest sum, 2^14 * 131056 < 2^31; mixed signs."""
    K = 131056
    announce(f"int8 extreme M={M} N={N} K={K}")
    xq = torch.full((M, K), -128, dtype=torch.int8)
    wq = torch.full((N, K), -128, dtype=torch.int8)
    wq[1::2] = 127
    xs, ws = rand_scales(M, 3), rand_scales(N, 4)
    y, _ = sg.skinny_gemm_int8(xq.to(DEV), xs.to(DEV), wq.to(DEV), ws.to(DEV))
    acc = torch.full((M, N), 2 ** 14 * K, dtype=torch.int64)
    acc[:, 1::2] = -128 * 127 * K
    same(y, acc.float() * ws[None] * xs[:, None], "extreme")


@pytest.mark.parametrize("M", [1, 16, 40, 130, 600])
def test_gemm_scales_that_are_not_finite(M):
    N, K = 70, 160
    xq, wq = rand_codes(M, K, 1), rand_codes(N, K, 2)
    xs, ws = rand_scales(M, 3), rand_scales(N, 4)
    xs[0], ws[3], ws[4], ws[5] = float("nan"), float("nan"), float("inf"), 0.0
    r = normal((M, N), 5)
    y, h = sg.skinny_gemm_int8(xq.to(DEV), xs.to(DEV), wq.to(DEV), ws.to(DEV),
                               y_f32=torch.empty((M, N), device=DEV),
                               y_bf16=torch.empty((M, N), device=DEV, dtype=BF16), r=r.to(DEV))
    want = ref.linear(xq, xs, wq, ws, r)
    same(y, want, "fp32")
    same(h, want.to(BF16), "bf16")


@pytest.mark.parametrize("M,N,K", [(1, 5, 16), (3, 8193, 144), (20, 131, 272), (60, 257, 1040),
                                   (61, 1027, 7168), (200, 6, 144), (333, 1001, 272), (700, 2051, 272)])
def test_gemm_rows_of_any_alignment(M, N, K):
    """Rows of y that start at odd elements are written one access for four elements: every
    element in its place, and nothing behind the last one."""
    announce(f"int8 odd rows M={M} N={N} K={K}")
    xq, wq = rand_codes(M, K, 6), rand_codes(N, K, 7)
    xs, ws = rand_scales(M, 8), rand_scales(N, 9)
    r = normal((M, N), 10)
    flat32, flat16 = torch.full((M * N + 16,), -7.0, device=DEV), torch.full((M * N + 16,), -7.0,
                                                                             device=DEV, dtype=BF16)
    sg.skinny_gemm_int8(xq.to(DEV), xs.to(DEV), wq.to(DEV), ws.to(DEV), r=r.to(DEV),
                        y_f32=flat32[:M * N].view(M, N), y_bf16=flat16[:M * N].view(M, N))
    want = ref.linear(xq, xs, wq, ws, r)
    for flat, t in ((flat32, torch.float32), (flat16, BF16)):
        same(flat[:M * N].view(M, N), want.to(t), str(t))
        assert (flat[M * N:] == -7.0).all(), f"{t}: behind the last element"


def test_gemm_empty_sizes():
    f = dict(device=DEV)
    for M, N, K in [(0, 5, 32), (5, 0, 32), (0, 0, 0)]:
        y, _ = sg.skinny_gemm_int8(torch.empty((M, K), dtype=torch.int8, **f), torch.empty(M, **f),
                                   torch.empty((N, K), dtype=torch.int8, **f), torch.empty(N, **f))
        assert y.shape == (M, N)
    for M in (1, 20, 200):  # K = 0: the empty sum
        r = normal((M, 9), 1).to(DEV)
        y, _ = sg.skinny_gemm_int8(torch.empty((M, 0), dtype=torch.int8, **f), torch.ones(M, **f),
                                   torch.empty((9, 0), dtype=torch.int8, **f), torch.ones(9, **f), r=r)
        same(y, r.float(), "K = 0")


def test_gemm_random_sizes():
    rng = gen(77)
    for i in range(40):
        e = torch.rand(3, generator=rng).tolist()
        M, N, K = int(2 ** (e[0] * 9.5)), int(2 ** (e[1] * 10)), 16 * int(2 ** (e[2] * 7))
        announce(f"int8 random {i} M={M} N={N} K={K}")
        xq, wq = rand_codes(M, K, 100 + i), rand_codes(N, K, 200 + i)
        xs, ws = rand_scales(M, 3), rand_scales(N, 4)
        y, _ = sg.skinny_gemm_int8(xq.to(DEV), xs.to(DEV), wq.to(DEV), ws.to(DEV))
        same(y, ref.linear(xq, xs, wq, ws), f"M={M} N={N} K={K}")


# ------------------------------------------------------------------ norm

ROW_K = [8, 72, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 7168, 8192, 8200, 16384, 16392,
         32768, 32776, 65536]


def norm_inputs(M, K, seed):
    x, r = normal((M, K), seed), normal((M, K), seed + 1, 3.0)
    g = (1.0 + 0.2 * torch.randn(K, generator=gen(seed + 2))).to(BF16)
    return x, r, g


def check_norm(x, r, g, eps, h, y, codes, scales, what):
    M, K = x.shape
    s, t = ref.norm_parts(x, r, g)
    want, amax, ok = ref.codes_of(t)
    ok &= torch.isfinite(s.float().square().sum(dim=1))
    want[~ok] = 0
    if h is not None:
        same(h, s.to(BF16), what + ": h")
    inv, y64 = ref.norm64(x, r, g, eps)
    rel = ref.norm_rel(K)
    if y is not None:
        got = y.cpu().double()
        # bf16 half a step, t's and the last product's roundings; under 2^-126 a step is 2^-133
        bound = (2.0 ** -8 + rel + 3 * ref.U) * y64.abs() + 2.0 ** -133
        assert ((got - y64).abs() <= bound)[ok].all(), what + ": y"
        assert torch.isnan(got[~ok]).all(), what + ": y of rows that are not finite"
    if codes is not None:
        same(codes, want, what + ": codes")
        sc = scales.cpu().double()
        s64 = amax.double() * inv / 127.0
        assert ((sc - s64).abs() <= (rel + 3 * ref.U) * s64 + 2.0 ** -149)[ok].all(), what + ": scales"
        assert torch.isnan(sc[~ok]).all(), what + ": scales of rows that are not finite"


@pytest.mark.parametrize("K", ROW_K)
@pytest.mark.parametrize("M", [1, 3, 70])
def test_norm(M, K):
    announce(f"rmsnorm M={M} K={K}")
    x, r, g = norm_inputs(M, K, 10 + K + M)
    dx, dr, dg = x.to(DEV), r.to(DEV), g.to(DEV)
    h, y = torch.empty_like(dx), torch.empty_like(dx)
    guard = torch.full((M + 1, K), 99, dtype=torch.int8, device=DEV)
    gs = torch.full((M + 1,), -7.0, device=DEV)
    before = sg.skinny_gemm_get_counters()
    sg.skinny_rmsnorm(dx, dg, EPS, r=dr, h=h, y_bf16=y, codes=guard[:M], scales=gs[:M])
    torch.cuda.synchronize()
    assert counters_delta(before, sg.skinny_gemm_get_counters())[sg.SG_KERNEL_RMSNORM] == 1
    check_norm(x, r, g, EPS, h, y, guard[:M], gs[:M], f"M={M} K={K}")
    assert (guard[M] == 99).all() and gs[M] == -7.0
    # no residual; codes allocated; bf16 alone
    _, _, c2, s2 = sg.skinny_rmsnorm(dx, dg, EPS)
    check_norm(x, None, g, EPS, None, None, c2, s2, "no residual")
    y2 = torch.empty_like(dx)
    assert sg.skinny_rmsnorm(dx, dg, 0.5, r=dr, y_bf16=y2)[2:] == (None, None)
    check_norm(x, r, g, 0.5, None, y2, None, None, "bf16 alone")
    # h over r, y over x
    hr, yx = dr.clone(), dx.clone()
    sg.skinny_rmsnorm(yx, dg, EPS, r=hr, h=hr, y_bf16=yx)
    same(hr, h, "h in place"), same(yx, y, "y in place")


def test_norm_rows_of_every_kind():
    """Zeros, one value, NaN, infinities, the largest and smallest values, side by side."""
    K = 1032
    x, _, g = norm_inputs(12, K, 5)
    x[0] = 0
    x[1], x[1, 7] = 0, 3.0
    x[2, 5] = float("nan")
    x[3, K - 1] = float("inf")
    x[4, 0] = float("-inf")
    x[5] = 3.0e38
    x[6] = 1e-38
    x[7] = 2.0 ** -133
    x[8] = torch.finfo(BF16).min
    x[9, 3] = 1e18
    for c in (True, False):
        r = normal((12, K), 9, 0.1) if c else None
        if c:
            r[:9] = 0
            r[10, 4] = float("inf")
        dx, dr, dg = x.to(DEV), None if r is None else r.to(DEV), g.to(DEV)
        h, y = torch.empty_like(dx), torch.empty_like(dx)
        _, _, codes, scales = sg.skinny_rmsnorm(dx, dg, EPS, r=dr, h=h, y_bf16=y,
                                                codes=torch.empty((12, K), dtype=torch.int8, device=DEV))
        check_norm(x, r, g, EPS, h, y, codes, scales, f"residual {c}")
        assert (codes[0] == 0).all() and scales[0] == 0.0
        assert codes[1].abs().sum() == 127


# ------------------------------------------------------------------ quantiser


def check_quant(x, gated, codes, scales, what):
    codes, sc = codes.cpu(), scales.cpu()
    if not gated:
        want, amax, ok = ref.codes_of(x.float())
        same(codes, want, what + ": codes")
        same(sc, torch.where(ok, amax / 127.0, torch.full_like(amax, float("nan"))), what + ": scales")
        return
    t, rel = ref.gated64(x), ref.gated_rel(x)
    ok = torch.isfinite(x.float()).all(dim=1) & torch.isfinite(t.float()).all(dim=1)
    err = rel * t.abs() + 2.0 ** -149
    amax, top = t.abs().amax(dim=1), (t.abs() + err).amax(dim=1)
    s64 = amax / 127.0
    slack = top / 127.0 - s64 + 2 * ref.U * s64 + 2.0 ** -149
    assert ((sc.double() - s64).abs() <= slack)[ok].all(), what + ": scales"
    assert torch.isnan(sc[~ok]).all() and (codes[~ok] == 0).all(), what + ": rows not finite"
    # half a step of rounding, the error of t, of 127 / amax and of the scale
    got = codes.double() * sc.double()[:, None]
    bound = 0.5 * sc.double()[:, None] + err + t.abs() * (slack / s64.clamp_min(1e-300) + 4 * ref.U)[:, None]
    assert ((got - t).abs() <= bound)[ok].all(), what + ": values"


@pytest.mark.parametrize("K", ROW_K)
@pytest.mark.parametrize("f32", [False, True])
def test_quant(K, f32):
    for M in (1, 5, 70):
        announce(f"quant_int8 M={M} K={K} f32={f32}")
        for gated in (False, True):
            x = torch.randn((M, 2 * K if gated else K), generator=gen(K + M)) * 2
            x = x if f32 else x.to(BF16)
            guard = torch.full((M + 1, K), 99, dtype=torch.int8, device=DEV)
            gs = torch.full((M + 1,), -7.0, device=DEV)
            before = sg.skinny_gemm_get_counters()
            sg.skinny_quant_int8(x.to(DEV), gated, guard[:M], gs[:M])
            torch.cuda.synchronize()
            assert counters_delta(before, sg.skinny_gemm_get_counters())[sg.SG_KERNEL_QUANT_INT8] == 1
            check_quant(x, gated, guard[:M], gs[:M], f"M={M} K={K} f32={f32} gated={gated}")
            assert (guard[M] == 99).all() and gs[M] == -7.0


@pytest.mark.parametrize("f32", [False, True])
def test_quant_rows_of_every_kind(f32):
    K = 1032
    x = torch.randn((12, K), generator=gen(5))
    x[0] = 0
    x[1], x[1, 7] = 0, 3.0
    x[2, 5] = float("nan")
    x[3, K - 1] = float("inf")
    x[4, 0] = float("-inf")
    x[5] = 3.0e38
    x[6] = 1e-38
    x[7] = 2.0 ** -133
    x[8] *= 1e-37
    x[9, 3] = 1e18
    if f32:
        x[10] = 1.5e-45
        x[11] = torch.tensor([0x7fc12345], dtype=torch.int32).view(torch.float32)  # NaN with a payload
    x = x if f32 else x.to(BF16)
    codes, scales = sg.skinny_quant_int8(x.to(DEV))
    check_quant(x, False, codes, scales, "every kind")
    # gated: very negative, very positive gates, infinities and NaN in either half
    z = torch.randn((8, 2 * K), generator=gen(6))
    z[0, :K], z[1, :K] = -300.0, 300.0
    z[2, 3], z[3, K + 3] = float("nan"), float("inf")
    z[4, 0] = float("-inf")
    z[5] = 0
    z[6, K:] = 0
    z = z if f32 else z.to(BF16)
    codes, scales = sg.skinny_quant_int8(z.to(DEV), gated=True)
    check_quant(z, True, codes, scales, "gated, every kind")
    assert scales[5] == 0 and scales[6] == 0 and scales[0] == 0


# ------------------------------------------------------------------ the operators together


def mlp_inputs(M, H, F, seed, res=True):
    x, r, g = norm_inputs(M, H, seed)
    wgu, sgu = rand_codes(2 * F, H, seed + 3, -127), rand_scales(2 * F, seed + 4)
    wd, sd = rand_codes(H, F, seed + 5, -127), rand_scales(H, seed + 6)
    return x, (r if res else None), g, wgu, sgu * (4 / H ** 0.5), wd, sd * (4 / F ** 0.5)


def parts(x, r, g, wgu, sgu, wd, sd):
    """The step as the public calls it is made of."""
    h = torch.empty_like(x)
    _, _, q, sq = sg.skinny_rmsnorm(x, g, EPS, r=r, h=h,
                                    codes=torch.empty(x.shape, dtype=torch.int8, device=DEV))
    u, _ = sg.skinny_gemm_int8(q, sq, wgu, sgu)
    p, sp = sg.skinny_quant_int8(u, gated=True)
    out = torch.empty_like(x)
    sg.skinny_gemm_int8(p, sp, wd, sd, r=h, y_bf16=out)
    return q, sq, u, p, sp, h, out


MLP = [(1, 512, 1024), (1, 16, 16), (2, 7168, 2064), (4, 1040, 2064), (16, 528, 272), (33, 272, 1040),
       (61, 1024, 4112), (65, 528, 1040), (130, 1040, 784), (300, 512, 1296), (1025, 272, 528),
       # every tile size with the gated product in its epilogue
       (65, 272, 8208), (129, 144, 8208), (257, 144, 12304), (400, 272, 8208),
       (1281, 528, 6160)]


@pytest.mark.parametrize("M,H,F", MLP)
def test_mlp_step_is_its_parts(M, H, F):
    """The step gives the bits of the public calls one after the other, and those of the parts
    are the references'."""
    announce(f"mlp M={M} H={H} F={F}")
    cpu = mlp_inputs(M, H, F, 40 + M, res=M % 2 == 0)
    x, r, g, wgu, sgu, wd, sd = [None if t is None else t.to(DEV) for t in cpu]
    q, sq, u, p, sp, h, want = parts(x, r, g, wgu, sgu, wd, sd)
    got = sg.skinny_mlp_int8_step(x, g, EPS, wgu, sgu, wd, sd, r=r)
    same(got, want, "step")
    # the parts' chain against the references
    check_norm(cpu[0], cpu[1], cpu[2], EPS, h, None, q, sq, "norm")
    same(u, ref.linear(q.cpu(), sq.cpu(), cpu[3], cpu[4]), "gate and up")
    check_quant(u.cpu(), True, p, sp, "gated codes")
    same(want, ref.linear(p.cpu(), sp.cpu(), cpu[5], cpu[6], h.cpu()).to(BF16), "down")
    # in place over x, and over the residual
    xi = x.clone()
    assert sg.skinny_mlp_int8_step(xi, g, EPS, wgu, sgu, wd, sd, r=r, out=xi) is xi
    same(xi, want, "over x")
    if r is not None:
        ri = r.clone()
        sg.skinny_mlp_int8_step(x, g, EPS, wgu, sgu, wd, sd, r=ri, out=ri)
        same(ri, want, "over r")


def test_mlp_row_that_is_not_finite_stays_alone():
    cpu = mlp_inputs(9, 272, 528, 3)
    cpu[0][4, 100] = float("nan")
    x, r, g, wgu, sgu, wd, sd = [t.to(DEV) for t in cpu]
    got = sg.skinny_mlp_int8_step(x, g, EPS, wgu, sgu, wd, sd, r=r)
    clean = x.clone()
    clean[4] = 1.0
    want = sg.skinny_mlp_int8_step(clean, g, EPS, wgu, sgu, wd, sd, r=r)
    assert torch.isnan(got[4].float()).all()
    keep = [i for i in range(9) if i != 4]
    same(got[keep], want[keep], "other rows")


@pytest.mark.parametrize("M,H,F", [(1, 512, 1024), (20, 1040, 2064), (130, 528, 1040)])
def test_mlp_captured_and_replayed(M, H, F):
    """Captured once with its workspace, replayed on changing inputs between eager calls."""
    announce(f"mlp graph M={M}")
    cpu = mlp_inputs(M, H, F, 60)
    x, r, g, wgu, sgu, wd, sd = [t.to(DEV) for t in cpu]
    ws = torch.empty(max(1, sg.skinny_mlp_int8_step_workspace(M, H, F)), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sg.skinny_mlp_int8_step(x, g, EPS, wgu, sgu, wd, sd, r=r, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.skinny_mlp_int8_step(x, g, EPS, wgu, sgu, wd, sd, r=r, out=out, workspace=ws)
    for i in range(4):
        x.copy_(normal((M, H), 70 + i))
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        same(got, sg.skinny_mlp_int8_step(x, g, EPS, wgu, sgu, wd, sd, r=r), f"replay {i}")


def test_calls_on_two_streams_at_once():
    """Two steps on two streams, each with memory of its own, give the bits of one alone."""
    sets = []
    for seed, M in ((80, 24), (90, 150)):
        x, r, g, wgu, sgu, wd, sd = [t.to(DEV) for t in mlp_inputs(M, 1040, 2064, seed)]
        sets.append(((x, g, EPS, wgu, sgu, wd, sd), r))
    want = [sg.skinny_mlp_int8_step(*a, r=r) for a, r in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(6):
        for k, (a, r) in enumerate(sets):
            got[k].append(sg.skinny_mlp_int8_step(*a, r=r, stream=streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for y in got[k]:
            same(y, want[k], f"stream {k}")


def test_weights_quantised_by_the_row_quantiser():
    """Per-channel weight codes come from the same call; the product of the two quantised
    matrices is near the plain product: each value is off by at most half a step."""
    M, N, K = 9, 130, 1040
    x, W = normal((M, K), 1), normal((N, K), 2, 0.02)
    xq, xs = sg.skinny_quant_int8(x.to(DEV))
    wq, ws = sg.skinny_quant_int8(W.to(DEV))
    y, _ = sg.skinny_gemm_int8(xq, xs, wq, ws)
    want = x.double() @ W.double().t()
    hx, hw = 0.5 * xs.cpu().double()[:, None], 0.5 * ws.cpu().double()[None, :]
    ax, aw = x.double().abs().sum(dim=1)[:, None], W.double().abs().sum(dim=1)[None, :]
    assert ((y.cpu().double() - want).abs() <= (hx * aw + hw * ax + K * hx * hw) * 1.001).all()


# ------------------------------------------------------------------ calls the documentation allows


def product_inputs(M, N, K, seed):
    cpu = rand_codes(M, K, seed), rand_scales(M, seed + 1), rand_codes(N, K, seed + 2), rand_scales(N, seed + 3)
    return cpu, [t.to(DEV) for t in cpu]


SPLIT = [(61, 512, 8192), (100, 257, 16384), (40, 4096, 7168)]


@pytest.mark.parametrize("M,N,K", SPLIT)
def test_gemm_split_between_workgroups(M, N, K):
    """A K that is split goes through the caller's workspace, whatever that held before; a
    workspace longer than needed is left alone behind its end."""
    announce(f"int8 split M={M} N={N} K={K}")
    need = sg.skinny_gemm_int8_workspace(M, N, K)
    cpu, d = product_inputs(M, N, K, 5)
    want = ref.linear(*cpu)
    for fill in (0, 255):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
        y, _ = sg.skinny_gemm_int8(*d, workspace=ws)
        same(y, want, f"workspace of {fill}")
        assert (ws[need:] == fill).all()
    if need:
        before = sg.skinny_gemm_get_counters()
        with pytest.raises(sg.SkinnyGemmError) as e:
            sg.skinny_gemm_int8(*d, workspace=torch.empty(need - 16, dtype=torch.uint8, device=DEV))
        assert e.value.status == 5
        assert counters_delta(before, sg.skinny_gemm_get_counters()) == [0] * sg.SG_NUM_COUNTERS


def test_two_captured_graphs_and_eager_calls():
    """Two graphs, each with a workspace of its own, replayed in turn with eager calls between."""
    sets = []
    for seed, (M, N, K) in ((5, SPLIT[0]), (50, SPLIT[1])):
        cpu, d = product_inputs(M, N, K, seed)
        ws = torch.empty(max(16, sg.skinny_gemm_int8_workspace(M, N, K)), dtype=torch.uint8, device=DEV)
        y = torch.empty((M, N), device=DEV)
        sg.skinny_gemm_int8(*d, y_f32=y, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sg.skinny_gemm_int8(*d, y_f32=y, workspace=ws)
        sets.append((g, d, y, cpu))
    for i in range(4):
        for g, d, y, cpu in sets:
            d[1].copy_(rand_scales(d[1].shape[0], 900 + i))
            y.zero_()
            g.replay()
            eager, _ = sg.skinny_gemm_int8(*d)
            same(y, eager, f"replay {i}")
            same(y, ref.linear(cpu[0], d[1].cpu(), cpu[2], cpu[3]), f"replay {i}")


def test_streams_given_and_current():
    """Work goes to the stream given (a Stream or a handle), else to the current one."""
    cpu, d = product_inputs(33, 300, 2064, 8)
    want = ref.linear(*cpu)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, _ = sg.skinny_gemm_int8(*d, stream=s)
    s.synchronize()
    same(y, want, "stream given")
    y, _ = sg.skinny_gemm_int8(*d, stream=s.cuda_stream)
    s.synchronize()
    same(y, want, "handle given")
    with torch.cuda.stream(s):
        y, _ = sg.skinny_gemm_int8(*d)
    s.synchronize()
    same(y, want, "current stream")
    x = normal((5, 1032), 1)
    with torch.cuda.stream(s):
        c, sc = sg.skinny_quant_int8(x.to(DEV))
    s.synchronize()
    check_quant(x, False, c, sc, "current stream")


def test_refusals_before_anything_runs():
    q, qs = torch.zeros((3, 64), dtype=torch.int8, device=DEV), torch.ones(3, device=DEV)
    w, ws = torch.zeros((5, 64), dtype=torch.int8, device=DEV), torch.ones(5, device=DEV)
    x = torch.zeros((3, 64), dtype=BF16, device=DEV)
    g = torch.ones(64, dtype=BF16, device=DEV)
    y, y16 = torch.empty((3, 5), device=DEV), torch.empty((3, 5), device=DEV, dtype=BF16)
    before = sg.skinny_gemm_get_counters()

    def refused(kind, f, *a, **kw):
        with pytest.raises(kind):
            f(*a, **kw)

    f = sg.skinny_gemm_int8
    refused(ValueError, f, q, qs[:2], w, ws)
    refused(ValueError, f, q, qs, w, ws[:4])
    refused(ValueError, f, q, qs, w[:, :48], ws)
    refused(ValueError, f, q[:, :48], qs, w[:, :48].contiguous(), ws)  # not contiguous
    refused(ValueError, f, q, qs, w.cpu(), ws)
    refused(ValueError, f, q, qs, w, ws, y_f32=y.t())
    refused(TypeError, f, q, qs, w, ws, y_f32=y16)
    refused(TypeError, f, q, qs.double(), w, ws)
    refused(TypeError, f, q, qs, w.to(torch.uint8), ws)
    refused(ValueError, f, q, qs, w, ws, r=y16[:2])
    refused(sg.SkinnyGemmError, f, q[:, :24].contiguous(), qs, w[:, :24].contiguous(), ws)
    refused(TypeError, f, q, qs, w, ws, workspace=qs)
    n = sg.skinny_rmsnorm
    refused(ValueError, n, x, g[:32], 1e-6)
    refused(ValueError, n, x, g, 1e-6, r=x[:2])
    refused(TypeError, n, x, g.float(), 1e-6)
    refused(sg.SkinnyGemmError, n, x, g, 0.0)
    refused(ValueError, n, x, g, 1e-6, codes=q[:2])
    refused(sg.SkinnyGemmError, sg.skinny_quant_int8, x[:, :12].contiguous())
    refused(ValueError, sg.skinny_quant_int8, x, gated=True, codes=q)
    wgu, wd = torch.zeros((64, 64), dtype=torch.int8, device=DEV), torch.zeros((64, 32), dtype=torch.int8, device=DEV)
    one = torch.ones(64, device=DEV)
    refused(ValueError, sg.skinny_mlp_int8_step, x, g, 1e-6, wgu[:48], one, wd, one)
    refused(sg.SkinnyGemmError, sg.skinny_mlp_int8_step, x, g, float("nan"), wgu, one, wd, one)
    refused(ValueError, sg.skinny_mlp_int8_step, x, g, 1e-6, wgu, one, wd, one, out=x.t())
    assert counters_delta(before, sg.skinny_gemm_get_counters()) == [0] * sg.SG_NUM_COUNTERS


def test_offsets_past_32_bits():
    """Outputs, activations and weights past 4 GB; sampled rows against the references."""
    f = dict(device=DEV)
    announce("int8 output past 2^31 elements")
    M, N, K = 65700, 32784, 32
    xq, wq = [torch.randint(-128, 128, s, dtype=torch.int8, **f) for s in ((M, K), (N, K))]
    xs, ws = torch.rand(M, **f) + 0.5, torch.rand(N, **f) + 0.5
    y = torch.empty((M, N), dtype=BF16, **f)
    sg.skinny_gemm_int8(xq, xs, wq, ws, y_bf16=y)
    at = torch.tensor([0, 1, 255, 256, 32767, 65533, 65535, 65536, M - 1])
    same(y[at.to(DEV)], ref.linear(xq.cpu()[at], xs.cpu()[at], wq.cpu(), ws.cpu()).to(BF16), "rows")
    del y
    announce("int8 weights and codes past 2^32 bytes")
    for M, N, K in ((3, 69000, 65536), (69000, 40, 65536), (300, 69000, 65536)):
        xq, wq = [torch.randint(-128, 128, s, dtype=torch.int8, **f) for s in ((M, K), (N, K))]
        xs, ws = torch.rand(M, **f), torch.rand(N, **f)
        y, _ = sg.skinny_gemm_int8(xq, xs, wq, ws)
        r, c = torch.tensor([0, M // 2, M - 1]), torch.tensor([0, N // 2, N - 2, N - 1])
        want = ref.linear(xq[r.to(DEV)].cpu(), xs.cpu()[r], wq[c.to(DEV)].cpu(), ws.cpu()[c])
        same(y.cpu()[r][:, c], want, f"M={M} N={N}")
    announce("rows past 2^32 bytes")
    M, K = 70000, 32776
    x = torch.randn((M, K), dtype=BF16, **f)
    g = torch.ones(K, dtype=BF16, **f)
    _, _, codes, scales = sg.skinny_rmsnorm(x, g, EPS)
    r = torch.tensor([0, 65535, 65536, M - 1], device=DEV)
    check_norm(x[r].cpu(), None, g.cpu(), EPS, None, None, codes[r], scales[r], "norm")
    codes, scales = sg.skinny_quant_int8(x, codes=codes, scales=scales)
    check_quant(x[r].cpu(), False, codes[r], scales[r], "codes")


@pytest.mark.parametrize("M,H,F", [(2, 65536, 48), (2, 48, 65536), (260, 65536, 8208), (5, 64, 32)])
def test_mlp_widest_rows(M, H, F):
    announce(f"mlp widest M={M} H={H} F={F}")
    f = dict(device=DEV)
    x, r = normal((M, H), 1).to(DEV), normal((M, H), 2).to(DEV)
    g = torch.ones(H, dtype=BF16, **f)
    wgu = torch.randint(-127, 128, (2 * F, H), dtype=torch.int8, **f)
    wd = torch.randint(-127, 128, (H, F), dtype=torch.int8, **f)
    sgu, sd = torch.rand(2 * F, **f) * 1e-3 / H ** 0.5, torch.rand(H, **f) * 1e-3 / F ** 0.5
    out = sg.skinny_mlp_int8_step(x, g, EPS, wgu, sgu, wd, sd, r=r)
    same(out, parts(x, r, g, wgu, sgu, wd, sd)[-1], "step")
    assert torch.isfinite(out.float()).all()
