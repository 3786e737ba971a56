"""Plain references of the block-scaled FP8 operators and of the sort by expert, on the CPU in 64
bits (test infrastructure).  Tolerances are derived from the roundings the kernels make; u = 2^-24
is half a step of fp32, relative."""
from __future__ import annotations

import torch

U = 2.0 ** -24
F64, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
B = 128


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def ceil(a, b=B):
    return -(-a // b)


def value(codes):
    """e4m3 by its definition: sign, 4 bits of exponent (bias 7), 3 of mantissa; 0x7f is NaN."""
    b = codes.to(torch.int64)
    ex, man = (b >> 3) & 15, (b & 7).to(F64)
    mag = torch.where(ex == 0, man * 2.0 ** -9, torch.ldexp(8 + man, ex.to(F64) - 10))
    mag = torch.where((b & 127) == 127, torch.full_like(mag, float("nan")), mag)
    return torch.where(b >= 128, -mag, mag)


def nearest(v):
    """The e4m3 value next to v (|v| <= 448), half to even."""
    ex = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    ex = torch.where(torch.ldexp(torch.ones_like(v), ex) > v.abs().clamp_min(2.0 ** -6), ex - 1, ex)
    step = torch.ldexp(torch.ones_like(v), ex - 3)
    return torch.round(v / step) * step


def blocks(v):
    """[M, K] as [M, blocks, 128], padded with zeros."""
    pad = -v.shape[1] % B
    return torch.nn.functional.pad(v, (0, pad)).view(v.shape[0], -1, B)


def unit_of(amax):
    """The least power of two >= amax / 448, from 2^-126 on (fp64)."""
    man, ex = torch.frexp(amax)  # 448 = 0.875 * 2^9
    s = (ex - 9 + (man > 0.875).to(ex.dtype)).clamp_min(-126)
    s = torch.where(amax > 0, s, torch.full_like(s, -126))
    return torch.ldexp(torch.ones_like(amax), s.to(F64))


def quant(v):
    """(code values [M, K], scales [blocks, M]) of fp64 rows; a bad block has zeros and NaN."""
    t = blocks(v.to(F64))
    ok = torch.isfinite(t).all(dim=2)
    t = torch.where(ok[:, :, None], t, torch.zeros_like(t))
    unit = unit_of(t.abs().amax(dim=2))
    q = nearest(t / unit[:, :, None]).flatten(1)[:, :v.shape[1]]
    unit = torch.where(ok, unit, torch.full_like(unit, float("nan")))
    return q, unit.t().contiguous()


def gated(x):
    K = x.shape[1] // 2
    g, u = x[:, :K].to(F64), x[:, K:].to(F64)
    return g * torch.sigmoid(g) * u


GATED_REL = 7 * U  # of silu(gate) * up in fp32, as the header promises


def rand_codes(rows, cols, seed, spread=40.0):
    """e4m3 codes of a normal matrix (bytes), all finite."""
    v = (torch.randn((rows, cols), generator=gen(seed)) * spread).clamp(-448, 448)
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def any_codes(rows, cols, seed):
    """Every finite code, equally often: products over the whole range of exponents."""
    c = torch.randint(0, 254, (rows, cols), generator=gen(seed), dtype=torch.int32)
    return (c + (c >= 127)).to(torch.uint8)  # without 0x7f and 0xff


def rand_scales(shape, seed):
    return torch.rand(shape, generator=gen(seed)) * 1e-2 + 1e-3


def rows64(xq, xs):
    """x [M, K] in 64 bits."""
    return value(xq) * xs.to(F64).t().repeat_interleave(B, 1)[:, :xq.shape[1]]


def weight64(wq, ws):
    N, K = wq.shape
    return value(wq) * ws.to(F64).repeat_interleave(B, 0)[:N].repeat_interleave(B, 1)[:, :K]


def product(xq, xs, wq, ws):
    """(y, A): the exact product and the sum of its terms' magnitudes, [M, N]."""
    x, w = rows64(xq, xs), weight64(wq, ws)
    return x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()


def wide_rel(K):
    """Error over A of the sums at fp32's precision: 128 products of a block added one after the
    other, the scale's product, the fused addition to the blocks before, sums of 16 parts; an
    addition may cut (2 u)."""
    return (B + 2 + ceil(K) + 16) * 2 * U


def fp8_rel(K):
    """Error over A of the sums by the FP8 instruction: 7 of 8 neighbouring products cut at 2^-13
    of the largest, below 2^-10; then as above."""
    return 2.0 ** -10 + wide_rel(K)


def table(ids, E):
    """(offsets, sorted, positions) by the definition, int32."""
    flat = ids.reshape(-1).tolist()
    buckets, order = [[] for _ in range(E)], []
    for p, e in enumerate(flat):
        if 0 <= e < E:
            buckets[e].append(p)
    offsets = [0]
    for b in buckets:
        order += b
        offsets.append(offsets[-1] + len(b))
    positions = [-1] * len(flat)
    for i, p in enumerate(order):
        positions[p] = i
    order += [-1] * (len(flat) - len(order))
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(order, dtype=i32),
            torch.tensor(positions, dtype=i32).view(ids.shape))


def routing(T, topk, E, total, seed):
    """ids [T, topk], distinct in a token where total allows it, and weights."""
    g = gen(seed)
    if topk <= total:
        ids = torch.rand((T, total), generator=g).topk(topk, dim=1).indices
    else:
        ids = torch.randint(0, total, (T, topk), generator=g)
    return ids.to(torch.int32).view(T, topk), torch.softmax(torch.randn((T, topk), generator=g), 1)


def combine(rows, positions, w, r):
    """(out, sum of magnitudes) in 64 bits."""
    pos = positions.long()
    on = pos >= 0
    v = rows.to(F64)[pos.clamp_min(0)]
    f = torch.ones(pos.shape, dtype=F64) if w is None else w.to(F64)
    f = torch.where(on, f, torch.zeros_like(f))
    v = torch.where(on[:, :, None], v, torch.zeros_like(v))
    out, mag = (v * f[:, :, None]).sum(1), (v * f[:, :, None]).abs().sum(1)
    return (out, mag) if r is None else (out + r.to(F64), mag + r.to(F64).abs())


def step_of(dtype):
    """Half a step, relative."""
    return torch.finfo(dtype).eps / 2
