"""Plain references of the 8-bit integer operators, on the CPU (test infrastructure).

Where the operators' definition fixes every rounding (codes of a row, the scaled product of
codes) the reference repeats those roundings and outputs are compared bit for bit; the rest is
in 64 bits with tolerances derived from the roundings the kernels make (u = 2^-24 is half a
step of fp32, relative)."""
from __future__ import annotations

import torch

U = 2.0 ** -24
F64, F32 = torch.float64, torch.float32


def codes_of(t):
    """Codes (int8), amax of rows of fp32 t: c = fl(127 / amax), code = rne(t * c) with the
    product exact (48 bits in fp64)."""
    t = t.float()
    ok = torch.isfinite(t).all(dim=1)
    amax = t.abs().nan_to_num(0, 0, 0).amax(dim=1)
    # rows under 2^-100 are scaled by 2^64 first, so that 127 / amax does not overflow
    up = torch.where(amax < 2.0 ** -100, 2.0 ** 64, 1.0).to(F32)
    # (tensor / tensor: torch computes scalar / tensor as scalar * reciprocal, two roundings)
    c = torch.where((amax > 0) & ok, torch.full_like(amax, 127.0) / (amax * up), torch.zeros_like(amax))
    q = torch.round((t * up[:, None]).to(F64).nan_to_num(0, 0, 0) * c.to(F64)[:, None])
    return q.to(torch.int8), amax, ok


def norm_parts(x, r, g):
    """fp32 s and t as the definition rounds them."""
    s = x.float() if r is None else x.float() + r.float()
    return s, s * g.float()


def norm64(x, r, g, eps):
    """(1 / rms, y) in 64 bits, from the fp32 s (its one rounding is part of h's definition)."""
    s = norm_parts(x, r, g)[0].to(F64)
    inv = 1.0 / torch.sqrt((s * s).mean(dim=1) + eps)
    return inv, s * inv[:, None] * g.to(F64)


def norm_rel(K):
    """Relative error of the kernel's 1 / rms: at most 64 squares are summed one after the
    other (2 roundings each), then a tree over lanes and waves and the last 16 sums (30), the
    mean, eps, square root and division (5), halved by the root except for the last two."""
    return (0.5 * (2 * 64 + 30 + 3) + 2) * U


def gated64(x):
    K = x.shape[1] // 2
    gate, up = x[:, :K].to(F64), x[:, K:].to(F64)
    return gate * torch.sigmoid(gate) * up


def gated_rel(x):
    """Relative error of silu(gate) * up in fp32: exp takes fl(-gate * log2 e) (|gate| u in its
    value, one product of |gate| * 1.4427 rounds by |gate| u more) and is off by 2 u itself;
    the sum, quotient (or reciprocal, 2 u, and product) and last product round 5 times."""
    K = x.shape[1] // 2
    return (2.5 * x[:, :K].to(F64).abs() + 2 + 2 + 5) * U


def product(xq, wq):
    """Exact sums of products of codes, int64 (as fp64 products: exact below 2^53)."""
    return (xq.to(F64) @ wq.to(F64).t().contiguous()).to(torch.int64)


def linear(xq, xs, wq, ws, r=None):
    """fp32 bits of the scaled product (and residual): one rounding for each operation."""
    y = product(xq, wq).to(F32) * ws[None, :].to(F32) * xs[:, None].to(F32)
    return y if r is None else r.float() + y
