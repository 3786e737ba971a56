"""Measured cases of the 8-bit integer operators: the root-mean-square norm with int8
output, the row quantiser (plain and gated), the int8 matrix product, and the gated
MLP block made of them.

Shapes: hidden 7168 and widths 1024..8192 are the decode workloads this repository is
benchmarked on, 18432 its widest measured weight; the others are generic odd sizes.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def listed():
    return [
        # one token through a small projection: what the call itself costs
        dict(name="gemm 1 token small", op="gemm", M=1, N=1024, K=1024, res=False, out="bf16"),
        # two tokens through a wide input projection: the weight stream
        dict(name="gemm 2 tokens wide", op="gemm", M=2, N=8192, K=7168, res=False, out="f32"),
        # a batch of 16 through the output projection, added to the residual stream
        dict(name="gemm 16 tokens residual", op="gemm", M=16, N=7168, K=8192, res=True, out="bf16"),
        # a batch of 61 (64 slots, three of them empty)
        dict(name="gemm 61 tokens", op="gemm", M=61, N=4096, K=7168, res=False, out="bf16"),
        # a short prompt, ragged in every size
        dict(name="gemm ragged prompt", op="gemm", M=333, N=5001, K=2064, res=False, out="f32"),
        # a long prompt: bound by the matrix cores
        dict(name="gemm long prompt", op="gemm", M=8192, N=8192, K=7168, res=False, out="bf16"),
        # one token's norm, added to the residual stream: latency
        dict(name="norm 1 token", op="norm", M=1, K=7168, res=True, bf16=False),
        # a long prompt's norm: both the int8 codes and the bf16 value (a router reads it)
        dict(name="norm long prompt", op="norm", M=8191, K=7168, res=True, bf16=True),
        # a batch's gated product in front of the down projection, from the gate and up
        # projections' fp32 outputs
        dict(name="quant gated batch", op="quant", M=64, K=18432, gated=True, x="f32"),
        # a long prompt's attention output in front of the output projection
        dict(name="quant long prompt", op="quant", M=5003, K=8192, gated=False, x="bf16"),
        # decode: the whole MLP block for four tokens
        dict(name="mlp 4 tokens", op="mlp", M=4, H=7168, F=18432, res=True),
        # a prompt of odd length through the same block
        dict(name="mlp prompt", op="mlp", M=1501, H=7168, F=18432, res=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "norm", "quant", "mlp"])
    if op == "gemm":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 16, 8192), K=16 * _log(rng, 4, 448),
                    res=rng.random() < 0.3, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "norm":
        return dict(op=op, M=_log(rng, 1, 8192), K=8 * _log(rng, 16, 1024),
                    res=rng.random() < 0.7, bf16=rng.random() < 0.4)
    if op == "quant":
        gated = rng.random() < 0.5
        return dict(op=op, M=_log(rng, 1, 4096), K=8 * _log(rng, 16, 1152), gated=gated,
                    x=rng.choice(["bf16", "f32"]))
    return dict(op=op, M=_log(rng, 1, 1400), H=16 * _log(rng, 32, 448), F=16 * _log(rng, 64, 1152),
                res=rng.random() < 0.7)


# ---------------------------------------------------------------- inputs


def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + salt) % (1 << 62))
    return g


def _act(shape, seed, salt, sigma=1.0):
    """Activations as a decoder's residual stream has them: normal, with every 509th channel
    some times larger than the others."""
    v = torch.randn(shape, generator=_gen(seed, salt), device=DEV) * sigma
    v[:, 5::509] *= 6.0
    return v.to(torch.bfloat16)


def _codes(rows, cols, seed, salt, sigma):
    """Symmetric int8 codes and one scale a row of a normal matrix: a quantised checkpoint's
    weight (a scale a channel), or a batch of quantised tokens (a scale a token)."""
    codes = torch.empty((rows, cols), dtype=torch.int8, device=DEV)
    scales = torch.empty((rows,), dtype=torch.float32, device=DEV)
    g = _gen(seed, salt)
    for a in range(0, rows, 4096):
        w = torch.randn((min(rows, a + 4096) - a, cols), generator=g, device=DEV) * sigma
        amax = w.abs().amax(dim=1).clamp_min(1e-12)
        codes[a:a + w.shape[0]] = torch.round(w * (127.0 / amax)[:, None]).to(torch.int8)
        scales[a:a + w.shape[0]] = amax / 127.0
    return codes, scales


def prepare(case, seed):
    c, s = dict(case), dict(case=dict(case))
    M = c["M"]
    if c["op"] == "gemm":
        s["xq"], s["xs"] = _codes(M, c["K"], seed, 1, 1.0)
        s["wq"], s["ws"] = _codes(c["N"], c["K"], seed, 2, 0.02)
        s["r"] = _act((M, c["N"]), seed, 3) if c["res"] else None
        s["out"] = torch.empty((M, c["N"]), device=DEV,
                               dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    elif c["op"] == "norm":
        K = c["K"]
        s["x"] = _act((M, K), seed, 1)
        s["r"] = _act((M, K), seed, 3, 3.0) if c["res"] else None
        s["g"] = (1.0 + 0.2 * torch.randn((K,), generator=_gen(seed, 4), device=DEV)).to(torch.bfloat16)
        s["h"] = torch.empty_like(s["x"]) if c["res"] else None
        s["y"] = torch.empty_like(s["x"]) if c["bf16"] else None
        s["codes"] = torch.empty((M, K), dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty((M,), dtype=torch.float32, device=DEV)
        s["values"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "quant":
        K = c["K"]
        s["x"] = _act((M, 2 * K if c["gated"] else K), seed, 1)
        if c["x"] == "f32":
            s["x"] = s["x"].float() * 1.0009765  # no longer bf16 values
        s["codes"] = torch.empty((M, K), dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty((M,), dtype=torch.float32, device=DEV)
        s["values"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    else:
        H, F = c["H"], c["F"]
        s["x"] = _act((M, H), seed, 1)
        s["r"] = _act((M, H), seed, 3, 3.0) if c["res"] else None
        s["g"] = (1.0 + 0.2 * torch.randn((H,), generator=_gen(seed, 4), device=DEV)).to(torch.bfloat16)
        s["wgu"], s["sgu"] = _codes(2 * F, H, seed, 5, 0.02)
        s["wd"], s["sd"] = _codes(H, F, seed, 6, 0.02)
        s["out"] = torch.empty((M, H), dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms


def _rows_int8(t):
    """Codes (as fp32 whole numbers) and scale-defining maximum of each row."""
    amax = t.abs().amax(dim=1)
    inv = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
    return torch.round(t * inv[:, None]), amax


def _norm(x, r, g):
    s = x.float() if r is None else x.float() + r.float()
    ms = (s * s).sum(dim=1) / s.shape[1]
    inv = 1.0 / torch.sqrt(ms + EPS)
    return s, s * g.float(), inv


def _gated(x):
    half = x.shape[1] // 2
    gate, up = x[:, :half].float(), x[:, half:].float()
    return gate / (1.0 + torch.exp(-gate)) * up


def _product(xq, wq):
    """The whole-number products in fp32: sums of at most 1024 products are exact (below 2^24),
    their sum is taken in 64 bits."""
    K = xq.shape[1]
    acc = torch.zeros((xq.shape[0], wq.shape[0]), dtype=torch.float64, device=DEV)
    for k in range(0, K, 1024):
        acc += xq[:, k:k + 1024].float() @ wq[:, k:k + 1024].float().t()
    return acc


def _linear(xq, xs, wq, ws):
    return _product(xq, wq).float() * ws[None, :] * xs[:, None]


def _values(codes, scales):
    """What int8 codes stand for, in the model's type."""
    return (codes * scales[:, None]).to(torch.bfloat16)


def _plain(s):
    c = s["case"]
    if c["op"] == "gemm":
        y = _linear(s["xq"], s["xs"], s["wq"], s["ws"])
        if s["r"] is not None:
            y = s["r"].float() + y
        return y.to(s["out"].dtype)
    if c["op"] == "norm":
        v, t, inv = _norm(s["x"], s["r"], s["g"])
        codes, amax = _rows_int8(t)
        scales = amax * inv / 127.0
        return {"h": v.to(torch.bfloat16) if c["res"] else None,
                "y": (t * inv[:, None]).to(torch.bfloat16) if c["bf16"] else None,
                "scales": scales, "values": _values(codes, scales)}
    if c["op"] == "quant":
        codes, amax = _rows_int8(_gated(s["x"]) if c["gated"] else s["x"].float())
        return {"scales": amax / 127.0, "values": _values(codes, amax / 127.0)}
    v, t, inv = _norm(s["x"], s["r"], s["g"])
    q, amax = _rows_int8(t)
    gu = _linear(q, amax * inv / 127.0, s["wgu"], s["sgu"])  # fp32 up to its own codes
    p, amax = _rows_int8(_gated(gu))
    y = _linear(p, amax / 127.0, s["wd"], s["sd"])
    return (v.to(torch.bfloat16).float() + y).to(torch.bfloat16)


# ---------------------------------------------------------------- the framework's calls


def _own(s):
    import skinny_gemm_projection_amd as sg

    c = s["case"]
    if c["op"] == "gemm":
        kind = "y_bf16" if c["out"] == "bf16" else "y_f32"
        sg.skinny_gemm_int8(s["xq"], s["xs"], s["wq"], s["ws"], r=s["r"], **{kind: s["out"]})
        return s["out"]
    if c["op"] == "norm":
        sg.skinny_rmsnorm(s["x"], s["g"], EPS, r=s["r"], h=s["h"], y_bf16=s["y"],
                          codes=s["codes"], scales=s["scales"])
        torch.mul(s["codes"], s["scales"][:, None], out=s["values"])  # what the codes stand for
        return {"h": s["h"], "y": s["y"], "scales": s["scales"], "values": s["values"]}
    if c["op"] == "quant":
        sg.skinny_quant_int8(s["x"], gated=c["gated"], codes=s["codes"], scales=s["scales"])
        torch.mul(s["codes"], s["scales"][:, None], out=s["values"])
        return {"scales": s["scales"], "values": s["values"]}
    sg.skinny_mlp_int8_step(s["x"], s["g"], EPS, s["wgu"], s["sgu"], s["wd"], s["sd"], r=s["r"],
                            out=s["out"])
    return s["out"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- work and exact values


def work(case):
    c, M = case, case["M"]
    if c["op"] == "gemm":
        N, K = c["N"], c["K"]
        size = 2 if c["out"] == "bf16" else 4
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * (size + (2 if c["res"] else 0)),
                "flops": 2 * M * N * K}
    if c["op"] == "norm":
        K = c["K"]
        return {"bytes": M * K * (2 + (4 if c["res"] else 0) + (2 if c["bf16"] else 0) + 1) + 2 * K + 4 * M,
                "flops": 8 * M * K}
    if c["op"] == "quant":
        K = c["K"]
        return {"bytes": M * K * ((2 if c["gated"] else 1) * (2 if c["x"] == "bf16" else 4) + 1) + 4 * M,
                "flops": (10 if c["gated"] else 4) * M * K}
    H, F = c["H"], c["F"]
    return {"bytes": 3 * H * F + 4 * (2 * F + H) + M * H * (4 + (2 if c["res"] else 0)) + 2 * H,
            "flops": 6 * M * H * F + 8 * M * H + 10 * M * F}


def _exact_codes(t):
    amax = t.abs().max(dim=1, keepdim=True).values
    unit = amax / 127.0
    return torch.where(amax > 0, torch.round(t / unit.masked_fill(amax == 0, 1.0)), torch.zeros_like(t)), unit


def _exact_dot(a, w):
    return torch.matmul(a.double(), w.double().transpose(0, 1).contiguous())


def _exact_norm(s):
    v = s["x"].double()
    if s["r"] is not None:
        v = v + s["r"].double()
    rms = torch.sqrt(torch.mean(v ** 2, dim=1, keepdim=True) + EPS)
    return v, v / rms * s["g"].double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        y = _exact_dot(s["xq"], s["wq"]) * s["xs"].double().unsqueeze(1) * s["ws"].double().unsqueeze(0)
        return y if s["r"] is None else y + s["r"].double()
    if op == "norm":
        v, n = _exact_norm(s)
        codes, unit = _exact_codes(n)
        return {"h": v if case["res"] else None, "y": n if case["bf16"] else None,
                "scales": unit.squeeze(1), "values": codes * unit}
    if op == "quant":
        x, K = s["x"].double(), case["K"]
        t = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:] if case["gated"] else x
        codes, unit = _exact_codes(t)
        return {"scales": unit.squeeze(1), "values": codes * unit}
    v, n = _exact_norm(s)
    q, unit = _exact_codes(n)
    gu = _exact_dot(q, s["wgu"]) * unit * s["sgu"].double()
    F = case["F"]
    p, unit = _exact_codes(gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:])
    return v + _exact_dot(p, s["wd"]) * unit * s["sd"].double()
