"""Measured cases of the operators for block-scaled FP8 checkpoints with routed experts: the
row quantiser (e4m3 codes, a power-of-two scale for each block of 128), the product of such
codes, tokens sorted by expert and back (with the gradient of both), and the experts' step
made of them.

Shapes: 7168 and 8192 are the projection sizes this repository is benchmarked on, 384 experts
of width 2048 with 8 a token its routed-expert workload (48 is one of eight ranks' share of
them), 18432 its widest weight; the others are generic odd sizes.
"""
import math

import torch

own = False

DEV = "cuda"
B = 128        # block of the scales
TOP = 448.0    # largest e4m3 value
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # a batch of 16 tokens through a wide input projection: the weight stream
        dict(name="gemm 16 tokens wide", op="gemm", M=16, N=8192, K=7168, res=False, out="bf16"),
        # a short prompt, ragged in every size (the last block of K holds 16 codes)
        dict(name="gemm ragged prompt", op="gemm", M=777, N=5001, K=2064, res=False, out="f32"),
        # a long prompt through the output projection, added to the residual stream
        dict(name="gemm long prompt", op="gemm", M=8192, N=8192, K=7168, res=True, out="bf16"),
        # a batch's gated product in front of the down projection
        dict(name="quant gated batch", op="quant", M=61, K=18432, gated=True, x="f32"),
        # a long prompt's norm output in front of the first projections
        dict(name="quant long prompt", op="quant", M=8191, K=7168, gated=False, x="bf16"),
        # one token to its 8 experts: what the calls themselves cost
        dict(name="dispatch 1 token", op="dispatch", T=1, topk=8, E=384, total=384, K=7168, x="bf16"),
        # a prompt's rows laid out by expert
        dict(name="dispatch prompt", op="dispatch", T=4099, topk=8, E=384, total=384, K=7168, x="bf16"),
        # a batch's expert outputs back to their tokens, on a rank that holds half of the experts
        dict(name="combine batch", op="combine", T=61, topk=8, E=192, total=384, K=7168, x="bf16", res=False),
        # a prompt's expert outputs back to their tokens, added to the residual stream
        dict(name="combine prompt", op="combine", T=4099, topk=8, E=384, total=384, K=7168, x="bf16", res=True),
        # a training step's way back through both: gradients of the expert outputs, of the
        # weights and of the tokens
        dict(name="combine backward", op="grad", T=2050, topk=8, E=384, total=384, K=7168, x="bf16"),
        # decode: the experts of four tokens
        dict(name="experts 4 tokens", op="experts", T=4, topk=8, E=48, total=48, H=7168, F=2048, res=True),
        # a prompt of odd length
        dict(name="experts prompt", op="experts", T=2003, topk=8, E=48, total=48, H=7168, F=2048, res=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "quant", "dispatch", "combine", "grad", "experts", "experts"])
    if op == "gemm":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 16, 8192), K=16 * _log(rng, 4, 448),
                    res=rng.random() < 0.3, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "quant":
        return dict(op=op, M=_log(rng, 1, 3000), K=8 * _log(rng, 16, 2304), gated=rng.random() < 0.5,
                    x=rng.choice(["bf16", "f32"]))
    E = _log(rng, 8, 384)
    topk = rng.randint(1, 8)
    total = E * rng.choice([1, 1, 2])  # twice: the other half of the experts is another rank's
    if op == "experts":
        E = min(E, 48)
        return dict(op=op, T=_log(rng, 1, 2000), topk=topk, E=E, total=min(total, 2 * E),
                    H=16 * _log(rng, 32, 448), F=16 * _log(rng, 16, 128), res=rng.random() < 0.5)
    c = dict(op=op, T=_log(rng, 1, 2000), topk=topk, E=E, total=total, K=8 * _log(rng, 16, 896),
             x=rng.choice(["bf16", "bf16", "f32"]))
    if op == "combine":
        c["res"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs


def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + salt) % (1 << 62))
    return g


def _normal(shape, seed, salt, sigma=1.0):
    return torch.randn(shape, generator=_gen(seed, salt), device=DEV) * sigma


def _act(shape, seed, salt, sigma=1.0, dtype=torch.bfloat16):
    """Activations as a decoder's residual stream has them: normal, with every 509th channel
    some times larger than the others."""
    v = _normal(shape, seed, salt, sigma)
    v[:, 5::509] *= 6.0
    return v.to(dtype)


def _ceil(a, b):
    return -(-a // b)


def _act_codes(rows, cols, seed, salt):
    """A quantised batch: e4m3 codes [rows, cols] and scales [ceil(cols / 128), rows]."""
    kb = _ceil(cols, B)
    v = torch.zeros((rows, kb * B), device=DEV)
    v[:, :cols] = _act((rows, cols), seed, salt, dtype=torch.float32)
    v = v.view(rows, kb, B)
    amax = v.abs().amax(dim=2).clamp_min(1e-12)
    codes = (v * (TOP / amax)[:, :, None]).to(E4M3).view(torch.uint8).view(rows, kb * B)
    return codes[:, :cols].contiguous(), (amax / TOP).t().contiguous()


def _weight_codes(lead, rows, cols, seed, salt, sigma=0.02):
    """A block-scaled checkpoint's weight: e4m3 codes [*lead, rows, cols], one fp32 scale for
    each 128 x 128 block; magnitudes differ from block to block."""
    nb, kb = _ceil(rows, B), _ceil(cols, B)
    g = _gen(seed, salt)
    codes = torch.empty((*lead, rows, cols), dtype=torch.uint8, device=DEV)
    flat = codes.view(-1, rows, cols)
    for e in range(flat.shape[0]):  # an expert at a time: few temporaries
        w = torch.randn((rows, cols), generator=g, device=DEV).mul_(TOP / 5.7).clamp_(-TOP, TOP)
        flat[e] = w.to(E4M3).view(torch.uint8)
    scales = torch.rand((*lead, nb, kb), generator=g, device=DEV).add_(0.5).mul_(sigma * 5.7 / TOP)
    return codes, scales


def _routing(T, topk, total, seed):
    """Distinct experts of each token by a router's scores, and their softmax weights; some
    experts are more popular than others."""
    s = _normal((T, total), seed, 90) + 0.5 * _normal((1, total), seed, 91)
    top, ids = torch.topk(s, topk, dim=1)
    return ids.to(torch.int32).contiguous(), torch.softmax(top, dim=1).contiguous()


def _dtype(case):
    return torch.bfloat16 if case["x"] == "bf16" else torch.float32


def prepare(case, seed):
    c, s = case, dict(case=dict(case))
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        s["xq"], s["xs"] = _act_codes(M, K, seed, 1)
        s["wq"], s["ws"] = _weight_codes((), N, K, seed, 2)
        s["r"] = _act((M, N), seed, 3) if c["res"] else None
        s["out"] = torch.empty((M, N), device=DEV,
                               dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
        return s
    if c["op"] == "quant":
        M, K = c["M"], c["K"]
        s["x"] = _act((M, 2 * K if c["gated"] else K), seed, 1, dtype=_dtype(c))
        s["codes"] = torch.empty((M, K), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty((_ceil(K, B), M), dtype=torch.float32, device=DEV)
        return s
    T, topk, E = c["T"], c["topk"], c["E"]
    P = T * topk
    s["ids"], s["w"] = _routing(T, topk, c["total"], seed)
    if c["op"] == "experts":
        H, F = c["H"], c["F"]
        s["x"] = _act((T, H), seed, 1)
        s["r"] = _act((T, H), seed, 3, 3.0) if c["res"] else None
        s["wgu"], s["sgu"] = _weight_codes((E,), 2 * F, H, seed, 5)
        s["wd"], s["sd"] = _weight_codes((E,), H, F, seed, 6)
        s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        return s
    K, dt = c["K"], _dtype(c)
    s["offsets"] = torch.empty((E + 1,), dtype=torch.int32, device=DEV)
    s["sorted"] = torch.empty((P,), dtype=torch.int32, device=DEV)
    s["positions"] = torch.empty((T, topk), dtype=torch.int32, device=DEV)
    if c["op"] == "dispatch":
        s["x"] = _act((T, K), seed, 1, dtype=dt)
        s["rows"] = torch.zeros((P, K), dtype=dt, device=DEV)  # rows of left-out pairs stay zeros
        return s
    # the way back has the way there's table in hand
    s["positions"].copy_(_table(s["ids"], E)[2])
    s["ys"] = _act((P, K), seed, 1, dtype=dt)
    if c["op"] == "combine":
        s["r"] = _act((T, K), seed, 3, 3.0, dtype=dt) if c["res"] else None
        s["out"] = torch.empty((T, K), dtype=dt, device=DEV)
    else:
        s["dout"] = _act((T, K), seed, 4, dtype=dt)
        s["dxs"] = _act((P, K), seed, 7, dtype=dt)
        s["dys"] = torch.zeros((P, K), dtype=dt, device=DEV)
        s["dw"] = torch.empty((T, topk), dtype=torch.float32, device=DEV)
        s["dx"] = torch.empty((T, K), dtype=dt, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms


def _values(codes):
    return codes.view(E4M3).float()


def _per_channel(ws, rows, cols):
    """[.., ceil(rows / 128), ceil(cols / 128)] block scales as [.., rows, cols]."""
    w = ws.repeat_interleave(B, dim=-2)[..., :rows, :]
    return w.repeat_interleave(B, dim=-1)[..., :cols]


def _weight(wq, ws):
    return _values(wq) * _per_channel(ws, wq.shape[-2], wq.shape[-1])


def _rows(xq, xs):
    return _values(xq) * xs.t().repeat_interleave(B, dim=1)[:, :xq.shape[1]]


def _quant(v):
    """Codes (float8) and scales [ceil(K / 128), M] of fp32 rows: the scale is the least power
    of two (from 2^-126 on) that brings the block's values to at most 448."""
    M, K = v.shape
    kb = _ceil(K, B)
    t = torch.zeros((M, kb * B), device=DEV)
    t[:, :K] = v
    t = t.view(M, kb, B)
    man, ex = torch.frexp(t.abs().amax(dim=2))  # man in [0.5, 1); 448 = 0.875 * 2^9
    ex = torch.where(man > 0, ex, torch.full_like(ex, -126))  # a block of zeros: the least scale
    unit = torch.ldexp(torch.ones_like(man), (ex - 9 + (man > 0.875).int()).clamp_min(-126))
    codes = (t / unit[:, :, None]).to(E4M3)  # the quotient is exact
    return codes.view(M, kb * B)[:, :K].contiguous(), unit.t().contiguous()


def _gated(x):
    half = x.shape[1] // 2
    gate, up = x[:, :half].float(), x[:, half:].float()
    return gate / (1.0 + torch.exp(-gate)) * up


def _table(ids, E):
    """offsets [E + 1], the pairs sorted by expert (-1 behind the last) and their positions."""
    flat = ids.reshape(-1).long()
    ok = (flat >= 0) & (flat < E)
    key = torch.where(ok, flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(counts, 0)
    positions = torch.empty_like(order)
    positions[order] = torch.arange(order.numel(), device=ids.device)
    positions = torch.where(ok, positions, torch.full_like(positions, -1))
    behind = torch.arange(order.numel(), device=ids.device) >= offsets[E]
    order = torch.where(behind, torch.full_like(order, -1), order)
    return offsets.to(torch.int32), order.to(torch.int32), positions.to(torch.int32).view(ids.shape)


def _combine(ys, positions, w, r):
    """sum_j w[t, j] ys[positions[t, j]] in fp32, left-out pairs skipped."""
    rows = ys[positions.clamp_min(0).long()].float()
    rows = torch.where((positions >= 0)[:, :, None], rows, torch.zeros_like(rows))
    out = (rows if w is None else rows * w[:, :, None]).sum(dim=1)
    return out if r is None else r.float() + out


def _expert_rows(xf, ids, E):
    """Rows padded to one length an expert [E, longest, K], and each pair's place among them."""
    offsets, _, positions = _table(ids, E)
    counts = offsets[1:] - offsets[:-1]
    longest = max(1, int(counts.max()))
    flat, pos = ids.reshape(-1).long(), positions.reshape(-1).long()
    valid = pos >= 0
    e = torch.where(valid, flat, torch.zeros_like(flat))
    place = torch.where(valid, e * longest + pos - offsets[e], torch.full_like(pos, E * longest))
    rows = torch.zeros((E * longest + 1, xf.shape[1]), device=DEV)
    token = torch.arange(ids.shape[0], device=DEV).repeat_interleave(ids.shape[1])
    rows[place] = xf[token]
    return rows[:-1].view(E, longest, -1), place, valid


def _experts(s):
    c = s["case"]
    T, topk, E, H, F = c["T"], c["topk"], c["E"], c["H"], c["F"]
    xf = _rows(*_as_bytes(_quant(s["x"].float())))
    if T * topk <= E:  # few pairs: each takes its expert's weights
        flat = s["ids"].reshape(-1).long()
        valid = (flat >= 0) & (flat < E)
        e = torch.where(valid, flat, torch.zeros_like(flat))
        token = torch.arange(T, device=DEV).repeat_interleave(topk)
        u = torch.bmm(_weight(s["wgu"][e], s["sgu"][e]), xf[token][:, :, None]).squeeze(2)
        p = _rows(*_as_bytes(_quant(_gated(u))))
        y = torch.bmm(_weight(s["wd"][e], s["sd"][e]), p[:, :, None]).squeeze(2)
    else:
        rows, place, valid = _expert_rows(xf, s["ids"], E)
        n = rows.shape[1]
        u = torch.bmm(rows, _weight(s["wgu"], s["sgu"]).transpose(1, 2).contiguous())
        p = _rows(*_as_bytes(_quant(_gated(u.view(E * n, 2 * F)))))
        y = torch.bmm(p.view(E, n, F), _weight(s["wd"], s["sd"]).transpose(1, 2).contiguous())
        y = y.view(E * n, H)[place.clamp_max(E * n - 1)]
    y = torch.where(valid[:, None], y, torch.zeros_like(y)).view(T, topk, H)
    out = (y * s["w"][:, :, None]).sum(dim=1)
    return (out if s["r"] is None else s["r"].float() + out).to(torch.bfloat16)


def _as_bytes(q):
    return q[0].view(torch.uint8), q[1]


def _plain(s):
    c = s["case"]
    if c["op"] == "gemm":
        y = _rows(s["xq"], s["xs"]) @ _weight(s["wq"], s["ws"]).t().contiguous()
        if s["r"] is not None:
            y = s["r"].float() + y
        return y.to(s["out"].dtype)
    if c["op"] == "quant":
        codes, scales = _quant(_gated(s["x"]) if c["gated"] else s["x"].float())
        return {"codes": codes, "scales": scales}
    if c["op"] == "dispatch":
        offsets, order, positions = _table(s["ids"], c["E"])
        rows = torch.zeros_like(s["rows"])
        rows[torch.arange(rows.shape[0], device=DEV)] = torch.where(
            (order >= 0)[:, None], s["x"][(order.clamp_min(0) // c["topk"]).long()], rows)
        return {"offsets": offsets, "sorted": order, "positions": positions, "rows": rows}
    if c["op"] == "combine":
        return _combine(s["ys"], s["positions"], s["w"], s["r"]).to(s["out"].dtype)
    if c["op"] == "grad":
        pos = s["positions"].reshape(-1).long()
        ok = pos >= 0
        place = torch.where(ok, pos, torch.full_like(pos, pos.numel()))
        d = s["dout"].float()
        dys = torch.zeros((pos.numel() + 1, c["K"]), device=DEV)
        dys[place] = (d[:, None, :] * s["w"][:, :, None]).view(-1, c["K"])
        rows = s["ys"][pos.clamp_min(0)].float().view(*s["w"].shape, -1)
        dw = (rows * d[:, None, :]).sum(dim=2)
        dx = _combine(s["dxs"], s["positions"], None, None)
        dt = s["dys"].dtype
        behind = torch.arange(pos.numel(), device=DEV) >= ok.sum()
        return {"dys": torch.where(behind[:, None], 0.0, dys[:-1]).to(dt),
                "dw": torch.where(ok.view_as(dw), dw, torch.zeros_like(dw)), "dx": dx.to(dt)}
    return _experts(s)


# ---------------------------------------------------------------- the framework's calls


def _own(s):
    import skinny_gemm_projection_amd as sg

    c = s["case"]
    if c["op"] == "gemm":
        kind = "y_bf16" if c["out"] == "bf16" else "y_f32"
        sg.skinny_gemm_fp8_block(s["xq"], s["xs"], s["wq"], s["ws"], r=s["r"], **{kind: s["out"]})
        return s["out"]
    if c["op"] == "quant":
        sg.skinny_quant_fp8(s["x"], gated=c["gated"], codes=s["codes"], scales=s["scales"])
        return {"codes": s["codes"].view(E4M3), "scales": s["scales"]}
    if c["op"] == "dispatch":
        sg.skinny_moe_sort(s["ids"], c["E"], expert_offsets=s["offsets"], sorted_pairs=s["sorted"],
                           positions=s["positions"])
        sg.skinny_moe_gather(s["x"], s["positions"], out=s["rows"])
        return {"offsets": s["offsets"], "sorted": s["sorted"], "positions": s["positions"],
                "rows": s["rows"]}
    if c["op"] == "combine":
        return sg.skinny_moe_combine(s["ys"], s["positions"], s["w"], r=s["r"], out=s["out"])
    if c["op"] == "grad":
        sg.skinny_moe_combine_grad(s["dout"], s["ys"], s["positions"], s["w"], d_rows=s["dys"],
                                   d_weights=s["dw"])
        sg.skinny_moe_combine(s["dxs"], s["positions"], None, out=s["dx"])
        return {"dys": s["dys"], "dw": s["dw"], "dx": s["dx"]}
    return sg.skinny_moe_fp8_step(s["x"], s["ids"], s["w"], s["wgu"], s["sgu"], s["wd"], s["sd"],
                                  r=s["r"], out=s["out"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- work and exact values


def work(case):
    c = case
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        size = (2 if c["out"] == "bf16" else 4) + (2 if c["res"] else 0)
        kb = _ceil(K, B)
        return {"bytes": M * K + N * K + 4 * kb * (M + _ceil(N, B)) + M * N * size, "flops": 2 * M * N * K}
    if c["op"] == "quant":
        M, K = c["M"], c["K"]
        size = (2 if c["x"] == "bf16" else 4) * (2 if c["gated"] else 1)
        return {"bytes": M * K * (size + 1) + 4 * M * _ceil(K, B), "flops": (10 if c["gated"] else 4) * M * K}
    T, E = c["T"], c["E"]
    P = T * c["topk"]
    here = P * E / c["total"]  # pairs of experts held here
    if c["op"] == "experts":
        H, F = c["H"], c["F"]
        touched = min(E, here) if here < 4 * E else E
        return {"bytes": int(touched * 3 * H * F + T * H * (4 + (2 if c["res"] else 0)) + 8 * P),
                "flops": int(here * 6 * H * F)}
    K, size = c["K"], 2 if c["x"] == "bf16" else 4
    if c["op"] == "dispatch":
        return {"bytes": int((T + here) * K * size + 12 * P + 4 * E), "flops": P}
    if c["op"] == "combine":
        return {"bytes": int((here + T * (2 if c["res"] else 1)) * K * size + 8 * P),
                "flops": int(2 * here * K)}
    return {"bytes": int((3 * here + 2 * T) * K * size + 12 * P), "flops": int(4 * here * K)}


def exact(case, seed):
    op = case["op"]
    if op == "dispatch":
        return None  # only copies
    s = prepare(case, seed)
    f64 = torch.float64

    def value(codes):  # e4m3 by its definition: sign, 4 bits of exponent (bias 7), 3 of mantissa
        b = codes.to(torch.int64)
        ex, man = (b >> 3) & 15, (b & 7).to(f64)
        mag = torch.where(ex == 0, man * 2.0 ** -9, torch.ldexp(8 + man, ex.to(f64) - 10))
        return torch.where(b >= 128, -mag, mag)

    def nearest(v):  # e4m3 value next to v, half to even
        step = torch.ldexp(torch.ones_like(v), torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        return torch.round(v / step) * step

    def blocks(v):
        pad = -v.shape[-1] % B
        return torch.nn.functional.pad(v, (0, pad)).unflatten(-1, (-1, B))

    def codes_of(v):
        t = blocks(v)
        ratio = (t.abs().amax(dim=-1) / TOP).clamp_min(2.0 ** -126)
        unit = torch.exp2(torch.floor(torch.log2(ratio)))
        unit = torch.where(unit * 2 <= ratio, unit * 2, unit)  # whichever way the logarithm rounded
        unit = torch.where(unit < ratio, unit * 2, unit)
        return nearest(t / unit[..., None]), unit

    def dequantised(v):
        q, unit = codes_of(v)
        return (q * unit[..., None]).flatten(-2)[..., :v.shape[-1]]

    def weight(wq, ws):
        n, k = wq.shape
        full = ws.to(f64).repeat_interleave(B, 0)[:n].repeat_interleave(B, 1)[:, :k]
        return value(wq) * full

    def swiglu(u):
        half = u.shape[1] // 2
        return u[:, :half] * torch.sigmoid(u[:, :half]) * u[:, half:]

    if op == "gemm":
        x = value(s["xq"]) * s["xs"].to(f64).t().repeat_interleave(B, 1)[:, :case["K"]]
        y = x @ weight(s["wq"], s["ws"]).t().contiguous()
        return y if s["r"] is None else y + s["r"].to(f64)
    if op == "quant":
        v = s["x"].to(f64)
        q, unit = codes_of(swiglu(v) if case["gated"] else v)
        return {"codes": q.flatten(1)[:, :case["K"]].contiguous(), "scales": unit.t().contiguous()}
    w = s["w"].to(f64)
    if op == "experts":
        x = dequantised(s["x"].to(f64))
        out = torch.zeros_like(x) if s["r"] is None else s["r"].to(f64)
        for e in range(case["E"]):
            t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
            if t.numel() == 0:
                continue
            u = x[t] @ weight(s["wgu"][e], s["sgu"][e]).t().contiguous()
            y = dequantised(swiglu(u)) @ weight(s["wd"][e], s["sd"][e]).t().contiguous()
            out[t] += y * w[t, j][:, None]  # a token meets an expert once
        return out
    pos = s["positions"].long()
    held = (pos >= 0).to(f64)
    out = torch.zeros((case["T"], case["K"]), dtype=f64, device=DEV)
    if op == "combine":
        if s["r"] is not None:
            out += s["r"].to(f64)
        for j in range(case["topk"]):
            out += s["ys"][pos[:, j].clamp_min(0)].to(f64) * (w[:, j] * held[:, j])[:, None]
        return out
    dys = torch.zeros(s["dys"].shape, dtype=f64, device=DEV)
    dw = torch.zeros_like(w)
    d = s["dout"].to(f64)
    for j in range(case["topk"]):
        on = pos[:, j] >= 0
        dys[pos[on, j]] = d[on] * w[on, j][:, None]
        dw[on, j] = (s["ys"][pos[on, j]].to(f64) * d[on]).sum(dim=1)
        out[on] += s["dxs"][pos[on, j]].to(f64)
    return {"dys": dys, "dw": dw, "dx": out}
