"""GPU tests of how the block-scaled FP8 operators and the rows by expert are used: captured into
HIP graphs and replayed with other inputs, on other streams, by two callers at once, with offsets
past 32 bits, no tokens, one expert's crowd and an expert named twice by a token.  The results of
eager calls, which other tests check against references, are what the graphs have to repeat bit
for bit."""
import pytest
import torch

import fp8_block_ref as ref
import skinny_gemm_projection_amd as sg
from gpu_common import DEV, announce, counters_delta
from test_gpu_fp8_block import normal, step_inputs, step_reference, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

BF16, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8


class Step:
    """One captured experts' step with buffers of its own."""

    def __init__(self, T, topk, E, H, F, seed):
        case = step_inputs(T, topk, E, H, F, E, seed)
        self.x, self.ids, self.w, *self.weights, self.r = [t.to(DEV) for t in case]
        self.E, self.seed = E, seed
        self.out = torch.zeros((T, H), dtype=BF16, device=DEV)
        self.ws = torch.empty(sg.skinny_moe_fp8_step_workspace(T, topk, E, H, F), dtype=U8, device=DEV)

    def call(self, out, ws):
        return sg.skinny_moe_fp8_step(self.x, self.ids, self.w, *self.weights, r=self.r, out=out,
                                      workspace=ws)

    def capture(self):
        self.call(self.out, self.ws)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=torch.cuda.Stream()):
            self.call(self.out, self.ws)
        torch.cuda.synchronize()

    def new_inputs(self, i):
        T, H = self.x.shape
        self.x.copy_(normal((T, H), 100 * i + self.seed))
        ids, w = ref.routing(T, self.ids.shape[1], self.E, self.E + i, 7 * i + self.seed)
        self.ids.copy_(ids)
        self.w.copy_(w)


@pytest.mark.parametrize("T", [3, 40, 900])
def test_two_captured_steps(T):
    """Replayed in turn and at once on two streams, with other tokens and routes in between."""
    announce(f"captured steps T={T}")
    a, b = Step(T, 6, 12, 272, 256, 1), Step(T + 1, 6, 9, 400, 144, 2)
    a.capture()
    b.capture()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        want = []
        for s in (a, b):
            s.new_inputs(i)
            want.append(s.call(None, None))  # eager, between the replays
            s.out.fill_(float("nan"))
            s.ws.fill_(255)
        torch.cuda.synchronize()
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s.graph.replay()
                if i % 2 == 0:
                    st.synchronize()
        torch.cuda.synchronize()
        for s, y in zip((a, b), want):
            assert torch.equal(s.out, y), f"replay {i}"


@pytest.mark.parametrize("T,topk,E", [(16, 8, 20), (700, 8, 20), (9001, 8, 33)])
def test_captured_parts(T, topk, E):
    """Sort (in one, two and three launches), rows there and back with gradients, the quantiser and
    products with and without a workspace, one after the other in one graph."""
    announce(f"captured parts T={T} topk={topk} E={E}")
    K, N = 144, 70
    ids, w = ref.routing(T, topk, E, E + 3, 3)
    ids, w = ids.to(DEV), w.to(DEV)
    x = normal((T, K), 4).to(DEV)
    wq = ref.rand_codes(E * N, K, 5).view(E, N, K).to(DEV)
    ws = ref.rand_scales((E, 1, 2), 6).to(DEV)
    big = [ref.rand_codes(200, 9008, 7), ref.rand_scales((71, 200), 8), ref.rand_codes(37, 9008, 9),
           ref.rand_scales((1, 71), 10)]
    big = [t.to(DEV) for t in big]
    assert sg.skinny_gemm_fp8_block_workspace(200, 37, 9008, True) > 0

    def issue():
        offsets, order, positions = sg.skinny_moe_sort(ids, E)
        rows = sg.skinny_moe_gather(x, positions)
        q, s = sg.skinny_quant_fp8(x)
        y, _ = sg.grouped_skinny_gemm_fp8(q, s, wq, ws, offsets, sorted_pairs=order, topk=topk)
        z = sg.skinny_moe_combine(rows, positions, w, r=x)
        d, dw = sg.skinny_moe_combine_grad(z, rows, positions, w)
        return (offsets, order, positions, rows, q, s, y, z, d, dw, *sg.skinny_gemm_fp8_block(*big)[:1])

    issue()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        outs = issue()
    torch.cuda.synchronize()
    for i in range(3):
        x.copy_(normal((T, K), 50 + i))
        ids.copy_(ref.routing(T, topk, E, E + i, 60 + i)[0])
        want = issue()
        for t in outs:
            t.fill_(0 if t.dtype is U8 else -3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for j, (got, y) in enumerate(zip(outs, want)):
            assert torch.equal(got, y), f"replay {i}, output {j}"


@pytest.mark.parametrize("T", [5, 600])
def test_on_a_stream_of_its_own(T):
    """Outputs and workspaces that a call allocates belong to the stream that it is given: inputs
    made on that stream, and late, are waited for, and nothing is handed out again too early."""
    topk, E, H, F = 4, 8, 272, 256
    case = [t.to(DEV) for t in step_inputs(T, topk, E, H, F, E)]
    want = sg.skinny_moe_fp8_step(*case[:7], r=case[7])
    offsets, order, positions = sg.skinny_moe_sort(case[1], E)
    rows = sg.skinny_moe_gather(case[0], positions)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            a = torch.randn((4096, 4096), device=DEV)
            for _ in range(20):
                a = a @ a * 1e-2
            late = [case[0] + (a[0, 0] * 0).nan_to_num().to(BF16), *case[1:]]
        got = sg.skinny_moe_fp8_step(*late[:7], r=late[7], stream=stream)
        o, s, p = sg.skinny_moe_sort(late[1], E, stream=stream)
        r = sg.skinny_moe_gather(late[0], p, stream=stream)
        junk = [torch.full((1 << 16,), 255, dtype=U8, device=DEV) for _ in range(8)]
        stream.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(r, rows)
        assert torch.equal(o, offsets) and torch.equal(s, order) and torch.equal(p, positions)
        del junk


def test_no_tokens():
    f = dict(device=DEV)
    for topk in (1, 8):
        ids = torch.empty((0, topk), dtype=I32, **f)
        w = torch.empty((0, topk), **f)
        offsets, order, positions = sg.skinny_moe_sort(ids, 5)
        assert offsets.tolist() == [0] * 6 and order.numel() == 0 and positions.shape == (0, topk)
        x = torch.empty((0, 16), dtype=BF16, **f)
        assert sg.skinny_moe_gather(x, positions).shape == (0, 16)
        assert sg.skinny_moe_combine(x, positions, w).shape == (0, 16)
        d, dw = sg.skinny_moe_combine_grad(x, x, positions, w)
        assert d.shape == (0, 16) and dw.shape == (0, topk)
        q, s = sg.skinny_quant_fp8(x)
        assert q.shape == (0, 16) and s.shape == (1, 0)
        wq, ws = torch.empty((5, 7, 16), dtype=U8, **f), torch.empty((5, 1, 1), **f)
        assert sg.grouped_skinny_gemm_fp8(q, s, wq, ws, offsets)[0].shape == (0, 7)
        up, us = torch.empty((5, 32, 16), dtype=U8, **f), torch.empty((5, 1, 1), **f)
        dn, ds = torch.empty((5, 16, 16), dtype=U8, **f), torch.empty((5, 1, 1), **f)
        assert sg.skinny_moe_fp8_step(x, ids, w, up, us, dn, ds).shape == (0, 16)


@pytest.mark.parametrize("T", [3, 30, 400])
def test_an_expert_named_twice(T):
    """A token that names an expert in two slots has two rows there, and one crowded expert with
    the others empty is no different."""
    topk, E, H, F = 4, 40, 144, 128
    x, _, w, *weights, r = step_inputs(T, topk, E, H, F, E)
    ids = torch.tensor([7, 3, 7, 7], dtype=I32).repeat(T, 1)
    ids[0] = torch.tensor([5, -1, 5, E], dtype=I32)
    want, bound = step_reference(x, ids, w, *weights, r, E)
    before = sg.skinny_gemm_get_counters()
    out = sg.skinny_moe_fp8_step(*[t.to(DEV) for t in (x, ids, w, *weights)], r=r.to(DEV))
    ran = counters_delta(before, sg.skinny_gemm_get_counters())
    within(out, want, bound, f"T={T}")
    # sort, codes (of the gated product too where it does not give its own), two products, rows
    assert ran[sg.SG_KERNEL_MOE_SORT] == 1 and ran[sg.SG_KERNEL_FP8_BLOCK] == 2
    assert ran[sg.SG_KERNEL_MOE_ROWS] == 1
    assert ran[sg.SG_KERNEL_QUANT_FP8] == (1 if T == 400 else 2)
    assert sum(ran) == 4 + ran[sg.SG_KERNEL_QUANT_FP8]


# ------------------------------------------------------------------ offsets past 32 bits


def codes_on_device(rows, cols, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = torch.randint(0, 256, (rows, cols), generator=g, device=DEV, dtype=U8)
    c &= 0xbf  # no code past 1.875, no NaN
    return c


def test_long_quant():
    M, K = 70001, 65536  # 4.6e9 codes
    announce(f"quant {M} x {K}")
    x = torch.empty((M, K), dtype=BF16, device=DEV).normal_()
    codes, scales = sg.skinny_quant_fp8(x)
    for i in (0, 32768, 65535, 65536, M - 1):
        q, s = ref.quant(x[i:i + 1].cpu())
        assert torch.equal(ref.value(codes[i:i + 1].cpu()), q), i
        assert torch.equal(scales[:, i:i + 1].cpu(), s.to(F32)), i


@pytest.mark.parametrize("M", [3, 40])
def test_long_weights(M):
    N, K = (1 << 20) - 3, 4112  # 4.3e9 codes
    announce(f"product {M} x {N} x {K}")
    wq, xq = codes_on_device(N, K, 1), codes_on_device(M, K, 2)
    xs = ref.rand_scales((ref.ceil(K), M), 3)
    ws = ref.rand_scales((ref.ceil(N), ref.ceil(K)), 4)
    cols = torch.tensor([0, 1, 4095, 524287, 1044479, 1044480, 1044481, N - 129, N - 2, N - 1])
    y, A = sampled(xq.cpu(), xs, wq[cols.to(DEV)].cpu(), ws[cols // 128])
    out, _ = sg.skinny_gemm_fp8_block(xq, xs.to(DEV), wq, ws.to(DEV))
    within(out[:, cols.to(DEV)], y, ref.wide_rel(K) * A, "fp32")
    y16 = torch.empty((M, N), dtype=BF16, device=DEV)
    sg.skinny_gemm_fp8_block(xq, xs.to(DEV), wq, ws.to(DEV), y_bf16=y16)
    loose = ref.fp8_rel(K) * A
    within(y16[:, cols.to(DEV)], y, loose + 2.0 ** -8 * (y.abs() + loose), "bf16")


def sampled(xq, xs, wq, ws):
    """ref.product for rows of W that have block scales of their own, [rows, blocks]."""
    K = xq.shape[1]
    x = ref.rows64(xq, xs)
    w = ref.value(wq) * ws.to(F64).repeat_interleave(ref.B, 1)[:, :K]
    return x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_outputs(dtype):
    M, N, K = 4500, 1000003, 48  # 4.5e9 outputs
    announce(f"product {M} x {N} x {K} {dtype}")
    wq, xq = codes_on_device(N, K, 1), codes_on_device(M, K, 2)
    xs, ws = ref.rand_scales((1, M), 3), ref.rand_scales((ref.ceil(N), 1), 4)
    rows = torch.tensor([0, 1, 2147, 4294, 4295, M - 1])
    cols = torch.tensor([0, 5, 483647, 967295, 967296, N - 2, N - 1])
    y, A = sampled(xq[rows.to(DEV)].cpu(), xs[:, rows], wq[cols.to(DEV)].cpu(), ws[cols // 128])
    out = torch.empty((M, N), dtype=dtype, device=DEV)
    sg.skinny_gemm_fp8_block(xq, xs.to(DEV), wq, ws.to(DEV), **{"y_f32" if dtype is F32 else "y_bf16": out})
    loose = ref.wide_rel(K) * A if dtype is F32 else ref.fp8_rel(K) * A
    if dtype is BF16:
        loose = loose + 2.0 ** -8 * (y.abs() + loose)
    within(out[rows.to(DEV)][:, cols.to(DEV)], y, loose, "sampled")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_rows_by_expert(dtype):
    """Rows by expert there and back, where rows * K * size passes 2^32, and x's does not."""
    T, topk, E, K = 33001, 8, 24, 16384 if dtype is BF16 else 8192
    announce(f"rows by expert {T} x {topk} x {K} {dtype}")
    ids, w = ref.routing(T, topk, E, E, 3)
    offsets, order, positions = sg.skinny_moe_sort(ids.to(DEV), E)
    x = torch.empty((T, K), dtype=dtype, device=DEV).normal_()
    rows = sg.skinny_moe_gather(x, positions)
    assert rows.numel() * rows.element_size() > 1 << 32
    pairs = torch.tensor([0, 65535, 131072, T * topk // 2, T * topk - 1], device=DEV)
    assert torch.equal(rows[pairs], x[order[pairs].long() // topk])
    out = sg.skinny_moe_combine(rows, positions, w.to(DEV))
    d, dw = sg.skinny_moe_combine_grad(x, rows, positions, w.to(DEV), d_rows=rows.clone())
    u = 2.0 ** -8 if dtype is BF16 else ref.U
    for t in (0, 16384, 32768, T - 1):
        mine, xt = positions[t].long(), x[t].cpu().to(F64)
        y = w[t].to(F64).sum() * xt  # rows are copies of x[t]
        within(out[t], y, (topk + 2) * ref.U * xt.abs() + u * y.abs() * (1 + u), "combine")
        want = w[t].to(F64)[:, None] * xt
        within(d[mine], want, 2 * u * want.abs(), "d_rows")
        dot = (xt * xt).sum()
        within(dw[t], dot.repeat(topk), (K / 64 + 20) * ref.U * dot.repeat(topk), "d_weights")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_experts(dtype):
    """Weights of experts past 2^32 codes, rows of codes past 2^31 and outputs past 2^32."""
    P, E, N, K = 140007, 9, 32005, 16384
    announce(f"grouped {P} x {E} x {N} x {K} {dtype}")
    wq = codes_on_device(E * N, K, 1).view(E, N, K)
    xq = codes_on_device(P, K, 2)
    xs = ref.rand_scales((ref.ceil(K), P), 3)
    ws = ref.rand_scales((E, ref.ceil(N), ref.ceil(K)), 4)
    sizes = [0, 1, 3, 300, 0, 0, 40000, 0, P - 40304 - 57]
    offsets = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=I32)
    out = torch.full((P, N), -7.0, dtype=dtype, device=DEV)
    assert wq.numel() > 1 << 32 and xq.numel() > 1 << 31 and out.numel() > 1 << 32
    sg.grouped_skinny_gemm_fp8(xq, xs.to(DEV), wq, ws.to(DEV), offsets.to(DEV),
                               **{"y_f32" if dtype is F32 else "y_bf16": out})
    cols = torch.tensor([0, 1, 16000, N - 2, N - 1])
    for e in (e for e in range(E) if sizes[e]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        rows = torch.tensor(sorted({lo, (lo + hi) // 2, max(lo, hi - 2), hi - 1}))
        y, A = sampled(xq[rows.to(DEV)].cpu(), xs[:, rows], wq[e][cols.to(DEV)].cpu(), ws[e][cols // 128])
        loose = ref.wide_rel(K) * A if dtype is F32 else ref.fp8_rel(K) * A
        if dtype is BF16:
            loose = loose + 2.0 ** -8 * (y.abs() + loose)
        within(out[rows.to(DEV)][:, cols.to(DEV)], y, loose, f"expert {e}")
    assert (out[int(offsets[E]):] == -7.0).all()
