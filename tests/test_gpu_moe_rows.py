"""GPU tests of the sort by expert, of rows brought to their experts and back, and of the gradients
of both, against fp8_block_ref.py in 64 bits."""
import pytest
import torch

import fp8_block_ref as ref
import skinny_gemm_projection_amd as sg
from gpu_common import DEV, announce, counters_delta

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64

SORT = [(0, 3, 5), (1, 1, 1), (1, 8, 384), (3, 32, 4096), (64, 1, 2), (65, 8, 7), (512, 8, 384),
        (4096, 1, 1), (4097, 1, 3), (513, 8, 130), (1025, 4, 4096), (5000, 8, 384), (2048, 2, 64),
        (100, 32, 50), (20011, 6, 48), (37, 7, 1025), (64, 4, 1024), (8191, 8, 4096), (8193, 8, 384),
        (32768, 2, 3)]


@pytest.mark.parametrize("T,topk,E", SORT)
@pytest.mark.parametrize("kind", ["routed", "one expert", "left out"])
def test_sort(T, topk, E, kind):
    announce(f"moe_sort T={T} topk={topk} E={E} {kind}")
    g = ref.gen(T + E)
    ids = torch.randint(0, E, (T, topk), generator=g, dtype=torch.int32)
    if kind == "one expert":
        ids[:] = E - 1
    if kind == "left out":
        out = torch.rand((T, topk), generator=g) < 0.4
        bad = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64)
        ids = torch.where(out, bad[torch.randint(0, 4, (T, topk), generator=g)].to(torch.int32), ids)
    offsets, order, positions = ref.table(ids, E)
    before = sg.skinny_gemm_get_counters()
    got = sg.skinny_moe_sort(ids.to(DEV), E)
    ran = counters_delta(before, sg.skinny_gemm_get_counters())
    P = T * topk
    assert ran[sg.SG_KERNEL_MOE_SORT] == sum(ran) == (
        1 if P <= 4096 else 2 if P <= 1 << 16 and P * E <= 1 << 27 else 3)
    for a, b, name in zip(got, (offsets, order, positions), ("offsets", "sorted", "positions")):
        assert torch.equal(a.cpu(), b), name


ROWS = [(1, 1, 1, 8), (1, 8, 40, 7168), (5, 3, 4, 136), (61, 8, 16, 520), (300, 2, 9, 2056), (33, 9, 40, 64),
        (7, 32, 64, 264), (130, 4, 3, 1032), (3, 8, 20, 65536)]


def rows_case(T, topk, E, K, dtype, seed=1):
    ids, w = ref.routing(T, topk, E, E + E // 2, seed)
    offsets, order, positions = ref.table(ids, E)
    make = lambda shape, s: torch.randn(shape, generator=ref.gen(s)).to(dtype)  # noqa: E731
    return ids, w, offsets, order, positions, make


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,topk,E,K", ROWS)
def test_gather_and_combine(T, topk, E, K, dtype):
    announce(f"moe rows T={T} topk={topk} E={E} K={K} {dtype}")
    ids, w, offsets, order, positions, make = rows_case(T, topk, E, K, dtype)
    P, valid = T * topk, int(offsets[E])
    x, rows, r = make((T, K), 2), make((P, K), 3), make((T, K), 4)
    pos = positions.to(DEV)
    guard = torch.full((P + 2, K), -7.0, dtype=dtype, device=DEV)
    sg.skinny_moe_gather(x.to(DEV), pos, out=guard[:P])
    assert torch.equal(guard[:valid].cpu(), x[order[:valid].long() // topk]), "gather"
    assert (guard[valid:] == -7.0).all(), "rows that no position names are left as they were"
    new = sg.skinny_moe_gather(x.to(DEV), pos)
    assert torch.equal(new[:valid], guard[:valid]) and (new[valid:] == 0).all()
    half = ref.step_of(dtype)
    for weights in (w, None):
        for res in (r, None):
            want, mag = ref.combine(rows, positions, weights, res)
            # topk fused additions and the residual's, in fp32, then the output's rounding
            acc = (topk + 1) * ref.U * mag
            bound = acc + (half * (want.abs() + acc) if dtype is BF16 else 0)
            out = sg.skinny_moe_combine(rows.to(DEV), pos, None if weights is None else w.to(DEV),
                                        r=None if res is None else r.to(DEV))
            err = (out.cpu().to(F64) - want).abs()
            assert (err <= bound).all(), f"combine: {float((err - bound).max())}"
    inplace = r.to(DEV)
    a = sg.skinny_moe_combine(rows.to(DEV), pos, w.to(DEV), r=r.to(DEV))
    sg.skinny_moe_combine(rows.to(DEV), pos, w.to(DEV), r=inplace, out=inplace)
    assert torch.equal(a, inplace), "out may be r"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,topk,E,K", ROWS)
def test_combine_grad(T, topk, E, K, dtype):
    announce(f"moe grad T={T} topk={topk} E={E} K={K} {dtype}")
    ids, w, offsets, order, positions, make = rows_case(T, topk, E, K, dtype)
    P, valid = T * topk, int(offsets[E])
    d_out, rows = make((T, K), 2), make((P, K), 3)
    guard = torch.full((P + 2, K), -7.0, dtype=dtype, device=DEV)
    args = [t.to(DEV) for t in (d_out, rows, positions, w)]
    d_rows, d_w = sg.skinny_moe_combine_grad(*args, d_rows=guard[:P])
    token, slot = order[:valid].long() // topk, order[:valid].long() % topk
    g = d_out.to(F64)[token]
    want = g * w.to(F64)[token, slot][:, None]
    # fp32: the product rounds once; bf16: its fp32 product, then the output
    rel = ref.U if dtype is F32 else ref.step_of(dtype) + 2 * ref.U
    assert ((d_rows[:valid].cpu().to(F64) - want).abs() <= rel * want.abs()).all()
    assert (guard[valid:] == -7.0).all(), "rows that no position names are left as they were"
    wantw, mag = torch.zeros((T, topk), dtype=F64), torch.zeros((T, topk), dtype=F64)
    prod = g * rows.to(F64)[:valid]
    wantw[token, slot], mag[token, slot] = prod.sum(1), prod.abs().sum(1)
    # a thread adds its products one after the other, then 6 + 4 additions join the workgroup
    per = -(-K // (256 * (4 if dtype is F32 else 8))) * (4 if dtype is F32 else 8)
    assert ((d_w.cpu().to(F64) - wantw).abs() <= (per + 11) * ref.U * mag).all()
    assert (d_w.cpu()[positions < 0] == 0).all()
    same = args[1].clone()
    a, b = sg.skinny_moe_combine_grad(args[0], same, *args[2:], d_rows=same)
    assert torch.equal(a[:valid], guard[:valid]) and torch.equal(b, d_w), "d_rows may be rows"


def test_gradients_against_differences():
    """Both ways' gradients, chained as a training step chains them, against differences of the
    forward calls: L = <c, combine(gather(x) * s, w)>, all in fp32 on values whose products are
    exact, so that a difference of L is exact too."""
    T, topk, E, K = 6, 3, 5, 16
    ids, _, offsets, order, positions, _ = rows_case(T, topk, E, K, F32)
    g = ref.gen(5)
    small = lambda shape: torch.randint(-4, 5, shape, generator=g).float()  # noqa: E731
    x, c, s, w = small((T, K)), small((T, K)), small((T * topk, K)), small((T, topk))
    pos = positions.to(DEV)

    def loss(x, w):
        rows = sg.skinny_moe_gather(x.to(DEV), pos) * s.to(DEV)
        return float((sg.skinny_moe_combine(rows, pos, w.to(DEV)).cpu() * c).sum())

    rows = sg.skinny_moe_gather(x.to(DEV), pos) * s.to(DEV)
    d_rows, d_w = sg.skinny_moe_combine_grad(c.to(DEV), rows, pos, w.to(DEV))
    d_x = sg.skinny_moe_combine(d_rows * s.to(DEV), pos, None).cpu()
    for t, k in [(0, 0), (2, 7), (5, 15), (3, 4)]:
        e = torch.zeros_like(x)
        e[t, k] = 1
        assert loss(x + e, w) - loss(x - e, w) == 2 * float(d_x[t, k])
    for t in range(T):
        for j in range(topk):
            e = torch.zeros_like(w)
            e[t, j] = 1
            assert loss(x, w + e) - loss(x, w - e) == 2 * float(d_w[t, j])


def test_left_out_pairs_and_values_that_are_not_finite():
    """Left-out pairs add nothing, whatever their weight or the rows behind the last; a NaN row
    reaches its own token alone."""
    T, topk, E, K = 4, 2, 3, 24
    ids = torch.tensor([[0, 7], [1, -1], [9, 9], [2, 0]], dtype=torch.int32)
    offsets, order, positions = ref.table(ids, E)
    rows = torch.randn((T * topk, K), generator=ref.gen(1))
    rows[int(offsets[E]):] = float("nan")
    w = torch.full((T, topk), 0.5)
    w[0, 1], w[1, 1], w[2, 0], w[2, 1] = float("nan"), float("inf"), float("nan"), -float("inf")
    out = sg.skinny_moe_combine(rows.to(DEV), positions.to(DEV), w.to(DEV)).cpu()
    assert torch.isfinite(out).all() and (out[2] == 0).all()
    d_rows, d_w = sg.skinny_moe_combine_grad(torch.ones((T, K), device=DEV), rows.to(DEV),
                                             positions.to(DEV), w.to(DEV))
    assert torch.isfinite(d_w).all() and torch.isfinite(d_rows).all()
    rows[int(positions[3, 0]), 5] = float("nan")
    out = sg.skinny_moe_combine(rows.to(DEV), positions.to(DEV), w.to(DEV)).cpu()
    nan = torch.isnan(out)
    assert nan[3, 5] and int(nan.sum()) == 1


def test_positions_out_of_range_are_left_out():
    T, topk, K = 3, 2, 16
    pos = torch.tensor([[0, 6], [-9, 1], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device=DEV)
    x, rows = torch.randn((T, K), device=DEV), torch.randn((T * topk, K), device=DEV)
    out = torch.full((T * topk, K), -7.0, device=DEV)
    sg.skinny_moe_gather(x, pos, out=out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[1], x[1]) and (out[2:] == -7.0).all()
    y = sg.skinny_moe_combine(rows, pos, None)
    assert torch.equal(y[0], rows[0]) and torch.equal(y[1], rows[1]) and (y[2] == 0).all()
    w = torch.ones((T, topk), device=DEV)
    d_rows, d_w = sg.skinny_moe_combine_grad(x, rows, pos, w, d_rows=out.fill_(-7.0))
    assert torch.equal(d_rows[0], x[0]) and (d_rows[2:] == -7.0).all() and (d_w.flatten()[[1, 2, 4, 5]] == 0).all()
