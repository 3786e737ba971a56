"""Refusals and sizes of the block-scaled FP8 operators and of the calls around routed experts
that need no GPU: every call here returns before anything is launched."""
import ctypes

import pytest
import torch

import skinny_gemm_projection_amd as sg
from skinny_gemm_projection_amd import _lib

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake device pointers are only passed on a host without a GPU")
A = 0x10000  # aligned, never dereferenced
NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 4, 5
BIG = 1 << 40


@pytest.fixture(autouse=True)
def nothing_launches():
    sg.skinny_gemm_reset_counters()
    yield
    if not torch.cuda.is_available():
        assert sum(sg.skinny_gemm_get_counters()) == 0


def refused(call, shape=(), align=(), null=()):
    for kw in shape:
        assert call(**kw) == SHAPE, kw
    for kw in align:
        assert call(**kw) == ALIGN, kw
    for kw in null:
        assert call(**kw) == NULL, kw


@no_gpu_only
def test_quant_refusals():
    c = _lib.load()

    def call(M=4, K=128, x16=A, x32=None, gated=0, codes=A, scales=A):
        return c.skinny_quant_fp8(M, K, x16, x32, gated, codes, scales, None)

    refused(call, (dict(M=-1), dict(M=(1 << 20) + 1), dict(K=0), dict(K=65544), dict(gated=2), dict(gated=-1)),
            (dict(K=12), dict(x16=A + 8), dict(x16=None, x32=A + 4), dict(codes=A + 4), dict(scales=A + 2)),
            (dict(x16=None), dict(x32=A), dict(codes=None), dict(scales=None)))
    assert call(M=0, x16=None) == 0


@no_gpu_only
def test_gemm_refusals():
    c = _lib.load()

    def call(M=4, N=64, K=128, xq=A, xs=A, wq=A, ws=A, r=None, y32=A, y16=None, work=A, nbytes=BIG):
        return c.skinny_gemm_fp8_block(M, N, K, xq, xs, wq, ws, r, y32, y16, work, nbytes, None)

    refused(call, (dict(M=-1), dict(M=(1 << 20) + 1), dict(N=-1), dict(N=(1 << 20) + 1), dict(K=-16),
                   dict(K=65552)),
            (dict(K=8), dict(K=131), dict(xq=A + 8), dict(wq=A + 4), dict(xs=A + 2), dict(ws=A + 1),
             dict(r=A + 2), dict(y32=A + 4), dict(y16=A + 8)),
            (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(y32=None)))
    assert call(M=0, xq=None, xs=None, y32=None) == 0 and call(N=0, wq=None, ws=None) == 0
    for M, N, K in [(300, 512, 16384), (100, 1024, 8192), (65, 128, 65536)]:
        for f32 in (False, True):
            need = sg.skinny_gemm_fp8_block_workspace(M, N, K, f32)
            out = dict(y32=A) if f32 else dict(y32=None, y16=A)
            if need:
                assert call(M=M, N=N, K=K, nbytes=need - 1, **out) == WORKSPACE
                assert call(M=M, N=N, K=K, work=None, **out) == WORKSPACE
                assert call(M=M, N=N, K=K, work=A + 8, **out) == ALIGN


@no_gpu_only
def test_sort_refusals():
    c = _lib.load()

    def call(T=4, topk=2, E=8, ids=A, offsets=A, order=A, positions=A, work=A, nbytes=BIG):
        return c.skinny_moe_sort(T, topk, E, ids, offsets, order, positions, work, nbytes, None)

    refused(call, (dict(T=-1), dict(topk=0), dict(topk=33), dict(E=0), dict(E=4097), dict(T=1 << 20, topk=5),
                   dict(T=(1 << 22) + 1, topk=1), dict(T=2 ** 31 - 1, topk=32)),
            (dict(ids=A + 2), dict(offsets=A + 1), dict(order=A + 2), dict(positions=A + 3)),
            (dict(ids=None), dict(offsets=None), dict(positions=None)))
    need = sg.skinny_moe_sort_workspace(10000, 8, 384)
    assert need > 0 and sg.skinny_moe_sort_workspace(512, 8, 384) == 0
    big = dict(T=10000, topk=8, E=384)
    assert call(**big, nbytes=need - 1) == WORKSPACE and call(**big, work=None) == WORKSPACE
    assert call(**big, work=A + 4) == ALIGN


@no_gpu_only
def test_row_refusals():
    c = _lib.load()

    def gather(T=4, topk=2, K=64, x=A, f32=0, positions=A, rows=A):
        return c.skinny_moe_gather(T, topk, K, x, f32, positions, rows, None)

    def combine(T=4, topk=2, K=64, rows=A, f32=0, positions=A, weights=A, r=A, out=A):
        return c.skinny_moe_combine(T, topk, K, rows, f32, positions, weights, r, out, None)

    def grad(T=4, topk=2, K=64, d_out=A, rows=A, f32=0, positions=A, weights=A, d_rows=A, d_w=A):
        return c.skinny_moe_combine_grad(T, topk, K, d_out, rows, f32, positions, weights, d_rows, d_w, None)

    sizes = (dict(T=-1), dict(topk=0), dict(topk=33), dict(K=0), dict(K=65544), dict(f32=2), dict(f32=-1),
             dict(T=1 << 20, topk=8))
    refused(gather, sizes, (dict(K=12), dict(x=A + 8), dict(rows=A + 4), dict(positions=A + 2)),
            (dict(x=None), dict(positions=None), dict(rows=None)))
    refused(combine, sizes, (dict(K=12), dict(rows=A + 8), dict(r=A + 8), dict(out=A + 2), dict(positions=A + 2),
                             dict(weights=A + 1)), (dict(rows=None), dict(positions=None), dict(out=None)))
    refused(grad, sizes, (dict(K=12), dict(d_out=A + 8), dict(rows=A + 8), dict(d_rows=A + 2),
                          dict(positions=A + 2), dict(weights=A + 1), dict(d_w=A + 2)),
            (dict(d_out=None), dict(rows=None), dict(positions=None), dict(weights=None), dict(d_rows=None),
             dict(d_w=None)))
    assert gather(T=0, x=None) == 0 and combine(T=0, rows=None) == 0 and grad(T=0, rows=None) == 0


@no_gpu_only
def test_grouped_refusals():
    c = _lib.load()

    def call(rows=8, X=8, E=4, N=64, K=128, xq=A, xs=A, wq=A, ws=A, offsets=A, pairs=None, topk=1, y32=A,
             y16=None):
        return c.grouped_skinny_gemm_fp8(rows, X, E, N, K, xq, xs, wq, ws, offsets, pairs, topk, y32, y16, None)

    refused(call, (dict(rows=-1), dict(rows=(1 << 22) + 1), dict(X=-1), dict(X=7), dict(E=0), dict(E=4097),
                   dict(N=-1), dict(N=(1 << 20) + 1), dict(K=-16), dict(K=65552), dict(topk=0), dict(topk=33),
                   dict(pairs=A, X=1 << 20, K=2048), dict(pairs=A, X=(1 << 22) + 1)),
            (dict(K=24), dict(xq=A + 8), dict(wq=A + 4), dict(xs=A + 2), dict(ws=A + 1), dict(offsets=A + 2),
             dict(pairs=A + 1), dict(y32=A + 4), dict(y16=A + 8)),
            (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(offsets=None), dict(y32=None)))
    assert call(rows=0, X=0, xq=None, xs=None) == 0 and call(N=0, wq=None, ws=None) == 0


@no_gpu_only
def test_step_refusals():
    c = _lib.load()
    base = dict(x=A, topk_ids=A, topk_weights=A, W_gate_up=A, gate_up_scales=A, W_down=A, down_scales=A, r=A,
                out=A, T=4, topk=2, E=8, H=128, F=256)

    def call(work=A, nbytes=BIG, **kw):
        s = _lib.SgMoeFp8Step(**dict(base, **kw))
        return c.skinny_moe_fp8_step(ctypes.byref(s), work, nbytes, None)

    assert c.skinny_moe_fp8_step(None, A, BIG, None) == NULL
    refused(call, (dict(T=-1), dict(topk=0), dict(topk=33), dict(E=0), dict(E=4097), dict(H=0), dict(F=0),
                   dict(H=65552), dict(F=-16), dict(T=1 << 20, topk=8), dict(T=1 << 20, topk=1, H=2048)),
            (dict(H=24), dict(F=8), dict(x=A + 2), dict(r=A + 2), dict(out=A + 8), dict(W_gate_up=A + 8),
             dict(gate_up_scales=A + 2), dict(W_down=A + 4), dict(down_scales=A + 1), dict(topk_ids=A + 2),
             dict(topk_weights=A + 2), dict(work=A + 8)),
            [{n: None} for n in ("x", "topk_ids", "topk_weights", "W_gate_up", "gate_up_scales", "W_down",
                                 "down_scales", "out")])
    need = sg.skinny_moe_fp8_step_workspace(4, 2, 8, 128, 256)
    assert call(nbytes=need - 1) == WORKSPACE and call(work=None) == WORKSPACE
    assert call(T=0, x=None, work=None, nbytes=0) == 0


def test_workspace_sizes():
    for args in [(-1, 4, 16), (4, -1, 16), (4, 4, -16), (4, 4, 24), (4, 4, 65552), (0, 4, 16), (4, 0, 16),
                 ((1 << 20) + 1, 4, 16), (4, (1 << 20) + 1, 16)]:
        assert sg.skinny_gemm_fp8_block_workspace(*args, True) == 0, args
    for args in [(-1, 8, 8, 64, 64), (4, 0, 8, 64, 64), (4, 8, 0, 64, 64), (4, 8, 8, 8, 64), (4, 8, 8, 64, 24),
                 (4, 8, 8, 64, 65552), (1 << 20, 5, 8, 64, 64), (1 << 20, 1, 8, 2048, 64)]:
        assert sg.skinny_moe_fp8_step_workspace(*args) == 0, args
    # the expert outputs alone (64-bit sizes)
    T, topk, H, F = 1 << 17, 32, 16368, 65536
    assert sg.skinny_moe_fp8_step_workspace(T, topk, 8, H, F) >= T * topk * (2 * H + F)
    for args in [(-1, 8, 8), (4, 0, 8), (4, 33, 8), (4, 8, 0), (4, 8, 4097), (1 << 20, 8, 8)]:
        assert sg.skinny_moe_sort_workspace(*args) == 0, args


def test_binding_refuses_what_the_library_cannot_see():
    """Types, shapes and host tensors, without a GPU: nothing reaches the library."""
    u8, bf = torch.zeros((8, 64), dtype=torch.uint8), torch.zeros((8, 64), dtype=torch.bfloat16)
    ids, w = torch.zeros((8, 2), dtype=torch.int32), torch.zeros((8, 2))
    long = torch.empty((2 ** 32 + 8, 0), dtype=torch.uint8)
    calls = [lambda: sg.skinny_quant_fp8(bf.half()), lambda: sg.skinny_quant_fp8(None),
             lambda: sg.skinny_quant_fp8(bf), lambda: sg.skinny_quant_fp8(bf[0]),
             lambda: sg.skinny_gemm_fp8_block(u8.to(torch.int8), w, u8, w),
             lambda: sg.skinny_gemm_fp8_block(u8, w, u8, w), lambda: sg.skinny_gemm_fp8_block(long, w, u8, w),
             lambda: sg.skinny_moe_sort(ids.long(), 4), lambda: sg.skinny_moe_sort(ids, 4),
             lambda: sg.skinny_moe_gather(bf, ids.long()), lambda: sg.skinny_moe_gather(bf, ids),
             lambda: sg.skinny_moe_combine(bf, ids, w), lambda: sg.skinny_moe_combine(bf, None, w),
             lambda: sg.skinny_moe_combine_grad(bf, bf, ids, w),
             lambda: sg.grouped_skinny_gemm_fp8(u8, w, u8[None], w, ids),
             lambda: sg.skinny_moe_fp8_step(bf, ids, w, u8[None], w, u8[None], w),
             lambda: sg.skinny_moe_fp8_step(bf.float(), ids, w, u8[None], w, u8[None], w)]
    for call in calls:
        with pytest.raises((TypeError, ValueError)):
            call()


def test_every_planned_form_is_in_the_gpu_tests():
    """The forms that sizes drawn over the whole range plan are those that the GPU tests' sizes
    reach, and each listed size plans the form it is listed for."""
    import random

    from fp8_block_forms import FORMS, form

    for M, N, K, f32, kind in FORMS:
        assert form(M, N, K, f32) == kind, (M, N, K, f32)
    reached = {f[4] for f in FORMS}
    rng = random.Random(1)

    def size(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    for _ in range(20000):
        M, N, K = size(1, 9000), size(1, 131000), 16 * size(1, 4096)
        for f32 in (True, False):
            assert form(M, N, K, f32) in reached, (M, N, K, f32, form(M, N, K, f32))
