"""Refusals and sizes of the 8-bit integer operators that need no GPU: every call here returns
before anything is launched."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import skinny_gemm_projection_amd as sg
from skinny_gemm_projection_amd import _lib

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake device pointers are only passed on a host without a GPU")
A = 0x10000  # aligned, never dereferenced
NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 4, 5
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def nothing_launches():
    sg.skinny_gemm_reset_counters()
    yield
    if not torch.cuda.is_available():
        assert sum(sg.skinny_gemm_get_counters()) == 0


@no_gpu_only
def test_gemm_refusals():
    c = _lib.load()

    def call(M=4, N=64, K=128, xq=A, xs=A, wq=A, ws=A, r=None, y32=A, y16=None, work=A, nbytes=1 << 40):
        return c.skinny_gemm_int8(M, N, K, xq, xs, wq, ws, r, y32, y16, work, nbytes, None)

    for kw in (dict(M=-1), dict(M=(1 << 20) + 1), dict(N=-1), dict(N=(1 << 20) + 1), dict(K=-16),
               dict(K=131072)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(K=8), dict(K=131), dict(xq=A + 8), dict(wq=A + 4), dict(xs=A + 2), dict(ws=A + 1),
               dict(r=A + 2), dict(y32=A + 4), dict(y16=A + 8)):
        assert call(**kw) == ALIGN, kw
    for kw in (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(y32=None)):
        assert call(**kw) == NULL, kw
    assert call(M=0, xq=None, xs=None, y32=None) == 0 and call(N=0, wq=None, ws=None, y32=None) == 0
    for M, N, K in [(64, 4096, 7168), (40, 1024, 8192), (300, 512, 16384), (16, 128, 65536)]:
        need = sg.skinny_gemm_int8_workspace(M, N, K)
        if need:
            assert call(M=M, N=N, K=K, nbytes=need - 1) == WORKSPACE
            assert call(M=M, N=N, K=K, work=None) == WORKSPACE
            assert call(M=M, N=N, K=K, work=A + 8) == ALIGN


def test_workspace_of_rejected_sizes_is_zero():
    for args in [(-1, 4, 16), (4, -1, 16), (4, 4, -16), (4, 4, 24), (4, 4, 131072), (0, 4, 16),
                 (4, 0, 16), ((1 << 20) + 1, 4, 16), (4, (1 << 20) + 1, 16)]:
        assert sg.skinny_gemm_int8_workspace(*args) == 0, args
    for args in [(-1, 64, 64), (4, 0, 64), (4, 64, 8), (4, 65552, 64), (4, 64, 65552), (4, 24, 64),
                 ((1 << 20) + 1, 64, 64)]:
        assert sg.skinny_mlp_int8_step_workspace(*args) == 0, args
    # codes, scales and the gated product's input fit behind each other (64-bit sizes)
    M, H, F = 1 << 20, 65536, 65536
    assert sg.skinny_mlp_int8_step_workspace(M, H, F) >= M * (H + F)
    assert sg.skinny_mlp_int8_step_workspace(3, 512, 1024) >= 3 * (512 + 1024 * 5 + 8)


@no_gpu_only
def test_norm_refusals():
    c = _lib.load()

    def call(M=4, K=128, x=A, r=A, g=A, eps=1e-6, h=A, y=A, codes=A, scales=A):
        return c.skinny_rmsnorm(M, K, x, r, g, eps, h, y, codes, scales, None)

    for kw in (dict(M=-1), dict(M=(1 << 20) + 1), dict(K=0), dict(K=-8), dict(K=65544), dict(eps=0.0),
               dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(K=12), dict(x=A + 2), dict(r=A + 8), dict(g=A + 4), dict(h=A + 2), dict(y=A + 2),
               dict(codes=A + 8), dict(scales=A + 2)):
        assert call(**kw) == ALIGN, kw
    for kw in (dict(x=None), dict(g=None), dict(y=None, codes=None, scales=None), dict(codes=None),
               dict(scales=None)):
        assert call(**kw) == NULL, kw
    assert call(M=0, x=None, g=None) == 0


@no_gpu_only
def test_quant_refusals():
    c = _lib.load()

    def call(M=4, K=128, x16=A, x32=None, gated=0, codes=A, scales=A):
        return c.skinny_quant_int8(M, K, x16, x32, gated, codes, scales, None)

    for kw in (dict(M=-1), dict(M=(1 << 20) + 1), dict(K=0), dict(K=65544), dict(gated=2), dict(gated=-1)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(K=12), dict(x16=A + 2), dict(x16=None, x32=A + 4), dict(codes=A + 8),
               dict(scales=A + 1)):
        assert call(**kw) == ALIGN, kw
    for kw in (dict(x16=None), dict(x32=A), dict(codes=None), dict(scales=None)):
        assert call(**kw) == NULL, kw
    assert call(M=0, x16=None) == 0


@no_gpu_only
def test_mlp_refusals():
    c = _lib.load()
    base = dict(x=A, r=A, g=A, W_gate_up=A, gate_up_scales=A, W_down=A, down_scales=A, out=A, M=4,
                H=128, F=256, eps=1e-6)

    def call(work=A, nbytes=1 << 40, **kw):
        s = _lib.SgMlpInt8Step(**dict(base, **kw))
        return c.skinny_mlp_int8_step(ctypes.byref(s), work, nbytes, None)

    assert c.skinny_mlp_int8_step(None, A, 1 << 40, None) == NULL
    for kw in (dict(M=-1), dict(M=(1 << 20) + 1), dict(H=0), dict(F=0), dict(H=65552), dict(F=-16),
               dict(eps=0.0), dict(eps=float("nan"))):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(H=24), dict(F=8), dict(x=A + 2), dict(r=A + 2), dict(g=A + 8), dict(W_gate_up=A + 8),
               dict(gate_up_scales=A + 2), dict(W_down=A + 4), dict(down_scales=A + 1), dict(out=A + 2),
               dict(work=A + 8)):
        assert call(**kw) == ALIGN, kw
    for name in ("x", "g", "W_gate_up", "gate_up_scales", "W_down", "down_scales", "out"):
        assert call(**{name: None}) == NULL, name
    need = sg.skinny_mlp_int8_step_workspace(4, 128, 256)
    assert call(nbytes=need - 1) == WORKSPACE and call(work=None) == WORKSPACE
    assert call(M=0, x=None, work=None) == 0


def test_binding_refuses_what_the_library_cannot_see():
    """Types, shapes and host tensors are refused before the call."""
    q, s = torch.zeros((2, 32), dtype=torch.int8), torch.ones(2)
    w, t = torch.zeros((3, 32), dtype=torch.int8), torch.ones(3)
    y = torch.empty((2, 3))
    with pytest.raises((ValueError, RuntimeError)):
        sg.skinny_gemm_int8(q, s, w, t, y_f32=y)  # host tensors
    with pytest.raises(TypeError):
        sg.skinny_gemm_int8(q.float(), s, w, t, y_f32=y)
    with pytest.raises(ValueError):
        sg.skinny_gemm_int8(q[0], s, w, t, y_f32=y)
    x, g = torch.zeros((2, 32), dtype=torch.bfloat16), torch.ones(32, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        sg.skinny_rmsnorm(x.float(), g, 1e-6, y_bf16=x)
    with pytest.raises(ValueError):
        sg.skinny_rmsnorm(x, g, 1e-6, y_bf16=x)
    with pytest.raises(TypeError):
        sg.skinny_quant_int8(x.half(), codes=q, scales=s)
    with pytest.raises(ValueError):
        sg.skinny_quant_int8(x[:, :31], gated=True, codes=q, scales=s)
    with pytest.raises(TypeError):
        sg.skinny_mlp_int8_step(x.half(), g, 1e-6, q, s, w, t, out=x)


def test_binding_refuses_sizes_past_int32():
    """The library's sizes are 32-bit: a longer tensor is refused, not taken modulo 2^32."""
    long, s = torch.empty((2 ** 32 + 8, 0), dtype=torch.int8), torch.ones(8)
    w, x, g = torch.empty((8, 0), dtype=torch.int8), long.bfloat16(), s.bfloat16()
    for call in (lambda: sg.skinny_gemm_int8(long, s, w, s), lambda: sg.skinny_quant_int8(x),
                 lambda: sg.skinny_rmsnorm(x, g, 1e-6),
                 lambda: sg.skinny_mlp_int8_step(x, g, 1e-6, w, s, w, s)):
        with pytest.raises(ValueError, match="past 2"):
            call()


@no_gpu_only
def test_eps_below_the_normal_range_is_refused():
    """Squares below the normal range lose bits: with eps there too the norm would be wrong (a
    row of 2e-23 with eps 2^-149 came out 13 % too large)."""
    c = _lib.load()
    for eps in (2.0 ** -149, 1e-40, 2.0 ** -126 * (1 - 2.0 ** -23)):
        assert c.skinny_rmsnorm(4, 128, A, None, A, eps, None, A, None, None, None) == SHAPE, eps
        step = _lib.SgMlpInt8Step(x=A, g=A, W_gate_up=A, gate_up_scales=A, W_down=A, down_scales=A,
                                  out=A, M=4, H=128, F=256, eps=eps)
        assert c.skinny_mlp_int8_step(ctypes.byref(step), A, 1 << 40, None) == SHAPE, eps
    assert c.skinny_rmsnorm(0, 128, None, None, None, 2.0 ** -126, None, None, None, None, None) == 0


def test_import_and_sizes_without_torchs_gpu_names():
    """Plans and workspace sizes are host code: they work on a torch that has no GPU back end,
    whose torch._C lacks the stream and device functions."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import skinny_gemm_projection_amd as sg\n"
            "assert sg.skinny_gemm_plan(1, 8192, 7168).M == 1\n"
            "assert sg.skinny_mlp_int8_step_workspace(1, 64, 64) > 0\n"
            "print('ok')")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stderr


def test_counters_of_a_caller_with_an_older_header():
    """skinny_gemm_get_counters of a program compiled when there were 11 counters writes 11; the
    sized form, which the header maps the name to now, writes as many as it is given room for."""
    lib = ctypes.CDLL(sg.library_path())
    mark = 0xabadcafe
    buf = (ctypes.c_uint64 * 20)(*[mark] * 20)
    lib.skinny_gemm_get_counters(buf)
    assert list(buf[11:]) == [mark] * 9 and mark not in buf[:11]
    for n in (0, 3, sg.SG_NUM_COUNTERS, 20):
        buf = (ctypes.c_uint64 * 20)(*[mark] * 20)
        lib.skinny_gemm_read_counters(buf, n)
        kept = min(n, sg.SG_NUM_COUNTERS)
        assert mark not in buf[:kept] and set(buf[kept:n]) <= {0} and list(buf[n:]) == [mark] * (20 - n)
    lib.skinny_gemm_read_counters(None, 3)
    lib.skinny_gemm_read_counters(buf, -1)
    assert len(sg.skinny_gemm_get_counters()) == sg.SG_NUM_COUNTERS
    assert sg.skinny_gemm_read_counters(3) == sg.skinny_gemm_get_counters()[:3]


def test_every_planned_form_is_in_the_gpu_tests():
    """The forms that sizes drawn over the whole range plan are those that the GPU tests' sizes
    reach, and each listed size plans the form it is listed for."""
    import random

    from int8_forms import BLOCKS, PRODUCTS, SPLITS, form
    from test_gpu_int8 import GEMM, MLP

    for M, N, K, kind in PRODUCTS + SPLITS:
        assert form(M, N, K) == kind, (M, N, K)
    for M, H, F, kind in BLOCKS:
        assert form(M, 2 * F, H) == kind, (M, H, F)
    products = {form(*s) for s in GEMM} | {s[3] for s in PRODUCTS + SPLITS}
    blocks = {form(M, 2 * F, H) for M, H, F in MLP} | {s[3] for s in BLOCKS}
    rng = random.Random(1)

    def size(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    for _ in range(30000):
        M, N, K = size(1, 9000), size(1, 66000), 16 * size(1, 4096)
        assert form(M, N, K) in products, (M, N, K, form(M, N, K))
        H, F = 16 * size(1, 512), 16 * size(1, 1300)
        kind = form(M, 2 * F, H)
        if kind[0].isdigit() and "split" not in kind:  # the gated product in the tiles' epilogue
            assert kind in blocks, (M, H, F, kind)
