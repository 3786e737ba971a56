"""The kernel form that the library plans for a block-scaled FP8 product by expert (test
infrastructure).  fp8_grouped_plan and fp8_gated_ok are functions inside the library."""
from __future__ import annotations

import ctypes

import skinny_gemm_projection_amd as sg
from fp8_block_forms import TILES, Plan


def grouped_form(rows, E, N, K, f32):
    """The name of the kernel that runs ("wide": by the bf16 instruction, for fp32 outputs)."""
    f = ctypes.CDLL(sg.library_path())._ZN2sg16fp8_grouped_planEiiiib
    f.argtypes, f.restype = [ctypes.c_int] * 4 + [ctypes.c_bool], Plan
    p = f(rows, E, N, K, f32)
    assert p.S == 1 and p.workspace == 0
    if p.kind == 0:
        return f"team waves {p.waves} rows {16 * p.rt} x {16 * p.mt}"
    return TILES[p.tile] + (" wide" if p.wide else "")


def step_forms(rows, E, H, F):
    """The experts' step's two products: "gated" gives the gated product's codes itself."""
    lib = ctypes.CDLL(sg.library_path())
    plan, gated = lib._ZN2sg16fp8_grouped_planEiiiib, lib._ZN2sg12fp8_gated_okERKNS_12Fp8BlockPlanEi
    plan.argtypes, plan.restype = [ctypes.c_int] * 4 + [ctypes.c_bool], Plan
    gated.argtypes, gated.restype = [ctypes.POINTER(Plan), ctypes.c_int], ctypes.c_bool
    up = plan(rows, E, 2 * F, H, False)
    return (grouped_form(rows, E, 2 * F, H, False) + (" gated" if gated(ctypes.byref(up), F) else ""),
            grouped_form(rows, E, H, F, False))
