"""The kernel form that the library plans for a block-scaled FP8 product, and sizes that reach each
form (test infrastructure).  fp8_block_plan is a function inside the library, not of its
interface."""
from __future__ import annotations

import ctypes

import skinny_gemm_projection_amd as sg

TILES = ["256x256", "128x256", "128x128", "64x128", "64x256"]


class Plan(ctypes.Structure):
    """Mirror of sg::Fp8BlockPlan."""
    _fields_ = [("kind", ctypes.c_int), ("mt", ctypes.c_int), ("rt", ctypes.c_int),
                ("waves", ctypes.c_int), ("tile", ctypes.c_int), ("S", ctypes.c_int),
                ("kc", ctypes.c_int), ("workspace", ctypes.c_size_t), ("wide", ctypes.c_bool)]


def plan(M, N, K, f32):
    f = ctypes.CDLL(sg.library_path())._ZN2sg14fp8_block_planEiiib
    f.argtypes, f.restype = [ctypes.c_int] * 3 + [ctypes.c_bool], Plan
    return f(M, N, K, f32)


def form(M, N, K, f32):
    """The name of the kernels that run: a team, or tiles (the K split between workgroups or not;
    "wide": by the bf16 instruction, for fp32 outputs)."""
    p = plan(M, N, K, f32)
    if p.kind == 0:
        return f"team waves {p.waves} rows {16 * p.rt} x {16 * p.mt}"
    return TILES[p.tile] + (" wide" if p.wide else "") + (" split" if p.S > 1 else "")


# (M, N, K, with an fp32 output, form): rows of y of every alignment, last blocks that are not whole
FORMS = [
    (5, 901, 2064, True, "team waves 8 rows 16 x 16"), (1, 4309, 272, True, "team waves 8 rows 32 x 16"),
    (13, 7319, 1008, False, "team waves 8 rows 32 x 16"), (4, 8999, 2528, True, "team waves 4 rows 32 x 16"),
    (23, 241, 720, True, "team waves 8 rows 16 x 32"), (20, 6235, 2192, True, "team waves 8 rows 32 x 32"),
    (18, 9293, 272, False, "team waves 4 rows 32 x 32"), (27, 9001, 688, True, "team waves 4 rows 32 x 32"),
    (135, 35271, 288, False, "256x256"), (2834, 3897, 432, False, "256x256"),
    (5513, 257, 9056, False, "256x256 split"),
    (70, 39315, 272, False, "128x256"), (264, 16711, 816, False, "128x256"),
    (70, 39315, 272, True, "128x256 wide"), (134, 5689, 7312, False, "128x256 split"),
    (73, 11016, 3296, True, "128x256 wide split"), (1452, 1434, 3152, True, "128x256 wide split"),
    (73, 16859, 288, False, "128x128"), (4547, 483, 1056, False, "128x128"),
    (4195, 834, 272, True, "128x128 wide"), (648, 10862, 464, True, "128x128 wide"),
    (78, 5782, 2592, False, "128x128 split"), (242, 2082, 9440, False, "128x128 split"),
    (76, 6435, 2576, True, "128x128 wide split"), (957, 617, 7232, True, "128x128 wide split"),
    (40, 165, 288, False, "64x128"), (40, 165, 288, True, "64x128 wide"),
    (574, 1645, 336, True, "64x128 wide"), (95, 649, 8176, False, "64x128 split"),
    (35, 158, 1248, False, "64x128 split"), (162, 289, 9744, True, "64x128 wide split"),
    (37, 38391, 272, False, "64x256"), (392, 8742, 576, False, "64x256"),
    (73, 16859, 288, True, "64x256 wide"), (35, 11255, 5680, False, "64x256 split"),
    (71, 5955, 1904, True, "64x256 wide split"), (95, 3651, 11200, True, "64x256 wide split")]
