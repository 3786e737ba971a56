"""The kernel form that the library plans for an int8 product, and sizes that reach each form
(test infrastructure).  int8_plan is a function inside the library, not of its interface."""
from __future__ import annotations

import ctypes

import skinny_gemm_projection_amd as sg

TILES = ["256x256", "128x256", "128x128", "64x128", "64x64"]


class Plan(ctypes.Structure):
    """Mirror of sg::Int8Plan."""
    _fields_ = [("kind", ctypes.c_int), ("waves", ctypes.c_int), ("rt", ctypes.c_int),
                ("slots", ctypes.c_int), ("tile", ctypes.c_int), ("S", ctypes.c_int),
                ("kc", ctypes.c_int), ("workspace", ctypes.c_size_t), ("cols", ctypes.c_int),
                ("rest", ctypes.c_int)]


def plan(M, N, K):
    f = ctypes.CDLL(sg.library_path())._ZN2sg9int8_planEiii
    f.argtypes, f.restype = [ctypes.c_int] * 3, Plan
    return f(M, N, K)


def form(M, N, K):
    """The name of the kernels that run: team or wide kernel, or tiles (the K split between
    workgroups or not; "+": the tiles of the second launch)."""
    p = plan(M, N, K)
    if p.kind == 0:
        waves = 8 if p.rt == 2 else p.waves  # two row tiles come with 8 waves only
        return f"team waves {waves} rows {16 * p.rt} x {16 * -(-M // 16)} slots {p.slots}"
    if p.kind == 1:
        return "wide"
    if p.cols:
        return f"{TILES[p.tile]} + {TILES[p.rest]}"
    return TILES[p.tile] + (" split" if p.S > 1 else "")


# products (M, N, K), with rows of y that are and are not 4-element aligned
PRODUCTS = [(513, 28853, 736, "256x256 + 128x256"), (513, 28852, 736, "256x256 + 128x256"),
            (516, 28161, 480, "256x256 + 128x128"), (646, 23891, 448, "256x256 + 64x128"),
            (646, 23892, 448, "256x256 + 64x128"), (646, 22006, 400, "256x256 + 64x64"),
            (646, 22001, 400, "256x256 + 64x64")]
# products whose K is split between workgroups: they need a workspace
SPLITS = [(61, 4096, 7168, "64x64 split"), (70, 16, 1696, "64x64 split"),
          (65, 1622, 4256, "64x128 split"), (2079, 65, 2720, "64x128 split"),
          (2934, 17, 3888, "128x128 split"), (129, 5596, 6384, "128x256 split"),
          (130, 16587, 5680, "256x256 split")]
# gated MLP blocks (M, H, F): the form of the gate and up product
BLOCKS = [(514, 752, 14400, "256x256 + 128x256"), (562, 464, 13568, "256x256 + 128x128"),
          (672, 448, 11776, "256x256 + 64x128"), (667, 400, 11136, "256x256 + 64x64")]
