"""Python binding of libskinny_gemm.so: the batch-1..64 decode projection
y = x W^T (+ fused residual) and its routed-expert variant on MI355X.

Each function has the name of the C entry point it calls (include/
skinny_gemm.h) and only marshals arguments: torch tensors become device
pointers, the current torch stream becomes the hipStream_t, and a missing
workspace is allocated with torch (PyTorch provides memory and streams; every
step of the computation runs in the library's HIP kernels).  A non-SG_OK
status raises SkinnyGemmError.  There is no fallback: if the library is not
built, importing it raises.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import (KERNEL_NAMES, SG_KERNEL_GEMV, SG_KERNEL_GROUPED, SG_KERNEL_MOE_TABLE,
                   SG_KERNEL_FP8, SG_KERNEL_MXFP4, SG_KERNEL_NONE, SG_KERNEL_PREFETCH, SG_KERNEL_REDUCE,
                   SG_KERNEL_ROUTER_TOPK,
                   SG_KERNEL_SPLITK_MFMA, SG_KERNEL_SPLITK_VALU, SG_NOALLOC_MAX_WORKSPACE,
                   SG_KERNEL_INT8, SG_KERNEL_QUANT_INT8, SG_KERNEL_RMSNORM,
                   SG_KERNEL_FP8_BLOCK, SG_KERNEL_MOE_ROWS, SG_KERNEL_MOE_SORT, SG_KERNEL_QUANT_FP8,
                   SG_NUM_COUNTERS, SgMlpInt8Step, SgMoeFp8Step, SgMoeStep,
                   SgPlan, SkinnyGemmError)

__all__ = [
    "skinny_gemm_plan", "skinny_gemm_plan_force", "skinny_gemm", "skinny_gemm_residual",
    "skinny_gemm_noalloc", "SG_NOALLOC_MAX_WORKSPACE", "grouped_skinny_gemm_workspace",
    "grouped_skinny_gemm", "skinny_gemm_prefetch", "skinny_gemm_read_probe",
    "skinny_gemm_router_topk", "router_topk", "skinny_moe_step_workspace", "skinny_moe_step",
    "concat_router_shared", "MOE_STEP_MODES", "skinny_gemm_mxfp4", "SG_KERNEL_MXFP4",
    "skinny_gemm_fp8", "SG_KERNEL_FP8", "skinny_gemm_fp8_workspace", "skinny_gemm_mxfp4_workspace",
    "skinny_rmsnorm", "skinny_quant_int8", "skinny_gemm_int8", "skinny_gemm_int8_workspace",
    "skinny_mlp_int8_step", "skinny_mlp_int8_step_workspace",
    "SG_KERNEL_INT8", "SG_KERNEL_RMSNORM", "SG_KERNEL_QUANT_INT8",
    "skinny_quant_fp8", "skinny_gemm_fp8_block", "skinny_gemm_fp8_block_workspace",
    "skinny_moe_sort", "skinny_moe_sort_workspace", "skinny_moe_gather", "skinny_moe_combine",
    "skinny_moe_combine_grad", "grouped_skinny_gemm_fp8", "skinny_moe_fp8_step",
    "skinny_moe_fp8_step_workspace",
    "SG_KERNEL_FP8_BLOCK", "SG_KERNEL_QUANT_FP8", "SG_KERNEL_MOE_SORT", "SG_KERNEL_MOE_ROWS",
    "skinny_gemm_status_str", "skinny_gemm_read_counters", "skinny_gemm_get_counters",
    "skinny_gemm_reset_counters",
    "SgPlan", "SkinnyGemmError", "KERNEL_NAMES", "SG_KERNEL_NONE", "SG_KERNEL_GEMV",
    "SG_KERNEL_SPLITK_VALU", "SG_KERNEL_SPLITK_MFMA", "SG_KERNEL_REDUCE", "SG_KERNEL_MOE_TABLE",
    "SG_KERNEL_GROUPED", "SG_KERNEL_PREFETCH", "SG_KERNEL_ROUTER_TOPK", "SG_NUM_COUNTERS",
    "library_path",
]


def library_path() -> str:
    return _lib.LIB_PATH


def _c():
    return _lib.load()


def _ptr(t, dtype, name, device=None):
    """Device pointer of a contiguous tensor of the expected dtype (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr() or None


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _shape(t, shape, name):
    """The C ABI cannot see buffer sizes: refuse tensors whose shape disagrees with the plan."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} does not match the plan's {tuple(shape)}")


def _at_least(t, count, name):
    if t is not None and t.numel() < count:
        raise ValueError(f"{name}: needs at least {count} elements, has {t.numel()}")


def _workspace(nbytes: int, workspace, device):
    if nbytes == 0:
        return workspace, (workspace.numel() if workspace is not None else 0)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise TypeError("workspace: expected a device tensor")
    return workspace, workspace.numel() * workspace.element_size()


def skinny_gemm_plan(M: int, N: int, K: int) -> SgPlan:
    """plan(M, N, K): kernel, split factor and workspace for y[M,N] = x[M,K] W[N,K]^T."""
    plan = SgPlan()
    _lib.check(_c().skinny_gemm_plan(M, N, K, ctypes.byref(plan)))
    return plan


def skinny_gemm_plan_force(M: int, N: int, K: int, kernel: int, split_k: int = 0,
                           two_pass: int = -1, tile_n: int = 0) -> SgPlan:
    """plan with the kernel (SG_KERNEL_*), split factor, reduction mode
    (0 in-kernel, 1 second pass, -1 library's choice) and, on the matrix
    cores, row tiling (16 team kernel, 128 or 256 chunk kernel, 0 library's
    choice) chosen by the caller."""
    plan = SgPlan()
    _lib.check(_c().skinny_gemm_plan_force(M, N, K, kernel, split_k, two_pass, tile_n,
                                           ctypes.byref(plan)))
    return plan


def skinny_gemm(plan: SgPlan, x: torch.Tensor, W: torch.Tensor, y_f32=None, y_bf16=None,
                workspace=None, stream=None):
    """y = x W^T into y_f32 (float32 [M,N]) and/or y_bf16 (bfloat16 [M,N])."""
    dev = x.device
    M, N, K = plan.M, plan.N, plan.K
    _shape(x, (M, K), "x"), _shape(W, (N, K), "W")
    _shape(y_f32, (M, N), "y_f32"), _shape(y_bf16, (M, N), "y_bf16")
    ws, ws_bytes = _workspace(plan.workspace_bytes, workspace, dev)
    st = _c().skinny_gemm(ctypes.byref(plan), _ptr(x, torch.bfloat16, "x", dev),
                          _ptr(W, torch.bfloat16, "W", dev),
                          _ptr(y_f32, torch.float32, "y_f32", dev),
                          _ptr(y_bf16, torch.bfloat16, "y_bf16", dev),
                          _ptr(ws, torch.uint8, "workspace", dev) if ws is not None else None,
                          ws_bytes, _stream(stream))
    _lib.check(st)
    return ws


def skinny_gemm_noalloc(plan: SgPlan, x: torch.Tensor, W: torch.Tensor, y_f32=None,
                        y_bf16=None, stream=None):
    """skinny_gemm without a workspace: split-K partials go to the library's own
    per-GPU scratch array (calls overlapping on one GPU race on it)."""
    dev = x.device
    M, N, K = plan.M, plan.N, plan.K
    _shape(x, (M, K), "x"), _shape(W, (N, K), "W")
    _shape(y_f32, (M, N), "y_f32"), _shape(y_bf16, (M, N), "y_bf16")
    st = _c().skinny_gemm_noalloc(ctypes.byref(plan), _ptr(x, torch.bfloat16, "x", dev),
                                  _ptr(W, torch.bfloat16, "W", dev),
                                  _ptr(y_f32, torch.float32, "y_f32", dev),
                                  _ptr(y_bf16, torch.bfloat16, "y_bf16", dev), _stream(stream))
    _lib.check(st)


def skinny_gemm_residual(plan: SgPlan, x: torch.Tensor, W: torch.Tensor, r: torch.Tensor,
                         out_bf16=None, out_f32=None, workspace=None, stream=None):
    """out = r + x W^T (one rounding) into out_bf16 (may be r itself) and/or out_f32."""
    dev = x.device
    M, N, K = plan.M, plan.N, plan.K
    _shape(x, (M, K), "x"), _shape(W, (N, K), "W"), _shape(r, (M, N), "r")
    _shape(out_f32, (M, N), "out_f32"), _shape(out_bf16, (M, N), "out_bf16")
    ws, ws_bytes = _workspace(plan.workspace_bytes, workspace, dev)
    st = _c().skinny_gemm_residual(ctypes.byref(plan), _ptr(x, torch.bfloat16, "x", dev),
                                   _ptr(W, torch.bfloat16, "W", dev),
                                   _ptr(r, torch.bfloat16, "r", dev),
                                   _ptr(out_bf16, torch.bfloat16, "out_bf16", dev),
                                   _ptr(out_f32, torch.float32, "out_f32", dev),
                                   _ptr(ws, torch.uint8, "workspace", dev) if ws is not None else None,
                                   ws_bytes, _stream(stream))
    _lib.check(st)
    return ws


def grouped_skinny_gemm_workspace(T: int, E: int, topk: int, N: int, K: int) -> int:
    return int(_c().grouped_skinny_gemm_workspace(T, E, topk, N, K))


def grouped_skinny_gemm(x: torch.Tensor, W: torch.Tensor, topk_ids: torch.Tensor, out: torch.Tensor,
                        expert_offsets=None, sorted_pairs=None, invalid_count=None,
                        workspace=None, stream=None):
    """out[t,j,:] = W[topk_ids[t,j]] @ x[t] for x [T,K], W [E,N,K], topk_ids [T,topk] int32."""
    dev = x.device
    T, K = x.shape
    E, N, K2 = W.shape
    if K2 != K or topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, W {tuple(W.shape)}, "
                         f"topk_ids {tuple(topk_ids.shape)}")
    topk = topk_ids.shape[1]
    _shape(out, (T, topk, N), "out")
    _at_least(expert_offsets, E + 1, "expert_offsets")
    _at_least(sorted_pairs, T * topk, "sorted_pairs")
    _at_least(invalid_count, 1, "invalid_count")
    need = grouped_skinny_gemm_workspace(T, E, topk, N, K)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = _c().grouped_skinny_gemm(
        _ptr(x, torch.bfloat16, "x", dev), T, _ptr(W, torch.bfloat16, "W", dev), E, N, K,
        _ptr(topk_ids, torch.int32, "topk_ids", dev), topk, _ptr(out, torch.float32, "out", dev),
        _ptr(expert_offsets, torch.int32, "expert_offsets", dev),
        _ptr(sorted_pairs, torch.int32, "sorted_pairs", dev),
        _ptr(invalid_count, torch.int32, "invalid_count", dev),
        _ptr(workspace, torch.uint8, "workspace", dev), ws_bytes, _stream(stream))
    _lib.check(st)
    return workspace


def skinny_gemm_prefetch(W: torch.Tensor, nbytes: int | None = None, stream=None) -> None:
    """Warm [W, W + nbytes) into the GPU caches on `stream` (static weights only)."""
    if not W.is_cuda or not W.is_contiguous():
        raise ValueError("W: must be a contiguous device tensor")
    total = W.numel() * W.element_size()
    nbytes = total if nbytes is None else int(nbytes)
    if nbytes > total:
        raise ValueError("nbytes exceeds the tensor")
    _lib.check(_c().skinny_gemm_prefetch(W.data_ptr() or None, nbytes, _stream(stream)))


def skinny_gemm_read_probe(W: torch.Tensor, rows_per_iter: int, grid: int, stream=None) -> None:
    """Read W ([rows, row_bytes] contiguous device tensor) with the M <= 2 projection
    kernel's load shape and no arithmetic (a measurement of the read rate alone)."""
    if not W.is_cuda or not W.is_contiguous() or W.dim() != 2:
        raise ValueError("W: must be a contiguous 2-D device tensor")
    rows, row_bytes = W.shape[0], W.shape[1] * W.element_size()
    _lib.check(_c().skinny_gemm_read_probe(W.data_ptr() or None, rows, row_bytes, rows_per_iter,
                                           grid, _stream(stream)))


def skinny_gemm_router_topk(scores: torch.Tensor, k: int, topk_ids=None, topk_scores=None,
                            stream=None):
    """topk_ids (int32 [T,k]) and, if given, topk_scores (float32 [T,k]) from router
    scores (float32 [T,E]): larger score first, ties to the lower expert id, NaN as -inf."""
    if scores.dtype != torch.float32 or scores.dim() != 2 or not scores.is_contiguous():
        raise ValueError("scores: expected a contiguous float32 [T, E] tensor")
    T, E = scores.shape
    dev = scores.device
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    _shape(topk_ids, (T, k), "topk_ids"), _shape(topk_scores, (T, k), "topk_scores")
    st = _c().skinny_gemm_router_topk(
        _ptr(scores, torch.float32, "scores", dev), T, E, k,
        _ptr(topk_ids, torch.int32, "topk_ids", dev),
        _ptr(topk_scores, torch.float32, "topk_scores", dev), _stream(stream))
    _lib.check(st)
    return topk_ids


def router_topk(x: torch.Tensor, W_router: torch.Tensor, k: int, stream=None):
    """Expert selection for MoE decode: router scores y = x W_router^T (fp32, the
    planned skinny projection), then their top-k.  Returns (topk_ids [T,k] int32,
    topk_scores [T,k] float32, scores [T,E] float32)."""
    T, E = x.shape[0], W_router.shape[0]
    plan = skinny_gemm_plan(T, E, x.shape[1])
    scores = torch.empty((T, E), dtype=torch.float32, device=x.device)
    skinny_gemm(plan, x, W_router, y_f32=scores, stream=stream)
    top = torch.empty((T, k), dtype=torch.float32, device=x.device)
    ids = skinny_gemm_router_topk(scores, k, topk_scores=top, stream=stream)
    return ids, top, scores


def skinny_moe_step_workspace(T: int, K: int, E: int, topk: int, N: int, N_shared: int) -> int:
    return int(_c().skinny_moe_step_workspace(T, K, E, topk, N, N_shared))


_SIDE = {}  # device -> (side stream, fork event, join event), made once per device


def _side_resources(device):
    res = _SIDE.get(device)
    if res is None:
        with torch.cuda.device(device):
            side = torch.cuda.Stream(device=device)  # default priority
            fork, join = torch.cuda.Event(), torch.cuda.Event()
            cur = torch.cuda.current_stream(device)
            fork.record(cur)  # torch creates the hipEvent_t at its first record
            join.record(cur)
        res = (side, fork, join)
        _SIDE[device] = res
    return res


def skinny_gemm_fp8_workspace(M: int, N: int, K: int) -> int:
    """Workspace bytes skinny_gemm_fp8 needs for an M x N x K projection (0 when none)."""
    return int(_c().skinny_gemm_fp8_workspace(M, N, K))


def skinny_gemm_mxfp4_workspace(M: int, N: int, K: int) -> int:
    """Workspace bytes skinny_gemm_mxfp4 needs for an M x N x K projection (0 when none)."""
    return int(_c().skinny_gemm_mxfp4_workspace(M, N, K))


def skinny_gemm_mxfp4(x: torch.Tensor, W_codes: torch.Tensor, W_scales: torch.Tensor,
                      y_f32=None, y_bf16=None, r=None, workspace=None, stream=None):
    """y = x W^T for MXFP4 weights: W_codes uint8 [N, K/2] (two e2m1 codes a byte, low
    nibble first), W_scales uint8 [N, K/32] (e8m0 block scales); x bf16 [M, K], M <= 64.
    Writes y_f32 and/or y_bf16 [M, N]; with r (bf16 [M, N]) the fused residual
    y = r + x W^T.  Allocates y_f32 when no output is given, and the workspace (when
    the chunk kernel splits K) when none is given; returns the outputs."""
    dev = x.device
    M, K = x.shape
    N = W_codes.shape[0]
    if W_codes.shape != (N, K // 2) or W_scales.shape != (N, K // 32) or K % 32:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, W_codes {tuple(W_codes.shape)}, "
                         f"W_scales {tuple(W_scales.shape)}")
    if y_f32 is None and y_bf16 is None:
        y_f32 = torch.empty((M, N), dtype=torch.float32, device=dev)
    for t, name in ((y_f32, "y_f32"), (y_bf16, "y_bf16"), (r, "r")):
        _shape(t, (M, N), name)
    ws, ws_bytes = _workspace(skinny_gemm_mxfp4_workspace(M, N, K), workspace, dev)
    st = _c().skinny_gemm_mxfp4(
        M, N, K, _ptr(x, torch.bfloat16, "x", dev), _ptr(W_codes, torch.uint8, "W_codes", dev),
        _ptr(W_scales, torch.uint8, "W_scales", dev), _ptr(r, torch.bfloat16, "r", dev),
        _ptr(y_f32, torch.float32, "y_f32", dev), _ptr(y_bf16, torch.bfloat16, "y_bf16", dev),
        _ptr(ws, torch.uint8, "workspace", dev) if ws is not None else None, ws_bytes,
        _stream(stream))
    _lib.check(st)
    return y_f32, y_bf16


def skinny_gemm_fp8(x: torch.Tensor, W_codes: torch.Tensor, W_scales: torch.Tensor,
                    y_f32=None, y_bf16=None, r=None, workspace=None, stream=None):
    """y = x W^T for FP8 weights: W_codes uint8 [N, K] (OCP E4M3 codes), W_scales float32
    [ceil(N/128), ceil(K/128)] (one scale per 128 x 128 block); x bf16 [M, K], M <= 64.
    Writes y_f32 and/or y_bf16 [M, N]; with r (bf16 [M, N]) the fused residual
    y = r + x W^T.  Allocates y_f32 when no output is given, and the workspace (when
    the chunk kernel splits K) when none is given; returns the outputs."""
    dev = x.device
    M, K = x.shape
    N = W_codes.shape[0]
    if W_codes.shape != (N, K) or W_scales.shape != (-(-N // 128), -(-K // 128)):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, W_codes {tuple(W_codes.shape)}, "
                         f"W_scales {tuple(W_scales.shape)}")
    if y_f32 is None and y_bf16 is None:
        y_f32 = torch.empty((M, N), dtype=torch.float32, device=dev)
    for t, name in ((y_f32, "y_f32"), (y_bf16, "y_bf16"), (r, "r")):
        _shape(t, (M, N), name)
    ws, ws_bytes = _workspace(skinny_gemm_fp8_workspace(M, N, K), workspace, dev)
    st = _c().skinny_gemm_fp8(
        M, N, K, _ptr(x, torch.bfloat16, "x", dev), _ptr(W_codes, torch.uint8, "W_codes", dev),
        _ptr(W_scales, torch.float32, "W_scales", dev), _ptr(r, torch.bfloat16, "r", dev),
        _ptr(y_f32, torch.float32, "y_f32", dev), _ptr(y_bf16, torch.bfloat16, "y_bf16", dev),
        _ptr(ws, torch.uint8, "workspace", dev) if ws is not None else None, ws_bytes,
        _stream(stream))
    _lib.check(st)
    return y_f32, y_bf16


# ---- 8-bit integer operators: codes with one scale per row (token or channel) ----


def _arg(t, dtype, shape, name, dev):
    """Device pointer of a contiguous tensor of exactly this type, shape and device."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev.index
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:  # not a tensor: _ptr says so
        pass
    _ptr(t, dtype, name, dev)
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows(x, name, dtypes):
    """(rows, columns, device, pointer) of a contiguous 2-D device tensor of one of the types."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(x).__name__}")
    if x.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {x.dtype}")
    try:
        M, K = x.shape
    except ValueError:
        raise ValueError(f"{name}: expected a 2-D tensor, got shape {tuple(x.shape)}") from None
    if M > 0x7fffffff or K > 0x7fffffff:  # the C ABI's sizes are int32 and would wrap around
        raise ValueError(f"{name}: shape {tuple(x.shape)} is past 2^31 - 1")
    if not x.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if not x.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return M, K, x.device, x.data_ptr()


def _as_stream(stream, dev):
    """The torch stream a call runs on: dev's current one by default."""
    if stream is None:
        return torch.cuda.current_stream(dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    return stream


def _new(shape, dtype, dev, stream):
    """A tensor the work on `stream` may use at once: taken from that stream's memory."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(_as_stream(stream, dev)):
        return torch.empty(shape, dtype=dtype, device=dev)


def _ws_arg(workspace, nbytes, dev, stream):
    """(tensor, pointer, bytes) of the given workspace, or of a new one when none is given."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = _new((nbytes,), torch.uint8, dev, stream)
    return workspace, _ptr(workspace, torch.uint8, "workspace", dev), workspace.numel()


# The functions behind torch.cuda.current_stream and current_device, without the Stream object
# and the initialisation check, which cost more host time than all checks of a call (its tensors
# are on the device already, so the runtime is up).  Private names: without them the public ones.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run_on(dev, stream, fn, *args):
    """fn(*args, stream handle) with dev current; the default stream is dev's current one."""
    index = dev.index
    handle = _raw_stream(index) if stream is None else _stream(stream)
    if _raw_device() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st:
        _lib.check(st)


@functools.lru_cache(maxsize=4096)
def _gemm_int8_workspace(M, N, K):
    return _c().skinny_gemm_int8_workspace(M, N, K)


def skinny_rmsnorm(x: torch.Tensor, g: torch.Tensor, eps: float, r=None, h=None, y_bf16=None,
                   codes=None, scales=None, stream=None):
    """Root-mean-square norm with the residual addition and int8 output: s = x (+ r), h = bf16(s),
    y = s * g / sqrt(mean(s^2) + eps).  x, r [M, K], g [K] bf16.  Writes what is given of h and
    y_bf16 (bf16 [M, K], each may be x or r itself) and codes int8 [M, K] with scales float32 [M]
    (y is about codes * scales[:, None]); allocates codes and scales when neither y_bf16 nor codes
    is given, and scales when only codes is.  Returns (h, y_bf16, codes, scales)."""
    bf16 = torch.bfloat16
    M, K, dev, px = _rows(x, "x", (bf16,))
    mk = (M, K)
    if codes is None and (y_bf16 is None or scales is not None):
        codes = _new((M, K), torch.int8, dev, stream)
    if codes is not None and scales is None:
        scales = _new((M,), torch.float32, dev, stream)
    _run_on(dev, stream, _c().skinny_rmsnorm, M, K, px,
            None if r is None else _arg(r, bf16, mk, "r", dev), _arg(g, bf16, (K,), "g", dev), eps,
            None if h is None else _arg(h, bf16, mk, "h", dev),
            None if y_bf16 is None else _arg(y_bf16, bf16, mk, "y_bf16", dev),
            None if codes is None else _arg(codes, torch.int8, mk, "codes", dev),
            None if scales is None else _arg(scales, torch.float32, (M,), "scales", dev))
    return h, y_bf16, codes, scales


def skinny_quant_int8(x: torch.Tensor, gated: bool = False, codes=None, scales=None, stream=None):
    """Codes int8 [M, K] and scales float32 [M] of rows of x (bf16 or float32): of x [M, K]
    itself, or with gated of silu(x[:, :K]) * x[:, K:] for x [M, 2K].  Rows are tokens in front
    of an integer projection, or the channels of a weight matrix.  Returns (codes, scales)."""
    M, K, dev, px = _rows(x, "x", (torch.bfloat16, torch.float32))
    if gated:
        if K % 2:
            raise ValueError(f"x: gated rows hold gate and up halves, got {K} columns")
        K //= 2
    if codes is None:
        codes = _new((M, K), torch.int8, dev, stream)
    if scales is None:
        scales = _new((M,), torch.float32, dev, stream)
    f32 = x.dtype is torch.float32
    _run_on(dev, stream, _c().skinny_quant_int8, M, K, None if f32 else px, px if f32 else None,
            1 if gated else 0, _arg(codes, torch.int8, (M, K), "codes", dev),
            _arg(scales, torch.float32, (M,), "scales", dev))
    return codes, scales


def skinny_gemm_int8_workspace(M: int, N: int, K: int) -> int:
    """Workspace bytes skinny_gemm_int8 needs for an M x N x K product (0 when none)."""
    return int(_c().skinny_gemm_int8_workspace(M, N, K))


def skinny_gemm_int8(x_codes: torch.Tensor, x_scales: torch.Tensor, W_codes: torch.Tensor,
                     W_scales: torch.Tensor, y_f32=None, y_bf16=None, r=None, workspace=None,
                     stream=None):
    """y[m, n] = sum_k x_codes[m, k] W_codes[n, k] * W_scales[n] * x_scales[m] for int8 codes
    x_codes [M, K], W_codes [N, K] and float32 scales [M], [N]; any M up to 2^20.  Writes y_f32
    and/or y_bf16 [M, N]; with r (bf16 [M, N]) the fused residual y = r + product (y_bf16 may
    be r).  Allocates y_f32 when no output is given, and the workspace when one is needed and
    none is given; returns the outputs."""
    i8, f32, bf16 = torch.int8, torch.float32, torch.bfloat16
    M, K, dev, px = _rows(x_codes, "x_codes", (i8,))
    N, _, _, pw = _rows(W_codes, "W_codes", (i8,))
    if W_codes.shape[1] != K or W_codes.get_device() != dev.index:
        _arg(W_codes, i8, (N, K), "W_codes", dev)  # raises
    mn = (M, N)
    if y_f32 is None and y_bf16 is None:
        y_f32 = _new(mn, torch.float32, dev, stream)
    ws, ws_ptr, ws_bytes = _ws_arg(workspace, _gemm_int8_workspace(M, N, K), dev, stream)
    _run_on(dev, stream, _c().skinny_gemm_int8, M, N, K, px,
            _arg(x_scales, f32, (M,), "x_scales", dev), pw,
            _arg(W_scales, f32, (N,), "W_scales", dev),
            None if r is None else _arg(r, bf16, mn, "r", dev),
            None if y_f32 is None else _arg(y_f32, f32, mn, "y_f32", dev),
            None if y_bf16 is None else _arg(y_bf16, bf16, mn, "y_bf16", dev), ws_ptr, ws_bytes)
    return y_f32, y_bf16


def skinny_mlp_int8_step_workspace(M: int, H: int, F: int) -> int:
    """Workspace bytes skinny_mlp_int8_step needs (0 if the sizes are rejected)."""
    return int(_c().skinny_mlp_int8_step_workspace(M, H, F))


def skinny_mlp_int8_step(x: torch.Tensor, g: torch.Tensor, eps: float, W_gate_up: torch.Tensor,
                         gate_up_scales: torch.Tensor, W_down: torch.Tensor,
                         down_scales: torch.Tensor, r=None, out=None, workspace=None, stream=None):
    """A gated MLP block with int8 weights: h = x (+ r), out = h + down(swiglu(gate_up(norm(h)))),
    the norm's output and the gated product quantised a token at a time.  x, r [M, H], g [H] bf16;
    W_gate_up int8 [2F, H] (gate rows, then up rows), W_down int8 [H, F], float32 scales per row.
    out bf16 [M, H] (may be x or r itself; allocated when not given).  Returns out."""
    M, H, dev, px = _rows(x, "x", (torch.bfloat16,))
    F = _rows(W_down, "W_down", (torch.int8,))[1]
    if out is None:
        out = _new((M, H), torch.bfloat16, dev, stream)
    ws, ws_ptr, ws_bytes = _ws_arg(workspace, _c().skinny_mlp_int8_step_workspace(M, H, F), dev,
                                   stream)
    i8, f32, bf16 = torch.int8, torch.float32, torch.bfloat16
    step = SgMlpInt8Step(
        px, None if r is None else _arg(r, bf16, (M, H), "r", dev),
        _arg(g, bf16, (H,), "g", dev), _arg(W_gate_up, i8, (2 * F, H), "W_gate_up", dev),
        _arg(gate_up_scales, f32, (2 * F,), "gate_up_scales", dev),
        _arg(W_down, i8, (H, F), "W_down", dev), _arg(down_scales, f32, (H,), "down_scales", dev),
        _arg(out, bf16, (M, H), "out", dev), M, H, F, eps)
    _run_on(dev, stream, _c().skinny_mlp_int8_step, ctypes.byref(step), ws_ptr, ws_bytes)
    return out


# ---- block-scaled FP8 rows, and tokens sorted by expert and back ----


def _blocks(n):
    return (n + 127) >> 7


def skinny_quant_fp8(x: torch.Tensor, gated: bool = False, codes=None, scales=None, stream=None):
    """e4m3 codes uint8 [M, K] and scales float32 [ceil(K/128), M] of rows of x (bf16 or
    float32): of x [M, K] itself, or with gated of silu(x[:, :K]) * x[:, K:] for x [M, 2K].  Each
    row's block of 128 columns has the least power of two as its scale that brings it to at most
    448.  Returns (codes, scales)."""
    M, K, dev, px = _rows(x, "x", (torch.bfloat16, torch.float32))
    if gated:
        if K % 2:
            raise ValueError(f"x: gated rows hold gate and up halves, got {K} columns")
        K //= 2
    if codes is None:
        codes = _new((M, K), torch.uint8, dev, stream)
    if scales is None:
        scales = _new((_blocks(K), M), torch.float32, dev, stream)
    f32 = x.dtype is torch.float32
    _run_on(dev, stream, _c().skinny_quant_fp8, M, K, None if f32 else px, px if f32 else None,
            1 if gated else 0, _arg(codes, torch.uint8, (M, K), "codes", dev),
            _arg(scales, torch.float32, (_blocks(K), M), "scales", dev))
    return codes, scales


def skinny_gemm_fp8_block_workspace(M: int, N: int, K: int, with_f32: bool) -> int:
    """Workspace bytes skinny_gemm_fp8_block needs for an M x N x K product (0 when none);
    with_f32: whether y_f32 is given."""
    return int(_c().skinny_gemm_fp8_block_workspace(M, N, K, 1 if with_f32 else 0))


@functools.lru_cache(maxsize=4096)
def _fp8_block_workspace(M, N, K, with_f32):
    return _c().skinny_gemm_fp8_block_workspace(M, N, K, with_f32)


def skinny_gemm_fp8_block(x_codes: torch.Tensor, x_scales: torch.Tensor, W_codes: torch.Tensor,
                          W_scales: torch.Tensor, y_f32=None, y_bf16=None, r=None, workspace=None,
                          stream=None):
    """y = x W^T for e4m3 codes on both sides (uint8): x_codes [M, K] with scales float32
    [ceil(K/128), M] (as skinny_quant_fp8 makes them), W_codes [N, K] with scales float32
    [ceil(N/128), ceil(K/128)]; any M up to 2^20.  Writes y_f32 and/or y_bf16 [M, N]; with r (bf16
    [M, N]) the fused residual y = r + product (y_bf16 may be r).  Allocates y_f32 when no output
    is given, and the workspace when one is needed and none is given; returns the outputs.
    (y_bf16 alone, past 32 rows, takes the FP8 matrix instruction: see the header on its sums.)"""
    u8, f32, bf16 = torch.uint8, torch.float32, torch.bfloat16
    M, K, dev, px = _rows(x_codes, "x_codes", (u8,))
    N, _, _, pw = _rows(W_codes, "W_codes", (u8,))
    if W_codes.shape[1] != K or W_codes.get_device() != dev.index:
        _arg(W_codes, u8, (N, K), "W_codes", dev)  # raises
    mn = (M, N)
    if y_f32 is None and y_bf16 is None:
        y_f32 = _new(mn, f32, dev, stream)
    ws, ws_ptr, ws_bytes = _ws_arg(workspace, _fp8_block_workspace(M, N, K, 0 if y_f32 is None else 1),
                                   dev, stream)
    _run_on(dev, stream, _c().skinny_gemm_fp8_block, M, N, K, px,
            _arg(x_scales, f32, (_blocks(K), M), "x_scales", dev), pw,
            _arg(W_scales, f32, (_blocks(N), _blocks(K)), "W_scales", dev),
            None if r is None else _arg(r, bf16, mn, "r", dev),
            None if y_f32 is None else _arg(y_f32, f32, mn, "y_f32", dev),
            None if y_bf16 is None else _arg(y_bf16, bf16, mn, "y_bf16", dev), ws_ptr, ws_bytes)
    return y_f32, y_bf16


def skinny_moe_sort_workspace(T: int, topk: int, E: int) -> int:
    """Workspace bytes skinny_moe_sort needs (0 when none)."""
    return int(_c().skinny_moe_sort_workspace(T, topk, E))


def skinny_moe_sort(topk_ids: torch.Tensor, E: int, expert_offsets=None, sorted_pairs=None,
                    positions=None, workspace=None, stream=None):
    """The pairs p = t * topk + j of topk_ids (int32 [T, topk]) sorted by expert, ascending in p
    inside an expert; ids outside [0, E) are left out.  Returns int32 (expert_offsets [E + 1],
    sorted_pairs [T * topk] with -1 behind the last, positions [T, topk]: a pair's place, -1 if
    left out), each allocated when not given."""
    T, topk, dev, pi = _rows(topk_ids, "topk_ids", (torch.int32,))
    i32 = torch.int32
    if not 0 < E <= 0x7fffffff:
        raise ValueError(f"E: expected a positive number of experts, got {E}")
    if expert_offsets is None:
        expert_offsets = _new((E + 1,), i32, dev, stream)
    if sorted_pairs is None:
        sorted_pairs = _new((T * topk,), i32, dev, stream)
    if positions is None:
        positions = _new((T, topk), i32, dev, stream)
    ws, ws_ptr, ws_bytes = _ws_arg(workspace, _c().skinny_moe_sort_workspace(T, topk, E), dev, stream)
    _run_on(dev, stream, _c().skinny_moe_sort, T, topk, E, pi,
            _arg(expert_offsets, i32, (E + 1,), "expert_offsets", dev),
            _arg(sorted_pairs, i32, (T * topk,), "sorted_pairs", dev),
            _arg(positions, i32, (T, topk), "positions", dev), ws_ptr, ws_bytes)
    return expert_offsets, sorted_pairs, positions


def _table_of(positions):
    T, topk, dev, pp = _rows(positions, "positions", (torch.int32,))
    return T, topk, dev, pp


_ROW_TYPES = (torch.bfloat16, torch.float32)


def skinny_moe_gather(x: torch.Tensor, positions: torch.Tensor, out=None, stream=None):
    """out[positions[t, j]] = x[t]: token rows (bf16 or float32 [T, K]) laid out by expert, [T *
    topk, K].  Rows that no position names are left as they were (zeros in an out allocated
    here).  Its gradient is skinny_moe_combine without weights.  Returns out."""
    T, topk, dev, pp = _table_of(positions)
    n, K, _, px = _rows(x, "x", _ROW_TYPES)
    if n != T or x.get_device() != dev.index:
        _arg(x, x.dtype, (T, K), "x", dev)  # raises
    if out is None:
        out = _new((T * topk, K), x.dtype, dev, stream)
        with torch.cuda.stream(_as_stream(stream, dev)):
            out.zero_()
    _run_on(dev, stream, _c().skinny_moe_gather, T, topk, K, px, 1 if x.dtype is torch.float32 else 0,
            pp, _arg(out, x.dtype, (T * topk, K), "out", dev))
    return out


def skinny_moe_combine(rows: torch.Tensor, positions: torch.Tensor, weights, r=None, out=None,
                       stream=None):
    """out[t] = (r[t] +) sum_j weights[t, j] * rows[positions[t, j]]: expert outputs (bf16 or
    float32 [T * topk, K]) back to their tokens, left-out pairs skipped; weights float32 [T, topk]
    or None (all 1).  r and out [T, K] of the rows' type, out may be r; fp32 sums, one rounding.
    Returns out."""
    T, topk, dev, pp = _table_of(positions)
    n, K, _, pr = _rows(rows, "rows", _ROW_TYPES)
    if n != T * topk or rows.get_device() != dev.index:
        _arg(rows, rows.dtype, (T * topk, K), "rows", dev)  # raises
    if out is None:
        out = _new((T, K), rows.dtype, dev, stream)
    _run_on(dev, stream, _c().skinny_moe_combine, T, topk, K, pr,
            1 if rows.dtype is torch.float32 else 0, pp,
            None if weights is None else _arg(weights, torch.float32, (T, topk), "weights", dev),
            None if r is None else _arg(r, rows.dtype, (T, K), "r", dev),
            _arg(out, rows.dtype, (T, K), "out", dev))
    return out


def skinny_moe_combine_grad(d_out: torch.Tensor, rows: torch.Tensor, positions: torch.Tensor,
                            weights: torch.Tensor, d_rows=None, d_weights=None, stream=None):
    """Gradient of skinny_moe_combine for d_out [T, K]: d_rows[positions[t, j]] = weights[t, j] *
    d_out[t] (bf16 or float32 [T * topk, K] like rows; may be rows itself; rows that no position
    names are left as they were, zeros in a d_rows allocated here) and d_weights[t, j] = <d_out[t],
    rows[positions[t, j]]> (float32 [T, topk], 0 where left out).  Returns (d_rows, d_weights)."""
    T, topk, dev, pp = _table_of(positions)
    n, K, _, pr = _rows(rows, "rows", _ROW_TYPES)
    if n != T * topk or rows.get_device() != dev.index:
        _arg(rows, rows.dtype, (T * topk, K), "rows", dev)  # raises
    if d_rows is None:
        d_rows = _new((T * topk, K), rows.dtype, dev, stream)
        with torch.cuda.stream(_as_stream(stream, dev)):
            d_rows.zero_()
    if d_weights is None:
        d_weights = _new((T, topk), torch.float32, dev, stream)
    _run_on(dev, stream, _c().skinny_moe_combine_grad, T, topk, K,
            _arg(d_out, rows.dtype, (T, K), "d_out", dev), pr,
            1 if rows.dtype is torch.float32 else 0, pp,
            _arg(weights, torch.float32, (T, topk), "weights", dev),
            _arg(d_rows, rows.dtype, (T * topk, K), "d_rows", dev),
            _arg(d_weights, torch.float32, (T, topk), "d_weights", dev))
    return d_rows, d_weights


def _experts(W, name, dev):
    """(E, N, K, pointer) of contiguous uint8 expert weights on dev."""
    _ptr(W, torch.uint8, name, dev)
    if W.dim() != 3 or max(W.shape) > 0x7fffffff:
        raise ValueError(f"{name}: expected [E, N, K], got shape {tuple(W.shape)}")
    return (*W.shape, W.data_ptr())


def grouped_skinny_gemm_fp8(x_codes: torch.Tensor, x_scales: torch.Tensor, W_codes: torch.Tensor,
                            W_scales: torch.Tensor, expert_offsets: torch.Tensor, sorted_pairs=None,
                            topk: int = 1, y_f32=None, y_bf16=None, stream=None):
    """y[i] = x_i W[e]^T for the rows expert_offsets[e] <= i < expert_offsets[e + 1] of every
    expert e: W_codes uint8 [E, N, K] with scales float32 [E, ceil(N/128), ceil(K/128)].  x_i is
    row i of x_codes [rows, K], or with sorted_pairs (int32 [rows], skinny_moe_sort's) row
    sorted_pairs[i] // topk of x_codes [T, K]; x_scales [ceil(K/128), rows of x_codes].  Writes
    y_f32 and/or y_bf16 [rows, N]; rows behind the last segment are left as they were (zeros in a
    y_f32 allocated here, which happens when no output is given).  Returns the outputs."""
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    if not 0 < topk <= 0x7fffffff:  # the C ABI's sizes are int32 and would wrap around
        raise ValueError(f"topk: expected a positive number of slots a token, got {topk}")
    X, K, dev, px = _rows(x_codes, "x_codes", (u8,))
    E, N, K2, pw = _experts(W_codes, "W_codes", dev)
    if K2 != K:
        raise ValueError(f"W_codes: {K2} columns, x_codes has {K}")
    if sorted_pairs is None:
        rows = X
    else:
        if not isinstance(sorted_pairs, torch.Tensor):
            raise TypeError(f"sorted_pairs: expected a torch.Tensor, got {type(sorted_pairs).__name__}")
        rows = sorted_pairs.numel()
        if rows > 0x7fffffff:
            raise ValueError(f"sorted_pairs: {rows} pairs are past 2^31 - 1")
    if y_f32 is None and y_bf16 is None:
        y_f32 = _new((rows, N), f32, dev, stream)
        with torch.cuda.stream(_as_stream(stream, dev)):
            y_f32.zero_()
    _run_on(dev, stream, _c().grouped_skinny_gemm_fp8, rows, X, E, N, K, px,
            _arg(x_scales, f32, (_blocks(K), X), "x_scales", dev), pw,
            _arg(W_scales, f32, (E, _blocks(N), _blocks(K)), "W_scales", dev),
            _arg(expert_offsets, i32, (E + 1,), "expert_offsets", dev),
            None if sorted_pairs is None else _arg(sorted_pairs, i32, (rows,), "sorted_pairs", dev),
            topk, None if y_f32 is None else _arg(y_f32, f32, (rows, N), "y_f32", dev),
            None if y_bf16 is None else _arg(y_bf16, torch.bfloat16, (rows, N), "y_bf16", dev))
    return y_f32, y_bf16


def skinny_moe_fp8_step_workspace(T: int, topk: int, E: int, H: int, F: int) -> int:
    """Workspace bytes skinny_moe_fp8_step needs (0 if the sizes are rejected)."""
    return int(_c().skinny_moe_fp8_step_workspace(T, topk, E, H, F))


def skinny_moe_fp8_step(x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                        W_gate_up: torch.Tensor, gate_up_scales: torch.Tensor,
                        W_down: torch.Tensor, down_scales: torch.Tensor, r=None, out=None,
                        workspace=None, stream=None):
    """The routed experts of any number of tokens, with block-scaled FP8 weights: out[t] = (r[t] +)
    sum_j topk_weights[t, j] * down_e(swiglu(gate_up_e(x[t]))) for e = topk_ids[t, j], x and the
    gated product quantised by skinny_quant_fp8; ids outside [0, E) are left out.  x, r [T, H] bf16,
    topk_ids int32 and topk_weights float32 [T, topk], W_gate_up uint8 [E, 2F, H] (gate rows, then
    up rows) and W_down uint8 [E, H, F] with float32 scales per 128 x 128 block.  out bf16 [T, H]
    (may be x or r itself; allocated when not given).  Returns out."""
    T, H, dev, px = _rows(x, "x", (torch.bfloat16,))
    topk = _rows(topk_ids, "topk_ids", (torch.int32,))[1]
    E, _, F, pd = _experts(W_down, "W_down", dev)
    if out is None:
        out = _new((T, H), torch.bfloat16, dev, stream)
    ws, ws_ptr, ws_bytes = _ws_arg(workspace, _c().skinny_moe_fp8_step_workspace(T, topk, E, H, F), dev,
                                   stream)
    u8, f32, bf16 = torch.uint8, torch.float32, torch.bfloat16
    hb, fb = _blocks(H), _blocks(F)
    step = SgMoeFp8Step(
        px, _arg(topk_ids, torch.int32, (T, topk), "topk_ids", dev),
        _arg(topk_weights, f32, (T, topk), "topk_weights", dev),
        _arg(W_gate_up, u8, (E, 2 * F, H), "W_gate_up", dev),
        _arg(gate_up_scales, f32, (E, _blocks(2 * F), hb), "gate_up_scales", dev),
        _arg(W_down, u8, (E, H, F), "W_down", dev),
        _arg(down_scales, f32, (E, hb, fb), "down_scales", dev),
        None if r is None else _arg(r, bf16, (T, H), "r", dev),
        _arg(out, bf16, (T, H), "out", dev), T, topk, E, H, F)
    _run_on(dev, stream, _c().skinny_moe_fp8_step, ctypes.byref(step), ws_ptr, ws_bytes)
    return out


def concat_router_shared(W_router: torch.Tensor, W_shared: torch.Tensor):
    """One [E + N_shared, K] tensor holding the router rows, then the shared expert's;
    returns its two views (W_router, W_shared) -- the weight layout the fused step reads."""
    both = torch.cat([W_router, W_shared], dim=0).contiguous()
    return both[:W_router.shape[0]], both[W_router.shape[0]:]


MOE_STEP_MODES = ("fused", "side_stream", "serial", "shared_in_routed")


def skinny_moe_step(x: torch.Tensor, W_router: torch.Tensor, W_experts: torch.Tensor,
                    W_shared, topk: int, mode: str = "fused", workspace=None, stream=None):
    """One MoE decode step: router scores, top-k and routed-expert projection on `stream`,
    plus the shared expert's projection (W_shared [N_shared,K], or None):
      "fused"       -- in the router's GEMM; W_shared must be stored right after W_router
                       (the two views concat_router_shared returns);
      "side_stream" -- on a side stream that overlaps the routing phase;
      "serial"      -- after the routed experts on `stream`;
      "shared_in_routed" -- up to 4 tokens (E <= 512), inside the routed-expert launch,
                       streamed while it ranks the scores (else as "serial").
    Returns (topk_ids [T,topk] int32, topk_scores [T,topk], scores [T,E], out [T,topk,N],
    shared_out [T,N_shared]; fp32).  In fused mode scores and shared_out are column
    views of one [T, E + N_shared] buffer."""
    if mode not in MOE_STEP_MODES:
        raise ValueError(f"mode: one of {MOE_STEP_MODES}")
    dev = x.device
    T, K = x.shape
    E, N, K2 = W_experts.shape
    N_shared = 0 if W_shared is None else W_shared.shape[0]
    if W_router.shape != (E, K) or K2 != K or (W_shared is not None and W_shared.shape[1] != K):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, W_router {tuple(W_router.shape)}, "
                         f"W_experts {tuple(W_experts.shape)}")
    fused = mode == "fused" and N_shared > 0
    if fused and W_shared.data_ptr() != W_router.data_ptr() + E * K * W_router.element_size():
        raise ValueError("fused mode: W_shared must follow W_router in memory "
                         "(use concat_router_shared)")
    f32 = dict(dtype=torch.float32, device=dev)
    ids = torch.empty((T, topk), dtype=torch.int32, device=dev)
    top = torch.empty((T, topk), **f32)
    out = torch.empty((T, topk, N), **f32)
    if fused:
        y = torch.empty((T, E + N_shared), **f32)
        scores, shared_out = y[:, :E], y[:, E:]
        w_router_ptr = _ptr(W_router, torch.bfloat16, "W_router", dev)
        scores_ptr, shared_ptr, w_shared_ptr = y.data_ptr() or None, None, None
    else:
        scores, shared_out = torch.empty((T, E), **f32), torch.empty((T, N_shared), **f32)
        w_router_ptr = _ptr(W_router, torch.bfloat16, "W_router", dev)
        scores_ptr = _ptr(scores, torch.float32, "scores", dev)
        shared_ptr = _ptr(shared_out, torch.float32, "shared_out", dev)
        w_shared_ptr = _ptr(W_shared, torch.bfloat16, "W_shared", dev)
    need = skinny_moe_step_workspace(T, K, E, topk, N, N_shared)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    step = SgMoeStep(
        _ptr(x, torch.bfloat16, "x", dev), w_router_ptr,
        _ptr(W_experts, torch.bfloat16, "W_experts", dev), w_shared_ptr, scores_ptr,
        _ptr(ids, torch.int32, "topk_ids", dev), _ptr(top, torch.float32, "topk_scores", dev),
        _ptr(out, torch.float32, "out", dev), shared_ptr, T, K, E, topk, N, N_shared,
        _lib.SG_MOE_STEP_FUSED_SHARED if fused
        else _lib.SG_MOE_STEP_SHARED_IN_ROUTED if mode == "shared_in_routed" else 0)
    side = fork = join = None
    if mode == "side_stream":
        s, f, j = _side_resources(dev)
        side, fork, join = s.cuda_stream, f.cuda_event, j.cuda_event
    st = _c().skinny_moe_step(ctypes.byref(step), _ptr(workspace, torch.uint8, "workspace", dev),
                              ws_bytes, _stream(stream), side, fork, join)
    _lib.check(st)
    return ids, top, scores, out, shared_out


def skinny_gemm_status_str(status: int) -> str:
    return _c().skinny_gemm_status_str(status).decode()


def skinny_gemm_read_counters(n: int) -> list[int]:
    """The first n launch counters, by SG_KERNEL_* (zeros behind the last one)."""
    arr = (ctypes.c_uint64 * n)()
    _c().skinny_gemm_read_counters(arr, n)
    return list(arr)


def skinny_gemm_get_counters() -> list[int]:
    return skinny_gemm_read_counters(SG_NUM_COUNTERS)


def skinny_gemm_reset_counters() -> None:
    _c().skinny_gemm_reset_counters()
