"""GB300-native bitmask N:M decode SpMV (the decode kernel of SparseDecoding).

This package is a thin ctypes binding over ``libnmspmv.so`` (C ABI in
``include/nmspmv.h``). Every step of the computation runs in the library's
CUDA kernels; this module only checks tensor types and passes pointers, sizes
and the current CUDA stream. PyTorch supplies device memory and streams.

There is no fallback: if the library is not built, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Iterable, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# NM_LIBRARY may name another build of the library (the bounds-checking one).
LIB_PATH = os.environ.get("NM_LIBRARY") or os.path.join(_HERE, "libnmspmv.so")

NM_OK = 0
NM_ERR_INVALID_ARG = 1
NM_ERR_SHAPE = 2
NM_ERR_ALIGN = 3
NM_ERR_UNSUPPORTED = 4
NM_ERR_NOT_NM = 5
NM_ERR_CUDA = 6
NM_ERR_TIMEOUT = 7
NM_ERR_NOT_PD = 8
NM_ERR_BOUNDS = 9

PATTERNS = ((2, 4), (4, 8), (8, 16), (16, 32))

NM_STACK_DENSE = 1
NM_STACK_PERSISTENT = 2
NM_LINEAR_SWIGLU = 1
NM_LINEAR_QKV = 2
NM_OBS_SGEMM = 1

# Every symbol the header declares (the CPU test checks they are exported).
EXPORTS = ("nm_abi_version", "nm_status_str", "nm_pack_host", "nm_select", "nm_pack", "nm_spmv",
           "nm_spmv_f32out", "dense_gemv", "dense_gemv_f32out", "nm_spmv_stack", "dense_gemv_stack",
           "nm_device_status", "nm_spmv_noalloc", "nm_stack_plan_create", "nm_stack_plan_run",
           "nm_stack_plan_destroy", "nm_pack_swiglu", "nm_spmv_swiglu", "nm_obs_hessian", "nm_obs_prune",
           "nm_spmv_f32out_atomic", "nm_select_pack", "nm_spmv_qkv", "nm_obs_release_workspace",
           "nm_kv4_page_bytes", "nm_kv4_workspace_bytes", "nm_kv4_init", "nm_kv4_reserve", "nm_kv4_fork",
           "nm_kv4_free", "nm_kv4_compact", "nm_kv4_copy_pages", "nm_kv4_append", "nm_kv4_read",
           "nm_kv4_attention",
           "nm_kv8_page_bytes", "nm_kv8_workspace_bytes", "nm_kv8_init", "nm_kv8_reserve", "nm_kv8_fork",
           "nm_kv8_free", "nm_kv8_compact", "nm_kv8_copy_pages", "nm_kv8_append", "nm_kv8_read",
           "nm_kv8_attention", "nm_kv8_select")


class NmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} (status {status})")


class NmLinear(ctypes.Structure):
    """Mirror of ``nm_linear`` in include/nmspmv.h."""
    _fields_ = [("masks", ctypes.c_void_p), ("values", ctypes.c_void_p), ("W", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("K", ctypes.c_int64), ("flags", ctypes.c_uint32), ("y_k", ctypes.c_void_p),
                ("y_v", ctypes.c_void_p), ("rows_q", ctypes.c_int64), ("rows_k", ctypes.c_int64)]


class NmKv4Cache(ctypes.Structure):
    """Mirror of ``nm_kv4_cache`` in include/nmspmv.h."""
    _fields_ = [("pool", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_tokens", ctypes.c_int32),
                ("n_layers", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("max_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("info", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("tables", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load libnmspmv.so (built by ``sparse_decoding_gb300.build``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m sparse_decoding_gb300.build` "
                           "(or __graft_entry__.build()) first")
    L = ctypes.CDLL(LIB_PATH)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    sig = {
        "nm_abi_version": ([], i32),
        "nm_status_str": ([i32], ctypes.c_char_p),
        "nm_pack_host": ([p, i64, i64, i32, i32, p, p], i32),
        "nm_select": ([p, p, i64, i64, i32, i32, p, p], i32),
        "nm_pack": ([p, i64, i64, i32, i32, p, p, p], i32),
        "nm_select_pack": ([p, p, i64, i64, i32, i32, p, p, p], i32),
        "nm_spmv": ([p, p, p, p, i64, i64, i32, p], i32),
        "nm_spmv_f32out": ([p, p, p, p, i64, i64, i32, p], i32),
        "nm_spmv_f32out_atomic": ([p, p, p, p, i64, i64, i32, p], i32),
        "nm_spmv_qkv": ([p, p, p, p, p, p, i64, i64, i64, i64, i32, p], i32),
        "dense_gemv": ([p, p, p, i64, i64, i32, p], i32),
        "dense_gemv_f32out": ([p, p, p, i64, i64, i32, p], i32),
        "nm_spmv_stack": ([ctypes.POINTER(NmLinear), i32, i32, p], i32),
        "dense_gemv_stack": ([ctypes.POINTER(NmLinear), i32, i32, p], i32),
        "nm_device_status": ([p], i32),
        "nm_spmv_noalloc": ([p, p, p, p, i64, i64, i32, p], i32),
        "nm_stack_plan_create": ([ctypes.POINTER(NmLinear), i32, i32, ctypes.c_uint, ctypes.POINTER(p)], i32),
        "nm_stack_plan_run": ([p, p], i32),
        "nm_stack_plan_destroy": ([p], i32),
        "nm_pack_swiglu": ([p, p, i64, i64, i32, i32, p, p, p], i32),
        "nm_spmv_swiglu": ([p, p, p, p, i64, i64, i32, p], i32),
        "nm_obs_hessian": ([p, i64, i64, p, i32, p], i32),
        "nm_obs_prune": ([p, p, i64, i64, i32, i32, ctypes.c_float, ctypes.c_uint, p, p, p, p], i32),
        "nm_obs_release_workspace": ([], i32),
        "nm_kv4_page_bytes": ([i32, i32, i32, i32], i64),
        "nm_kv4_workspace_bytes": ([i64, i32], i64),
        "nm_kv4_init": ([p, p], i32),
        "nm_kv4_reserve": ([p, p, p, i32, p], i32),
        "nm_kv4_fork": ([p, p, p, i32, p], i32),
        "nm_kv4_free": ([p, p, i32, p], i32),
        "nm_kv4_compact": ([p, p], i32),
        "nm_kv4_copy_pages": ([p, p, p, p, i64, p], i32),
        "nm_kv4_append": ([p, i32, p, p, i32, i64, p, i64, p, i64, p, i64, i32, p, i64, p, i64, p], i32),
        "nm_kv4_read": ([p, i32, p, p, i32, i64, p, p, i32, p], i32),
        "nm_kv4_attention": ([p, i32, p, p, i32, i64, i64, p, i64, i32, ctypes.c_float, p, i64, p, p], i32),
    }
    for call in ("page_bytes", "workspace_bytes", "init", "reserve", "fork", "free", "compact", "copy_pages", "append", "read"):
        sig["nm_kv8_" + call] = sig["nm_kv4_" + call]
    sig["nm_kv8_attention"] = ([p, i32, p, p, i32, i64, i64, p, i64, i32, ctypes.c_float, p, i32, p, i64, p, p], i32)
    sig["nm_kv8_select"] = ([p, i32, p, p, i32, i64, p, i64, i32, i32, i32, i32, p, p], i32)
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def status_str(status: int) -> str:
    return lib().nm_status_str(int(status)).decode()


def _check(status: int, where: str):
    if status != NM_OK:
        raise NmError(status, where)


def _stream(t: Optional[torch.Tensor] = None) -> int:
    dev = t.device if t is not None else None
    return torch.cuda.current_stream(dev).cuda_stream


def _cuda(t: torch.Tensor, dtype, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise TypeError(f"{name} must be contiguous")
    return t


def _x2d(x: torch.Tensor) -> torch.Tensor:
    return x.unsqueeze(0) if x.dim() == 1 else x


# --- calls ---------------------------------------------------------------------

def init(device: Optional[torch.device] = None) -> None:
    """Allocate the per-device scratch now (do this before any CUDA graph capture)."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _check(lib().nm_device_status(ctypes.c_void_p(_stream())), "nm_device_status")


def device_status() -> int:
    """Wait for the current stream; return and clear the device status word."""
    return lib().nm_device_status(ctypes.c_void_p(_stream()))


def select(W: torch.Tensor, a: torch.Tensor, N: int, M: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Wanda N:M selection on the GPU: keep the N largest |W|*a_j per M-column subgroup."""
    _cuda(W, torch.bfloat16, "W")
    _cuda(a, torch.float32, "a")
    rows, K = W.shape
    out = torch.empty_like(W) if out is None else _cuda(out, torch.bfloat16, "out")
    _check(lib().nm_select(W.data_ptr(), a.data_ptr(), rows, K, N, M, out.data_ptr(),
                           ctypes.c_void_p(_stream(W))), "nm_select")
    return out


def select_pack(W: torch.Tensor, a: torch.Tensor, N: int, M: int):
    """Wanda N:M selection and pack in one pass: dense W (bf16, CUDA) and column norms a (fp32)
    -> (masks int32-viewed uint32 [rows][K/32], values bf16 [rows][K/2]); equal to pack(select(W, a))."""
    _cuda(W, torch.bfloat16, "W")
    _cuda(a, torch.float32, "a")
    rows, K = W.shape
    masks = torch.empty(rows, K // 32, dtype=torch.int32, device=W.device)
    values = torch.empty(rows, K // 2, dtype=torch.bfloat16, device=W.device)
    _check(lib().nm_select_pack(W.data_ptr(), a.data_ptr(), rows, K, N, M, masks.data_ptr(), values.data_ptr(),
                                ctypes.c_void_p(_stream(W))), "nm_select_pack")
    return masks, values


def pack(W: torch.Tensor, N: int, M: int):
    """Pruned dense W (bf16, CUDA) -> (masks int32-viewed uint32 [rows][K/32], values bf16 [rows][K/2])."""
    _cuda(W, torch.bfloat16, "W")
    rows, K = W.shape
    masks = torch.empty(rows, K // 32, dtype=torch.int32, device=W.device)
    values = torch.empty(rows, K // 2, dtype=torch.bfloat16, device=W.device)
    _check(lib().nm_pack(W.data_ptr(), rows, K, N, M, masks.data_ptr(), values.data_ptr(),
                         ctypes.c_void_p(_stream(W))), "nm_pack")
    return masks, values


def pack_host(W: torch.Tensor, N: int, M: int):
    """Host packer: CPU bf16 W -> CPU (masks int32-viewed uint32, values bf16)."""
    if W.is_cuda or W.dtype != torch.bfloat16 or not W.is_contiguous():
        raise TypeError("W must be a contiguous CPU bf16 tensor")
    rows, K = W.shape
    masks = torch.empty(rows, K // 32, dtype=torch.int32)
    values = torch.empty(rows, K // 2, dtype=torch.bfloat16)
    _check(lib().nm_pack_host(W.data_ptr(), rows, K, N, M, masks.data_ptr(), values.data_ptr()), "nm_pack_host")
    return masks, values


def spmv(masks: torch.Tensor, values: torch.Tensor, x: torch.Tensor, out: Optional[torch.Tensor] = None,
         f32: bool = False, atomic: bool = False) -> torch.Tensor:
    """y[b][r] = sum_j W[r][j] x[b][j] over the bitmask format; bf16 (or fp32 with f32=True).

    atomic=True (fp32 only): the split-K variant that combines row-block parts
    with atomicAdd (nm_spmv_f32out_atomic)."""
    if atomic and not f32:
        raise ValueError("the atomicAdd split-K variant writes fp32 (f32=True)")
    _cuda(masks, torch.int32, "masks")
    _cuda(values, torch.bfloat16, "values")
    x = _cuda(_x2d(x), torch.bfloat16, "x")
    rows = masks.shape[0]
    K = masks.shape[1] * 32
    batch = x.shape[0]
    if values.shape != (rows, K // 2) or x.shape[1] != K:
        raise ValueError("shape mismatch between masks, values and x")
    odt = torch.float32 if f32 else torch.bfloat16
    out = torch.empty(batch, rows, dtype=odt, device=x.device) if out is None else _cuda(out, odt, "out")
    name = "nm_spmv_f32out_atomic" if atomic else "nm_spmv_f32out" if f32 else "nm_spmv"
    _check(getattr(lib(), name)(masks.data_ptr(), values.data_ptr(), x.data_ptr(), out.data_ptr(), rows, K, batch,
                                ctypes.c_void_p(_stream(x))), name)
    return out


def spmv_qkv(masks: torch.Tensor, values: torch.Tensor, x: torch.Tensor, rows_q: int, rows_k: int,
             out: Optional[Sequence[torch.Tensor]] = None):
    """The SpMV of a fused q/k/v matrix (q rows, then k rows, then v rows) into three bf16
    buffers q [batch][rows_q], k [batch][rows_k], v [batch][rows_v]; returns (q, k, v)."""
    _cuda(masks, torch.int32, "masks")
    _cuda(values, torch.bfloat16, "values")
    x = _cuda(_x2d(x), torch.bfloat16, "x")
    rows = masks.shape[0]
    K = masks.shape[1] * 32
    batch = x.shape[0]
    rows_v = rows - rows_q - rows_k
    if values.shape != (rows, K // 2) or x.shape[1] != K or rows_q < 0 or rows_k < 0 or rows_v < 0:
        raise ValueError("shape mismatch between masks, values, x and the q/k/v row counts")
    if out is None:
        out = [torch.empty(batch, r, dtype=torch.bfloat16, device=x.device) for r in (rows_q, rows_k, rows_v)]
    q, k, v = (_cuda(t, torch.bfloat16, n) for t, n in zip(out, ("q", "k", "v")))
    _check(lib().nm_spmv_qkv(masks.data_ptr(), values.data_ptr(), x.data_ptr(), q.data_ptr(), k.data_ptr(),
                             v.data_ptr(), rows_q, rows_k, rows_v, K, batch, ctypes.c_void_p(_stream(x))),
           "nm_spmv_qkv")
    return q, k, v


def pack_swiglu(W_gate: torch.Tensor, W_up: torch.Tensor, N: int, M: int):
    """Pruned gate and up matrices (bf16, CUDA, [rows_h][K]) -> (masks, values) in the pair
    layout of nm_pack_swiglu: [2*rows_h][K/32] and [2*rows_h][K/2]."""
    _cuda(W_gate, torch.bfloat16, "W_gate")
    _cuda(W_up, torch.bfloat16, "W_up")
    if W_gate.shape != W_up.shape:
        raise ValueError("W_gate and W_up must have the same shape")
    rows_h, K = W_gate.shape
    masks = torch.empty(2 * rows_h, K // 32, dtype=torch.int32, device=W_gate.device)
    values = torch.empty(2 * rows_h, K // 2, dtype=torch.bfloat16, device=W_gate.device)
    _check(lib().nm_pack_swiglu(W_gate.data_ptr(), W_up.data_ptr(), rows_h, K, N, M, masks.data_ptr(),
                                values.data_ptr(), ctypes.c_void_p(_stream(W_gate))), "nm_pack_swiglu")
    return masks, values


def spmv_swiglu(masks: torch.Tensor, values: torch.Tensor, x: torch.Tensor,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h[b][r] = bf16(silu(g) * u), g and u the gate and up rows of a pair-layout matrix times x."""
    _cuda(masks, torch.int32, "masks")
    _cuda(values, torch.bfloat16, "values")
    x = _cuda(_x2d(x), torch.bfloat16, "x")
    rows = masks.shape[0]
    K = masks.shape[1] * 32
    batch = x.shape[0]
    if values.shape != (rows, K // 2) or x.shape[1] != K or rows % 32 != 0:
        raise ValueError("shape mismatch between masks, values and x (rows must be a multiple of 32)")
    out = torch.empty(batch, rows // 2, dtype=torch.bfloat16, device=x.device) if out is None else \
        _cuda(out, torch.bfloat16, "out")
    _check(lib().nm_spmv_swiglu(masks.data_ptr(), values.data_ptr(), x.data_ptr(), out.data_ptr(), rows // 2, K,
                                batch, ctypes.c_void_p(_stream(x))), "nm_spmv_swiglu")
    return out


def dense_gemv(W: torch.Tensor, x: torch.Tensor, out: Optional[torch.Tensor] = None,
               f32: bool = False) -> torch.Tensor:
    """Dense bf16 reference: y[b][r] = sum_j W[r][j] x[b][j]."""
    _cuda(W, torch.bfloat16, "W")
    x = _cuda(_x2d(x), torch.bfloat16, "x")
    rows, K = W.shape
    batch = x.shape[0]
    if x.shape[1] != K:
        raise ValueError("shape mismatch between W and x")
    odt = torch.float32 if f32 else torch.bfloat16
    out = torch.empty(batch, rows, dtype=odt, device=x.device) if out is None else _cuda(out, odt, "out")
    fn = lib().dense_gemv_f32out if f32 else lib().dense_gemv
    _check(fn(W.data_ptr(), x.data_ptr(), out.data_ptr(), rows, K, batch, ctypes.c_void_p(_stream(x))),
           "dense_gemv")
    return out


def _linear_array(ops: Sequence[dict]) -> ctypes.Array:
    arr = (NmLinear * len(ops))()
    for i, op in enumerate(ops):
        t = arr[i]
        for f in ("masks", "values", "W", "x", "y"):
            v = op.get(f)
            setattr(t, f, v.data_ptr() if v is not None else None)
        t.rows = int(op["rows"])
        t.K = int(op["K"])
        t.flags = int(op.get("flags", 0))
        for f in ("y_k", "y_v"):
            v = op.get(f)
            setattr(t, f, v.data_ptr() if v is not None else None)
        t.rows_q = int(op.get("rows_q", 0))
        t.rows_k = int(op.get("rows_k", 0))
    return arr


def spmv_stack(ops: Sequence[dict], batch: int) -> None:
    """Run a decode-token linear stack: ops[i] = {masks, values, x, y, rows, K}, in order."""
    arr = _linear_array(ops)
    _check(lib().nm_spmv_stack(arr, len(ops), batch, ctypes.c_void_p(_stream())), "nm_spmv_stack")


def dense_gemv_stack(ops: Sequence[dict], batch: int) -> None:
    """Dense counterpart of spmv_stack: ops[i] = {W, x, y, rows, K}."""
    arr = _linear_array(ops)
    _check(lib().dense_gemv_stack(arr, len(ops), batch, ctypes.c_void_p(_stream())), "dense_gemv_stack")


class StackPlan:
    """A decode-token stack prepared once (``nm_stack_plan``); ``run()`` launches it.

    By default each op is its own kernel, chained with programmatic dependent
    launch; with ``persistent=True`` the whole stack is one persistent kernel
    launch with a grid barrier between ops (when every op is on the TMA path).
    The plan holds the ops' device pointers: it keeps their tensors alive
    until ``close()``.
    """

    def __init__(self, ops: Sequence[dict], batch: int, dense: bool = False, persistent: bool = False):
        self._keep = list(ops)
        self.batch = batch
        self.dense = dense
        arr = _linear_array(self._keep)
        flags = (NM_STACK_DENSE if dense else 0) | (NM_STACK_PERSISTENT if persistent else 0)
        h = ctypes.c_void_p()
        _check(lib().nm_stack_plan_create(arr, len(self._keep), batch, flags, ctypes.byref(h)),
               "nm_stack_plan_create")
        self._h = h

    def run(self) -> None:
        if self._h is None:
            raise RuntimeError("StackPlan is closed")
        _check(lib().nm_stack_plan_run(self._h, ctypes.c_void_p(_stream())), "nm_stack_plan_run")

    def close(self) -> None:
        if getattr(self, "_h", None) is not None:
            h, self._h = self._h, None
            _check(lib().nm_stack_plan_destroy(h), "nm_stack_plan_destroy")
            self._keep = []

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --- N:M pruning by the OBS rule --------------------------------------------------

def obs_hessian(X: torch.Tensor, H: Optional[torch.Tensor] = None, accumulate: bool = False) -> torch.Tensor:
    """H = 2 X^T X (or H += 2 X^T X) for calibration inputs X, bf16 [T][K] -> fp32 [K][K]."""
    _cuda(X, torch.bfloat16, "X")
    T, K = X.shape
    if H is None:
        if accumulate:
            raise ValueError("accumulate needs H")
        H = torch.empty(K, K, dtype=torch.float32, device=X.device)
    _cuda(H, torch.float32, "H")
    if tuple(H.shape) != (K, K):
        raise ValueError("H must be [K][K]")
    _check(lib().nm_obs_hessian(X.data_ptr(), T, K, H.data_ptr(), int(bool(accumulate)),
                                ctypes.c_void_p(_stream(X))), "nm_obs_hessian")
    return H


def obs_prune(W: torch.Tensor, H: torch.Tensor, N: int, M: int, percdamp: float = 0.01, sgemm: bool = False,
              masks: bool = True, f32: bool = False):
    """OBS N:M pruning of W (bf16 [rows][K]) against H (fp32 [K][K]). Synchronous.

    Returns (W_pruned bf16 [rows][K], keep masks int32-viewed uint32 [rows][K/32] or
    None, W_pruned fp32 or None)."""
    _cuda(W, torch.bfloat16, "W")
    _cuda(H, torch.float32, "H")
    rows, K = W.shape
    if tuple(H.shape) != (K, K):
        raise ValueError("H must be [K][K]")
    out = torch.empty_like(W)
    m = torch.empty(rows, K // 32, dtype=torch.int32, device=W.device) if masks else None
    wf = torch.empty(rows, K, dtype=torch.float32, device=W.device) if f32 else None
    _check(lib().nm_obs_prune(W.data_ptr(), H.data_ptr(), rows, K, N, M, float(percdamp),
                              NM_OBS_SGEMM if sgemm else 0, out.data_ptr(),
                              m.data_ptr() if m is not None else None,
                              wf.data_ptr() if wf is not None else None,
                              ctypes.c_void_p(_stream(W))), "nm_obs_prune")
    return out, m, wf


def obs_release_workspace():
    """Return the memory the OBS calls keep for their workspaces on the current device."""
    _check(lib().nm_obs_release_workspace(), "nm_obs_release_workspace")


# --- the paged KV caches --------------------------------------------------------------

def _pad4(n: int) -> int:
    return (n + 3) // 4 * 4


class Kv4Cache:
    """A paged KV cache in 4 bits (``nm_kv4_*``): grouped-query attention's keys and values of
    every layer, in pages of ``page_tokens`` tokens (16, 32, 64 or 128), head_dim 64 or 128.

    ``pool`` (uint8 [n_pages][page bytes]) holds the pages and ``book`` (int32) the bookkeeping:
    the views ``info`` [16], ``lens`` [max_seqs], ``refs`` [n_pages] and ``tables``
    [max_seqs][max_pages] (see include/nmspmv.h). Both are made here, empty, or taken over as
    they are. All calls are asynchronous on the current stream; calls on one cache must not
    overlap on the GPU. ``seqs`` (int32, CUDA) names the sequences of a call, None: 0, 1, ...;
    ``starts`` (int32 [n + 1], CUDA) bounds each one's new tokens in the token tensors, None: one
    token each. Token tensors are bf16 [tokens][heads][head_dim] or [tokens][heads * head_dim];
    the token stride is free. After an NM_ERR_TIMEOUT, go on with a new Kv4Cache over this one's
    ``pool`` and ``book`` (its workspace starts clean).
    """

    _calls = "nm_kv4_"  # the C calls of the format

    def __init__(self, n_pages: int, page_tokens: int, n_layers: int, n_kv_heads: int, head_dim: int, max_seqs: int,
                 max_pages: int, device: Optional[torch.device] = None, pool: Optional[torch.Tensor] = None,
                 book: Optional[torch.Tensor] = None):
        L = lib()
        per = getattr(L, self._calls + "page_bytes")(page_tokens, n_layers, n_kv_heads, head_dim)
        if per == 0 or n_pages < 0 or max_seqs < 0 or max_pages < 0:
            raise NmError(NM_ERR_UNSUPPORTED, type(self).__name__)
        given = pool if pool is not None else book
        device = given.device if given is not None else torch.device(device if device is not None else "cuda")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device, self.n_pages, self.page_tokens = device, n_pages, page_tokens
        self._index = device.index
        self._f = {x: getattr(L, self._calls + x) for x in ("init", "reserve", "fork", "free", "compact", "copy_pages", "append",
                                                            "read", "attention")}
        self.n_layers, self.n_kv_heads, self.head_dim = n_layers, n_kv_heads, head_dim
        ints = self.book_ints(n_pages, max_seqs, max_pages)
        fresh = book is None
        self.pool = torch.empty(n_pages, per, dtype=torch.uint8, device=device) if pool is None else \
            _cuda(pool, torch.uint8, "pool")
        self.book = torch.empty(ints, dtype=torch.int32, device=device) if fresh else _cuda(book, torch.int32, "book")
        if tuple(self.pool.shape) != (n_pages, per) or self.book.numel() != ints:
            raise ValueError(f"pool must be [{n_pages}][{per}] and book have {ints} ints")
        if self.pool.device != device or self.book.device != device:
            raise ValueError("pool and book must be on one device")
        a = 16 + _pad4(max_seqs)
        b = a + _pad4(n_pages)
        self.info, self.lens, self.refs = self.book[:16], self.book[16:16 + max_seqs], self.book[a:a + n_pages]
        self.tables = self.book[b:b + max_seqs * max_pages].view(max_seqs, max_pages)
        self._work = torch.empty(getattr(L, self._calls + "workspace_bytes")(n_pages, head_dim), dtype=torch.uint8, device=device)
        self._work[:8192].zero_()  # the join counters
        base = self.book.data_ptr()
        self._c = NmKv4Cache(self.pool.data_ptr(), n_pages, page_tokens, n_layers, n_kv_heads, head_dim, max_seqs,
                             max_pages, base, base + 64, base + 4 * a, base + 4 * b, self._work.data_ptr(),
                             self._work.numel())
        self._ref = ctypes.byref(self._c)
        if fresh:
            self._ok(self._f["init"](self._ref, self._s()), "init")

    @staticmethod
    def book_ints(n_pages: int, max_seqs: int, max_pages: int) -> int:
        """Ints of ``book``: info, lens, refs and tables, each padded to a multiple of four."""
        return 16 + _pad4(max_seqs) + _pad4(n_pages) + _pad4(max_seqs * max_pages)

    def _ok(self, status: int, call: str):
        if status != NM_OK:
            raise NmError(status, self._calls + call)

    def _s(self) -> int:
        if torch.cuda.current_device() != self._index:
            raise ValueError(f"the cache is on {self.device}: make it the current device")
        return torch._C._cuda_getCurrentRawStream(self._index)

    def _ids(self, t: Optional[torch.Tensor], name: str):
        if t is None:
            return None
        _cuda(t, torch.int32, name)
        if t.device != self.device or t.dim() != 1:
            raise ValueError(f"{name} must be one-dimensional on {self.device}")
        return t.data_ptr()

    def _batch(self, seqs, starts, n_tokens=None):
        """(seqs pointer, starts pointer, n_seqs) of a call."""
        if seqs is None and starts is None and n_tokens is not None:
            return None, None, n_tokens
        n = starts.numel() - 1 if starts is not None else seqs.numel() if seqs is not None else n_tokens
        if n is None or n < 0 or (seqs is not None and seqs.numel() != n) or \
                (starts is None and n_tokens is not None and n != n_tokens):
            raise ValueError("seqs, starts and the token count do not agree")
        return self._ids(seqs, "seqs"), self._ids(starts, "starts"), n

    def _tokens(self, t: torch.Tensor, name: str):
        """(pointer, token stride, heads) of a token tensor."""
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or not t.is_cuda or \
                t.get_device() != self._index:
            raise TypeError(f"{name} must be a bfloat16 tensor on {self.device}")
        D, shape, stride = self.head_dim, t.shape, t.stride()
        if len(shape) == 3 and shape[2] == D and stride[2] == 1 and (stride[1] == D or shape[1] == 1):
            heads = shape[1]
        elif len(shape) == 2 and shape[1] % D == 0 and stride[1] == 1:
            heads = shape[1] // D
        else:
            raise ValueError(f"{name} must be [tokens][heads][{D}] or [tokens][heads * {D}], contiguous in a token")
        return t.data_ptr(), stride[0] if shape[0] > 1 else heads * D, heads

    def reserve(self, seqs: Optional[torch.Tensor] = None, starts: Optional[torch.Tensor] = None,
                n: Optional[int] = None) -> None:
        """Room for the new tokens of each sequence (``n`` sequences with both None): lens grow, pages
        are added. All or nothing; ``info[1]`` (on the device) tells. After a refusal nothing may be
        appended: the tokens would fall on the sequences' last ones."""
        p, st, m = self._batch(seqs, starts, n)
        self._ok(self._f["reserve"](self._ref, p, st, m, self._s()), "reserve")

    def fork(self, src: torch.Tensor, dst: torch.Tensor) -> None:
        """The empty sequences dst become copies of src, sharing its full pages. ``info[1]`` tells."""
        if src.numel() != dst.numel():
            raise ValueError("src and dst must have the same length")
        self._ok(self._f["fork"](self._ref, self._ids(src, "src"), self._ids(dst, "dst"), src.numel(), self._s()), "fork")

    def free(self, seqs: torch.Tensor) -> None:
        """Empties the listed sequences."""
        self._ok(self._f["free"](self._ref, self._ids(seqs, "seqs"), seqs.numel(), self._s()), "free")

    def compact(self) -> None:
        """Moves the pages in use to the front of the pool; the tables follow."""
        self._ok(self._f["compact"](self._ref, self._s()), "compact")

    def copy_pages(self, src_pages: torch.Tensor, dst_pages: torch.Tensor, dst: Optional["Kv4Cache"] = None) -> None:
        """Copies whole pages of this pool to pages of ``dst``'s (default: this one)."""
        dst = self if dst is None else dst
        if src_pages.numel() != dst_pages.numel() or dst.device != self.device or dst._calls != self._calls:
            raise ValueError("page lists must have the same length, and the caches one device and format")
        self._ok(self._f["copy_pages"](self._ref, self._ids(src_pages, "src_pages"), dst._ref,
                                       self._ids(dst_pages, "dst_pages"), src_pages.numel(), self._s()), "copy_pages")

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, q: Optional[torch.Tensor] = None,
               rope: Optional[torch.Tensor] = None, seqs: Optional[torch.Tensor] = None,
               starts: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None):
        """Writes the new tokens' k (rotated by ``rope``, fp32 [positions][head_dim]: cos, then sin) and v to
        the cache; returns q rotated (None without q). q_out may be q itself."""
        kp, ks, kh = self._tokens(k, "k")
        vp, vs, vh = self._tokens(v, "v")
        T = k.shape[0]
        if kh != self.n_kv_heads or vh != kh or v.shape[0] != T:
            raise ValueError(f"k and v must have {self.n_kv_heads} heads and the same tokens")
        qp = op = None
        qs = os_ = qh = 0
        if q is not None:
            qp, qs, qh = self._tokens(q, "q")
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            op, os_, oh = self._tokens(q_out, "q_out")
            if q.shape[0] != T or q_out.shape[0] != T or oh != qh:
                raise ValueError("q and q_out must have the tokens of k, and the same heads")
        rp, rows = None, 0
        if rope is not None:
            _cuda(rope, torch.float32, "rope")
            if rope.dim() != 2 or rope.shape[1] != self.head_dim or rope.device != self.device:
                raise ValueError(f"rope must be [positions][{self.head_dim}] on {self.device}")
            rp, rows = rope.data_ptr(), rope.shape[0]
        sp, st, n = self._batch(seqs, starts, T if starts is None else None)
        self._ok(self._f["append"](self._ref, layer, sp, st, n, T, kp, ks, vp, vs, qp, qs, qh, op, os_, rp, rows,
                                   self._s()), "append")
        return q_out if q is not None else None

    def read(self, layer: int, n_tokens: int, seqs: Optional[torch.Tensor] = None,
             starts: Optional[torch.Tensor] = None, f32: bool = False):
        """The values held for the last tokens of each sequence: (k, v), [n_tokens][n_kv_heads][head_dim]
        in bf16 (fp32 with f32)."""
        sp, st, n = self._batch(seqs, starts, n_tokens if starts is None else None)
        shape = (n_tokens, self.n_kv_heads, self.head_dim)
        dt = torch.float32 if f32 else torch.bfloat16
        k, v = torch.empty(shape, dtype=dt, device=self.device), torch.empty(shape, dtype=dt, device=self.device)
        self._ok(self._f["read"](self._ref, layer, sp, st, n, n_tokens, k.data_ptr(), v.data_ptr(), int(f32),
                                 self._s()), "read")
        return k, v

    def attention(self, layer: int, q: torch.Tensor, seqs: Optional[torch.Tensor] = None,
                  starts: Optional[torch.Tensor] = None, max_new: Optional[int] = None,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None, lse: bool = False):
        """Causal attention of the new tokens' q over the cache of one layer; bf16, shaped as q.

        ``max_new``: the most new tokens a sequence has, where the caller knows. It chooses the kernel only,
        but without it (and with ``starts``) all tokens count as one sequence's: eight sequences of five
        drafted tokens then take the kernel for prompts, which is slower for them.
        ``scale`` defaults to head_dim ** -0.5. lse=True: (out, lse), lse fp32 [tokens][heads]."""
        return self._attend(layer, q, seqs, starts, max_new, scale, out, lse)

    def _attend(self, layer, q, seqs, starts, max_new, scale, out, lse, *listed):
        qp, qs, qh = self._tokens(q, "q")
        T = q.shape[0]
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            op, os_ = out.data_ptr(), qh * self.head_dim
        else:
            op, os_, oh = self._tokens(out, "out")
            if out.shape[0] != T or oh != qh:
                raise ValueError("out must have q's tokens and heads")
        sp, st, n = self._batch(seqs, starts, T if starts is None else None)
        ls = torch.empty((T, qh), dtype=torch.float32, device=self.device) if lse else None
        status = self._f["attention"](self._ref, layer, sp, st, n, T, (T or 1) if max_new is None else max_new, qp, qs, qh,
                                      self.head_dim ** -0.5 if scale is None else scale, *listed, op, os_,
                                      ls.data_ptr() if lse else None, self._s())
        self._ok(status, "attention")
        return (out, ls) if lse else out


class Kv8Cache(Kv4Cache):
    """A paged KV cache in 8 bits (``nm_kv8_*``), used as a ``Kv4Cache``: 8-bit floats with a power of two for
    each 16 tokens and kv head (see include/nmspmv.h).

    A full page holds bounds of its keys, from which ``select`` finds the pages that matter to each new
    token; ``attention`` reads the whole cache or the pages listed for each token."""

    _calls = "nm_kv8_"

    def attention(self, layer: int, q: torch.Tensor, seqs: Optional[torch.Tensor] = None,
                  starts: Optional[torch.Tensor] = None, max_new: Optional[int] = None,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None, lse: bool = False,
                  pages: Optional[torch.Tensor] = None):
        """Causal attention of the new tokens' q over the cache of one layer; bf16, shaped as q.

        ``pages`` (int32 [tokens][n_kv_heads][n], from ``select`` or of the caller's own): the pages of its
        sequence that each token attends, ascending, -1 behind; None: all. The rest as ``Kv4Cache.attention``."""
        if pages is None:
            return self._attend(layer, q, seqs, starts, max_new, scale, out, lse, None, 0)
        _cuda(pages, torch.int32, "pages")
        if pages.device != self.device or pages.dim() != 3 or pages.shape[:2] != (q.shape[0], self.n_kv_heads) or \
                pages.shape[2] < 1:
            raise ValueError(f"pages must be [tokens][{self.n_kv_heads}][n], n >= 1, on {self.device}")
        return self._attend(layer, q, seqs, starts, max_new, scale, out, lse, pages.data_ptr(), pages.shape[2])

    def select(self, layer: int, q: torch.Tensor, n: int, seqs: Optional[torch.Tensor] = None,
               starts: Optional[torch.Tensor] = None, first: int = 1, last: int = 1,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The n pages of each new token and kv head (int32 [tokens][n_kv_heads][n], ascending, -1 behind) whose
        keys can have the largest scores with its query heads; the ``first`` pages of the sequence and the
        ``last`` (at least one) up to the token's own are always among them: n >= first + last."""
        qp, qs, qh = self._tokens(q, "q")
        shape = (q.shape[0], self.n_kv_heads, n)
        if out is None:
            out = torch.empty(shape, dtype=torch.int32, device=self.device)
        elif tuple(_cuda(out, torch.int32, "out").shape) != shape or out.device != self.device:
            raise ValueError(f"out must be {list(shape)} on {self.device}")
        sp, st, m = self._batch(seqs, starts, shape[0] if starts is None else None)
        self._ok(lib().nm_kv8_select(self._ref, layer, sp, st, m, shape[0], qp, qs, qh, n, first, last, out.data_ptr(), self._s()),
                 "select")
        return out
