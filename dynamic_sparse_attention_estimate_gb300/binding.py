"""ctypes binding of libdsv.so (the C ABI declared in include/dsv.h).

Argument marshalling only: each function checks dtypes/shapes of the torch tensors it
is given, allocates outputs with torch on the input's device, and passes raw device
pointers, sizes and the current CUDA stream to the library.  Every step of the
computation runs in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple, Optional, Sequence, Tuple, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libdsv.so"
_lib = None

DSV_OK = 0
STATUS_NAMES = {0: "DSV_OK", 1: "DSV_ERR_INVALID_ARG", 2: "DSV_ERR_UNSUPPORTED", 3: "DSV_ERR_WORKSPACE",
                4: "DSV_ERR_CUDA", 5: "DSV_ERR_DEVICE_CHECK"}

EXPORTED = (
    "dsv_estimate_topk_workspace", "dsv_estimate_topk", "dsv_sparse_attn_fwd",
    "dsv_sparse_attn_bwd_workspace", "dsv_sparse_attn_bwd_workspace_min", "dsv_sparse_attn_bwd",
    "dsv_status_string", "dsv_last_error_message", "dsv_last_device_status",
    "dsv_profile_enable", "dsv_profile_read", "dsv_sparse_attn_bwd_noalloc",
    "dsv_estimate_mass_k", "dsv_estimate_topk_csr", "dsv_sparse_attn_fwd_csr",
    "dsv_sparse_attn_bwd_csr_workspace", "dsv_sparse_attn_bwd_csr", "dsv_csr_launch_order",
    "dsv_adaln_fwd", "dsv_adaln_bwd_workspace", "dsv_adaln_bwd",
    "dsv_sparse_attn_bwd_prepare", "dsv_sparse_attn_bwd_prepared", "dsv_sparse_attn_fwd_workspace",
    "dsv_rope3d_table_bytes", "dsv_rope3d_table", "dsv_rope3d_fwd", "dsv_rope3d_bwd",
    "dsv_qk_norm_rope_fwd", "dsv_qk_norm_rope_bwd_workspace", "dsv_qk_norm_rope_bwd",
    "dsv_ffn_gated_fwd_workspace", "dsv_ffn_gated_fwd", "dsv_ffn_gated_bwd_workspace", "dsv_ffn_gated_bwd",
)


class DSVError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}" + (f" ({detail})" if detail else ""))


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("H", ctypes.c_int64), ("N", ctypes.c_int64),
                ("d", ctypes.c_int64), ("r", ctypes.c_int64), ("block", ctypes.c_int64),
                ("k", ctypes.c_int64), ("scale", ctypes.c_float)]


class AdalnDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("N", ctypes.c_int64), ("D", ctypes.c_int64), ("eps", ctypes.c_float)]


class RopeDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("H", ctypes.c_int64), ("N", ctypes.c_int64), ("d", ctypes.c_int64),
                ("rot", ctypes.c_int64 * 3), ("len", ctypes.c_int64 * 3), ("pairing", ctypes.c_int32),
                ("pos_batched", ctypes.c_int32), ("eps", ctypes.c_float)]


class FfnDims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("D", ctypes.c_int64), ("F", ctypes.c_int64), ("act", ctypes.c_int32)]


class ViewStrides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("n", ctypes.c_int64)]


# dsv_view_strides[2] and [3]: sample, head and token strides of each tensor in turn
_Strides6, _Strides9 = ctypes.c_int64 * 6, ctypes.c_int64 * 9


def library_path() -> str:
    """The in-tree libdsv.so, or the file the DSV_LIBRARY variable names (another build of the same
    sources, e.g. one made with different compiler flags)."""
    return os.environ.get("DSV_LIBRARY") or os.path.join(_HERE, _LIB_NAME)


def load_library(path: Optional[str] = None):
    """Load libdsv.so (once).  Raises if it has not been built: there is no fallback."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or library_path()
    if not os.path.exists(p):
        raise RuntimeError(f"{p} not found: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(p)
    vp, sz, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    dp = ctypes.POINTER(Dims)
    lib.dsv_estimate_topk_workspace.argtypes = [dp]
    lib.dsv_estimate_topk_workspace.restype = sz
    lib.dsv_estimate_topk.argtypes = [dp, vp, vp, vp, vp, sz, vp]
    lib.dsv_estimate_topk.restype = st
    lib.dsv_sparse_attn_fwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsv_sparse_attn_fwd.restype = st
    lib.dsv_sparse_attn_fwd_workspace.argtypes = [dp]
    lib.dsv_sparse_attn_fwd_workspace.restype = sz
    lib.dsv_sparse_attn_bwd_workspace.argtypes = [dp]
    lib.dsv_sparse_attn_bwd_workspace.restype = sz
    lib.dsv_sparse_attn_bwd_workspace_min.argtypes = [dp]
    lib.dsv_sparse_attn_bwd_workspace_min.restype = sz
    lib.dsv_sparse_attn_bwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsv_sparse_attn_bwd.restype = st
    lib.dsv_status_string.argtypes = [st]
    lib.dsv_status_string.restype = ctypes.c_char_p
    lib.dsv_last_error_message.argtypes = []
    lib.dsv_last_error_message.restype = ctypes.c_char_p
    lib.dsv_last_device_status.argtypes = [vp]
    lib.dsv_last_device_status.restype = st
    lib.dsv_sparse_attn_bwd_noalloc.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.dsv_sparse_attn_bwd_noalloc.restype = st
    lib.dsv_estimate_mass_k.argtypes = [dp, vp, vp, ctypes.c_float, ctypes.c_uint32, ctypes.c_uint32, vp, vp, vp, vp]
    lib.dsv_estimate_mass_k.restype = st
    lib.dsv_estimate_topk_csr.argtypes = [dp, vp, vp, vp, vp, vp, vp]
    lib.dsv_estimate_topk_csr.restype = st
    lib.dsv_csr_launch_order.argtypes = [dp, vp, vp, vp]
    lib.dsv_csr_launch_order.restype = st
    lib.dsv_sparse_attn_fwd_csr.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.dsv_sparse_attn_fwd_csr.restype = st
    lib.dsv_sparse_attn_bwd_csr_workspace.argtypes = [dp, ctypes.c_int64]
    lib.dsv_sparse_attn_bwd_csr_workspace.restype = sz
    lib.dsv_sparse_attn_bwd_csr.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int64, vp, vp, vp, vp, sz,
                                            vp]
    lib.dsv_sparse_attn_bwd_csr.restype = st
    lib.dsv_sparse_attn_bwd_prepare.argtypes = [dp, vp, vp, sz, vp]
    lib.dsv_sparse_attn_bwd_prepare.restype = st
    lib.dsv_sparse_attn_bwd_prepared.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsv_sparse_attn_bwd_prepared.restype = st
    ap = ctypes.POINTER(AdalnDims)
    lib.dsv_adaln_fwd.argtypes = [ap, vp, vp, vp, vp, vp]
    lib.dsv_adaln_fwd.restype = st
    lib.dsv_adaln_bwd_workspace.argtypes = [ap]
    lib.dsv_adaln_bwd_workspace.restype = sz
    lib.dsv_adaln_bwd.argtypes = [ap, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsv_adaln_bwd.restype = st
    rp, vs = ctypes.POINTER(RopeDims), ctypes.POINTER(ViewStrides)
    lib.dsv_rope3d_table_bytes.argtypes = [rp]
    lib.dsv_rope3d_table_bytes.restype = sz
    lib.dsv_rope3d_table.argtypes = [rp, ctypes.POINTER(ctypes.c_double), vp, vp]
    lib.dsv_rope3d_table.restype = st
    for f in (lib.dsv_rope3d_fwd, lib.dsv_rope3d_bwd):
        f.argtypes = [rp, vp, vs, vp, vp, vp, vs, vp]
        f.restype = st
    lib.dsv_qk_norm_rope_fwd.argtypes = [rp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.dsv_qk_norm_rope_fwd.restype = st
    lib.dsv_qk_norm_rope_bwd_workspace.argtypes = [rp]
    lib.dsv_qk_norm_rope_bwd_workspace.restype = sz
    lib.dsv_qk_norm_rope_bwd.argtypes = [rp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsv_qk_norm_rope_bwd.restype = st
    fp = ctypes.POINTER(FfnDims)
    lib.dsv_ffn_gated_fwd.argtypes = [fp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsv_ffn_gated_fwd.restype = st
    for f in (lib.dsv_ffn_gated_fwd_workspace, lib.dsv_ffn_gated_bwd_workspace):
        f.argtypes = [fp]
        f.restype = sz
    lib.dsv_ffn_gated_bwd.argtypes = [fp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsv_ffn_gated_bwd.restype = st
    lib.dsv_profile_enable.argtypes = [st]
    lib.dsv_profile_enable.restype = st
    lib.dsv_profile_read.argtypes = [ctypes.c_char_p, sz]
    lib.dsv_profile_read.restype = sz
    if path is None:
        _lib = lib
    return lib


def make_dims(B, H, N, d, r, k, block=64, scale: Optional[float] = None) -> Dims:
    return Dims(int(B), int(H), int(N), int(d), int(r), int(block), int(k),
                float(scale) if scale is not None else 0.0)


def _check(status: int, what: str):
    if status != DSV_OK:
        lib = load_library()
        msg = lib.dsv_last_error_message()
        raise DSVError(status, what, msg.decode() if msg else "")


def _stream_ptr(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or t.dim() != ndim or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: need a contiguous CUDA {dtype} tensor with {ndim} dims, got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()} device={t.device}")


# ---------------------------------------------------------------- entry points (same names as the C ABI)

def dsv_estimate_topk_workspace(dims: Dims) -> int:
    return int(load_library().dsv_estimate_topk_workspace(ctypes.byref(dims)))


def dsv_estimate_topk(q_lr: torch.Tensor, k_lr: torch.Tensor, k: int, block: int = 64,
                      idx: Optional[torch.Tensor] = None) -> torch.Tensor:
    """idx [B, H, N/block, k] int32 of the top-k keys per query block (ascending)."""
    _need(q_lr, "q_lr", torch.bfloat16, 4)
    _need(k_lr, "k_lr", torch.bfloat16, 4)
    B, H, N, r = q_lr.shape
    if k_lr.shape != q_lr.shape:
        raise ValueError("q_lr and k_lr must have the same shape")
    dims = make_dims(B, H, N, 0, r, k, block)
    if idx is None:
        idx = torch.empty((B, H, max(N // block, 0), int(k)), dtype=torch.int32, device=q_lr.device)
    lib = load_library()
    ws_bytes = int(lib.dsv_estimate_topk_workspace(ctypes.byref(dims)))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q_lr.device) if ws_bytes else None
    _check(lib.dsv_estimate_topk(ctypes.byref(dims), _ptr(q_lr), _ptr(k_lr), _ptr(idx), _ptr(ws), ws_bytes,
                                 _stream_ptr(q_lr)), "dsv_estimate_topk")
    return idx


def mass_parameters(tau: float, mass: float) -> Tuple[float, int]:
    """(tau_log2, mass_num) as dsv_estimate_mass_k takes them: tau * log2(e) rounded to fp32,
    and the mass fraction in units of 2^-16 (rounded, 1 .. 65536)."""
    import numpy as np
    tau_log2 = float(np.float32(float(tau) / 0.6931471805599453))
    mass_num = int(min(65536, max(1, round(float(mass) * 65536))))
    return tau_log2, mass_num


def dsv_estimate_mass_k(q_lr: torch.Tensor, k_lr: torch.Tensor, tau: float = 1.0 / 64, mass: float = 0.9,
                        block: int = 64, out: Optional[Tuple] = None, with_order: bool = True,
                        dense_above: Optional[float] = None):
    """(k_row int32 [B, H, N/block], rowptr int64 [B*H*N/block + 1], order int32 [B*H*N/block] or
    None): per query block the smallest number of top keys that carry the fraction `mass` of
    the estimated attention mass softmax_j(tau s[b, j]), the CSR offsets, and a launch order
    (longest rows first) for the CSR attention calls (see include/dsv.h).  With `dense_above`, a block whose k exceeds
    that fraction of the keys attends to all of them (the per-block sparse/dense switch)."""
    _need(q_lr, "q_lr", torch.bfloat16, 4)
    _need(k_lr, "k_lr", torch.bfloat16, 4)
    B, H, N, r = q_lr.shape
    if k_lr.shape != q_lr.shape:
        raise ValueError("q_lr and k_lr must have the same shape")
    dims = make_dims(B, H, N, 0, r, max(N, 1), block)
    NB = max(N // block, 0)
    if out is None:
        k_row = torch.empty((B, H, NB), dtype=torch.int32, device=q_lr.device)
        rowptr = torch.empty((B * H * NB + 1,), dtype=torch.int64, device=q_lr.device)
        order = torch.empty((B * H * NB,), dtype=torch.int32, device=q_lr.device) if with_order else None
    else:
        k_row, rowptr, order = out
    tau_log2, mass_num = mass_parameters(tau, mass)
    dense_num = 0 if dense_above is None else int(min(65536, max(0, round(float(dense_above) * 65536))))
    _check(load_library().dsv_estimate_mass_k(ctypes.byref(dims), _ptr(q_lr), _ptr(k_lr), tau_log2, mass_num,
                                              dense_num, _ptr(k_row), _ptr(rowptr), _ptr(order), _stream_ptr(q_lr)),
           "dsv_estimate_mass_k")
    return k_row, rowptr, order


def dsv_estimate_topk_csr(q_lr: torch.Tensor, k_lr: torch.Tensor, k_row: torch.Tensor, rowptr: torch.Tensor,
                          block: int = 64, cols: Optional[torch.Tensor] = None) -> torch.Tensor:
    """cols int32 [rowptr[-1]]: row i's k_row[i] top keys (ascending) at cols[rowptr[i]:rowptr[i+1]].
    Without `cols` the total is read from the device (a synchronisation)."""
    _need(q_lr, "q_lr", torch.bfloat16, 4)
    _need(k_lr, "k_lr", torch.bfloat16, 4)
    B, H, N, r = q_lr.shape
    dims = make_dims(B, H, N, 0, r, max(N, 1), block)
    if cols is None:
        cols = torch.empty((int(rowptr[-1].item()),), dtype=torch.int32, device=q_lr.device)
    _check(load_library().dsv_estimate_topk_csr(ctypes.byref(dims), _ptr(q_lr), _ptr(k_lr), _ptr(k_row), _ptr(rowptr),
                                                _ptr(cols), _stream_ptr(q_lr)), "dsv_estimate_topk_csr")
    return cols


def dsv_sparse_attn_fwd_workspace(dims: Dims) -> int:
    return int(load_library().dsv_sparse_attn_fwd_workspace(ctypes.byref(dims)))


def dsv_sparse_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: Optional[torch.Tensor], block: int = 64,
                        scale: Optional[float] = None, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                        workspace: Optional[torch.Tensor] = None):
    """(O bf16 [B,H,N,d], LSE fp32 [B,H,N]) of softmax attention over the selected keys.  Without a
    workspace argument the workspace the library asks for (for key passes) is allocated here."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 4)
    B, H, N, d = q.shape
    if idx is None:   # every key selected (k = N): the dense path, which reads no idx
        kk = N
    else:
        _need(idx, "idx", torch.int32, 4)
        kk = idx.shape[3]
    dims = make_dims(B, H, N, d, 0, kk, block, scale)
    if out is None:
        o = torch.empty_like(q)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
    lib = load_library()
    if workspace is None:
        nbytes = int(lib.dsv_sparse_attn_fwd_workspace(ctypes.byref(dims)))
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
    _check(lib.dsv_sparse_attn_fwd(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(o), _ptr(lse),
                                   _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream_ptr(q)),
           "dsv_sparse_attn_fwd")
    return o, lse


def dsv_sparse_attn_bwd_workspace(dims: Dims, minimum: bool = False) -> int:
    lib = load_library()
    f = lib.dsv_sparse_attn_bwd_workspace_min if minimum else lib.dsv_sparse_attn_bwd_workspace
    return int(f(ctypes.byref(dims)))


def dsv_sparse_attn_bwd(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                        lse: torch.Tensor, idx: Optional[torch.Tensor], block: int = 64, scale: Optional[float] = None,
                        workspace: Optional[torch.Tensor] = None, out=None):
    """(dQ, dK, dV) bf16 [B,H,N,d]; dK/dV reduced deterministically per key."""
    for t, n in ((do, "do"), (q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, n, torch.bfloat16, 4)
    _need(lse, "lse", torch.float32, 3)
    B, H, N, d = q.shape
    if idx is None:   # every key selected (k = N): the dense backward, which reads no idx
        kk = N
    else:
        _need(idx, "idx", torch.int32, 4)
        kk = idx.shape[3]
    dims = make_dims(B, H, N, d, 0, kk, block, scale)
    lib = load_library()
    if workspace is None:
        nbytes = int(lib.dsv_sparse_attn_bwd_workspace(ctypes.byref(dims)))
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    else:
        dq, dk, dv = out
    _check(lib.dsv_sparse_attn_bwd(ctypes.byref(dims), _ptr(do), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                   _ptr(idx), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel(),
                                   _stream_ptr(q)), "dsv_sparse_attn_bwd")
    return dq, dk, dv


def dsv_sparse_attn_bwd_prepare(idx: torch.Tensor, d: int, workspace: torch.Tensor, block: int = 64) -> None:
    """First half of a split backward: the key-major rank structure of idx, written into `workspace`
    (which must hold every head in one wave: dsv_sparse_attn_bwd_workspace).  Reads idx only, so it
    may run on another stream beside the forward; order dsv_sparse_attn_bwd_prepared after it."""
    _need(idx, "idx", torch.int32, 4)
    B, H, NB, kk = idx.shape
    dims = make_dims(B, H, NB * block, d, 0, kk, block)
    _check(load_library().dsv_sparse_attn_bwd_prepare(ctypes.byref(dims), _ptr(idx), _ptr(workspace),
                                                      workspace.numel(), _stream_ptr(idx)),
           "dsv_sparse_attn_bwd_prepare")


def dsv_sparse_attn_bwd_prepared(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                 o: torch.Tensor, lse: torch.Tensor, idx: torch.Tensor, workspace: torch.Tensor,
                                 block: int = 64, scale: Optional[float] = None, out=None):
    """Second half of a split backward, on the workspace dsv_sparse_attn_bwd_prepare filled: the same
    (dQ, dK, dV) as dsv_sparse_attn_bwd, bit for bit."""
    for t, n in ((do, "do"), (q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, n, torch.bfloat16, 4)
    _need(lse, "lse", torch.float32, 3)
    _need(idx, "idx", torch.int32, 4)
    B, H, N, d = q.shape
    dims = make_dims(B, H, N, d, 0, idx.shape[3], block, scale)
    if out is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    else:
        dq, dk, dv = out
    _check(load_library().dsv_sparse_attn_bwd_prepared(ctypes.byref(dims), _ptr(do), _ptr(q), _ptr(k), _ptr(v),
                                                       _ptr(o), _ptr(lse), _ptr(idx), _ptr(dq), _ptr(dk), _ptr(dv),
                                                       _ptr(workspace), workspace.numel(), _stream_ptr(q)),
           "dsv_sparse_attn_bwd_prepared")
    return dq, dk, dv


def dsv_csr_launch_order(rowptr: torch.Tensor, B: int, H: int, N: int, block: int = 64) -> torch.Tensor:
    """int32 [B*H*N/block]: the CSR rows by descending number of 128-key chunks."""
    _need(rowptr, "rowptr", torch.int64, 1)
    dims = make_dims(B, H, N, 0, 16, max(N, 1), block)
    order = torch.empty((B * H * (N // block),), dtype=torch.int32, device=rowptr.device)
    _check(load_library().dsv_csr_launch_order(ctypes.byref(dims), _ptr(rowptr), _ptr(order), _stream_ptr(rowptr)),
           "dsv_csr_launch_order")
    return order


def dsv_sparse_attn_fwd_csr(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rowptr: torch.Tensor, cols: torch.Tensor,
                            block: int = 64, scale: Optional[float] = None,
                            out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, order: Optional[torch.Tensor] = None):
    """(O, LSE) of attention where query block i attends to cols[rowptr[i]:rowptr[i+1]]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 4)
    _need(rowptr, "rowptr", torch.int64, 1)
    _need(cols, "cols", torch.int32, 1)
    B, H, N, d = q.shape
    dims = make_dims(B, H, N, d, 0, max(N, 1), block, scale)
    if out is None:
        o = torch.empty_like(q)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
    _check(load_library().dsv_sparse_attn_fwd_csr(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(rowptr),
                                                  _ptr(cols), _ptr(order), _ptr(o), _ptr(lse), _stream_ptr(q)),
           "dsv_sparse_attn_fwd_csr")
    return o, lse


def dsv_sparse_attn_bwd_csr_workspace(dims: Dims, total_pairs: int) -> int:
    return int(load_library().dsv_sparse_attn_bwd_csr_workspace(ctypes.byref(dims), int(total_pairs)))


def dsv_sparse_attn_bwd_csr(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                            lse: torch.Tensor, rowptr: torch.Tensor, cols: torch.Tensor, block: int = 64,
                            scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None, out=None,
                            order: Optional[torch.Tensor] = None):
    """(dQ, dK, dV) for the CSR attention above (one wave; total pairs = cols.numel())."""
    for t, n in ((do, "do"), (q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, n, torch.bfloat16, 4)
    _need(lse, "lse", torch.float32, 3)
    _need(rowptr, "rowptr", torch.int64, 1)
    _need(cols, "cols", torch.int32, 1)
    B, H, N, d = q.shape
    dims = make_dims(B, H, N, d, 0, max(N, 1), block, scale)
    pairs = cols.numel()
    lib = load_library()
    if workspace is None:
        nbytes = int(lib.dsv_sparse_attn_bwd_csr_workspace(ctypes.byref(dims), pairs))
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    else:
        dq, dk, dv = out
    _check(lib.dsv_sparse_attn_bwd_csr(ctypes.byref(dims), _ptr(do), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                       _ptr(rowptr), _ptr(cols), _ptr(order), pairs, _ptr(dq), _ptr(dk), _ptr(dv),
                                       _ptr(workspace),
                                       workspace.numel(), _stream_ptr(q)), "dsv_sparse_attn_bwd_csr")
    return dq, dk, dv


# ---------------------------------------------------------------- fused AdaLN

def _adaln_dims(x: torch.Tensor, eps: float) -> AdalnDims:
    B, N, D = x.shape
    return AdalnDims(int(B), int(N), int(D), float(eps))


def _need_mod(t: torch.Tensor, name: str, x: torch.Tensor):
    _need(t, name, torch.bfloat16, 2)
    if t.shape != (x.shape[0], x.shape[2]):
        raise ValueError(f"{name} must be [B, D] = {(x.shape[0], x.shape[2])}, got {tuple(t.shape)}")


def dsv_adaln_fwd(x: torch.Tensor, scale: torch.Tensor, shift: torch.Tensor, eps: float = 1e-6,
                  y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [B, N, D] bf16 = LayerNorm(x) * (1 + scale[b]) + shift[b] (see include/dsv.h)."""
    _need(x, "x", torch.bfloat16, 3)
    _need_mod(scale, "scale", x)
    _need_mod(shift, "shift", x)
    if y is None:
        y = torch.empty_like(x)
    dims = _adaln_dims(x, eps)
    _check(load_library().dsv_adaln_fwd(ctypes.byref(dims), _ptr(x), _ptr(scale), _ptr(shift), _ptr(y),
                                        _stream_ptr(x)), "dsv_adaln_fwd")
    return y


def dsv_adaln_bwd_workspace(B: int, N: int, D: int, eps: float = 1e-6) -> int:
    dims = AdalnDims(int(B), int(N), int(D), float(eps))
    return int(load_library().dsv_adaln_bwd_workspace(ctypes.byref(dims)))


def dsv_adaln_bwd(x: torch.Tensor, scale: torch.Tensor, dy: torch.Tensor, eps: float = 1e-6,
                  out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None,
                  workspace: Optional[torch.Tensor] = None):
    """(dx bf16 [B, N, D], d_scale fp32 [B, D], d_shift fp32 [B, D]) for the loss gradient dy."""
    _need(x, "x", torch.bfloat16, 3)
    _need(dy, "dy", torch.bfloat16, 3)
    _need_mod(scale, "scale", x)
    if dy.shape != x.shape:
        raise ValueError("dy must have the shape of x")
    B, N, D = x.shape
    if out is None:
        out = (torch.empty_like(x), torch.empty((B, D), dtype=torch.float32, device=x.device),
               torch.empty((B, D), dtype=torch.float32, device=x.device))
    dx, d_scale, d_shift = out
    dims = _adaln_dims(x, eps)
    lib = load_library()
    need = int(lib.dsv_adaln_bwd_workspace(ctypes.byref(dims)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check(lib.dsv_adaln_bwd(ctypes.byref(dims), _ptr(x), _ptr(scale), _ptr(dy), _ptr(dx), _ptr(d_scale),
                             _ptr(d_shift), _ptr(workspace), workspace.numel(), _stream_ptr(x)), "dsv_adaln_bwd")
    return dx, d_scale, d_shift


# ---------------------------------------------------------------- rotary positions, qk norm
# The calls below take tens of microseconds on the GPU at most sizes, so their host side is kept lean:
# what depends on sizes alone (the dims struct, workspace sizes) is made once per size, and each output
# is its own allocation (three cost 4.5 us, one allocation and its unbinding 8.7).

_PAIRINGS = {"interleaved": 0, "halves": 1}


class RopeTable(NamedTuple):
    """(cos, sin) of every axis' positions, as the rotation calls read them (layout in include/dsv.h).

    data: fp32, flat, on the GPU; axes: rotated features of (time, height, width); lengths: positions of
    each axis; pairing: "interleaved" (features 2j, 2j+1 turn together) or "halves" (j, j + R/2)."""
    data: torch.Tensor
    axes: Tuple[int, int, int]
    lengths: Tuple[int, int, int]
    pairing: str = "interleaved"


@functools.lru_cache(maxsize=256)
def _rope_dims(shape: Tuple[int, ...], axes: Tuple, lengths: Tuple, pairing: str, pos_batched: bool, eps: float):
    """(dims struct, numbers its table holds) for tensors of `shape`."""
    B, H, N, d = shape
    if len(axes) != 3 or len(lengths) != 3:
        raise ValueError("axes and lengths need three entries (time, height, width)")
    if pairing not in _PAIRINGS:
        raise ValueError(f"pairing must be one of {sorted(_PAIRINGS)}, got {pairing!r}")
    dims = RopeDims(B, H, N, d, (ctypes.c_int64 * 3)(*axes), (ctypes.c_int64 * 3)(*lengths), _PAIRINGS[pairing],
                    int(pos_batched), eps)
    return dims, 2 * sum((r // 2) * n for r, n in zip(axes, lengths))


# strides as the calls take them (read only, and the same for every call on one layout)
@functools.lru_cache(maxsize=256)
def _view_strides(strides: Tuple[int, ...]) -> ViewStrides:
    return ViewStrides(*strides)


@functools.lru_cache(maxsize=256)
def _strides6(strides: Tuple[int, ...]):
    return _Strides6(*strides)


@functools.lru_cache(maxsize=256)
def _strides9(strides: Tuple[int, ...]):
    return _Strides9(*strides)


@functools.lru_cache(maxsize=256)
def _qk_norm_rope_ws(B: int, H: int, N: int, d: int) -> int:
    return int(load_library().dsv_qk_norm_rope_bwd_workspace(ctypes.byref(RopeDims(B, H, N, d))))


def _need_view(t: torch.Tensor, name: str, shape=None, device: Optional[int] = None):
    """The strides of a bf16 CUDA [B, H, N, d] view whose features are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    strides = t.stride()
    if t.dtype is torch.bfloat16 and len(strides) == 4 and strides[3] == 1 and t.is_cuda and \
            (shape is None or (t.shape == shape and t.get_device() == device)):
        return strides[:3]
    raise ValueError(f"{name}: need a CUDA bfloat16 [B, H, N, d] tensor with contiguous features"
                     + ("" if shape is None else f" of shape {tuple(shape)} on cuda:{device}")
                     + f", got {t.dtype} {tuple(t.shape)} strides={strides} device={t.device}")


def _need_on(dtype, shape, device: int, *named):
    """Contiguous CUDA tensors of this type and shape on this device: (tensor, name) pairs.  None is passed over: the
    library refuses it where the tensor is needed."""
    for t, name in named:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
            raise ValueError(f"{name}: need a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{device}, got "
                             f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()} device={t.device}")


def _workspace(workspace: Optional[torch.Tensor], nbytes: int, like: torch.Tensor):
    """(pointer, bytes, the tensor) of the caller's workspace, or of a new one of nbytes."""
    if workspace is None:
        if not nbytes:
            return None, 0, None
        workspace = torch.empty((nbytes,), dtype=torch.uint8, device=like.device)
    elif not workspace.is_contiguous() or workspace.get_device() != like.get_device():
        raise ValueError(f"workspace: need a contiguous tensor on {like.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _rope_args(x: torch.Tensor, pos: Optional[torch.Tensor], rope: Optional[RopeTable], eps: float):
    """(dims struct, pos pointer, table pointer) for x [B, H, N, d]."""
    shape = x.shape
    if rope is None:
        if pos is not None:
            raise ValueError("pos without a RopeTable")
        return _rope_dims(shape, (0, 0, 0), (0, 0, 0), "interleaved", False, float(eps))[0], None, None
    device = x.get_device()
    if pos is None:
        raise ValueError("a RopeTable needs pos")
    if not isinstance(pos, torch.Tensor):
        raise TypeError("pos must be a torch.Tensor")
    batched = pos.dim() == 3
    dims, numbers = _rope_dims(shape, tuple(rope.axes), tuple(rope.lengths), rope.pairing, batched, float(eps))
    _need_on(torch.int32, (shape[0], shape[2], 3) if batched else (shape[2], 3), device, (pos, "pos"))
    table = rope.data
    if table.dtype != torch.float32 or table.numel() < numbers or not table.is_contiguous() or \
            table.get_device() != device:
        raise ValueError(f"rope.data: need a contiguous float32 tensor of {numbers} numbers on {x.device}, got "
                         f"{table.dtype} {tuple(table.shape)} on {table.device}")
    return dims, pos.data_ptr(), table.data_ptr()


def _call(name: str, device: int, *args):
    """One library call on this device's current stream, with the device made current for it."""
    f = getattr(load_library(), name)
    if torch._C._cuda_getDevice() == device:
        status = f(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            status = f(*args, torch._C._cuda_getCurrentRawStream(device))
    if status != DSV_OK:
        _check(status, name)


def dsv_rope3d_table(axes: Sequence[int], lengths: Sequence[int], theta: Union[float, Sequence[float]] = 10000.0,
                     pairing: str = "interleaved", device: Union[str, torch.device] = "cuda") -> RopeTable:
    """The (cos, sin) table of positions 0 .. lengths[a] - 1 of each axis: pair i of axis a turns by
    p * theta_a^(-2 i / axes[a]) at position p (angles in fp64).  Made once per model."""
    axes, lengths = tuple(int(r) for r in axes), tuple(int(n) for n in lengths)
    dims, numbers = _rope_dims((1, 1, 1, 64 if sum(axes) <= 64 else 128), axes, lengths, pairing, False, 0.0)
    theta = (float(theta),) * 3 if isinstance(theta, (int, float)) else tuple(float(t) for t in theta)
    if len(theta) != 3:
        raise ValueError("theta must be one number or three (time, height, width)")
    data = torch.empty((max(numbers, 0),), dtype=torch.float32, device=device)
    if not data.is_cuda:
        raise ValueError(f"the table lives on a CUDA device, got {data.device}")
    _call("dsv_rope3d_table", data.get_device(), dims, (ctypes.c_double * 3)(*theta), data.data_ptr())
    return RopeTable(data, axes, lengths, pairing)


def _rope3d(fn: str, name: str, x: torch.Tensor, pos: torch.Tensor, rope: RopeTable, out: Optional[torch.Tensor]):
    xs = _view_strides(_need_view(x, name))
    if rope is None:
        raise ValueError("need a RopeTable")
    dims, pos_ptr, table_ptr = _rope_args(x, pos, rope, 0.0)
    device, os_ = x.get_device(), None
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        os_ = _view_strides(_need_view(out, "out", x.shape, device))
    _call(fn, device, dims, x.data_ptr(), xs, pos_ptr, table_ptr, out.data_ptr(), os_)
    return out


def dsv_rope3d_fwd(x: torch.Tensor, pos: torch.Tensor, rope: RopeTable,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [B, H, N, d] (any view with contiguous features) rotated at pos [N, 3] or [B, N, 3] (int32
    (t, h, w) of each token); `out` defaults to a contiguous tensor and may be x itself (in place)."""
    return _rope3d("dsv_rope3d_fwd", "x", x, pos, rope, out)


def dsv_rope3d_bwd(dy: torch.Tensor, pos: torch.Tensor, rope: RopeTable,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dx of dsv_rope3d_fwd for the loss gradient dy: the rotation by the negative angles."""
    return _rope3d("dsv_rope3d_bwd", "dy", dy, pos, rope, out)


def dsv_qk_norm_rope_fwd(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor], wq: Optional[torch.Tensor],
                         wk: Optional[torch.Tensor], pos: Optional[torch.Tensor], rope: Optional[RopeTable],
                         eps: float = 1e-6, out: Optional[Tuple] = None):
    """(q, k, v) contiguous [B, H, N, d] for the attention calls: q and k RMS-normed for each head, times
    wq / wk [d] (None: ones), rotated at pos; v copied (None: not part of the call).  The inputs are
    [B, H, N, d] views with contiguous features, e.g. the three slices of a packed projection
    [B, N, 3, H, d].  rope = pos = None: the norm alone.  out: the three outputs (v's None without v)."""
    strides = _need_view(q, "q")
    shape, device = q.shape, q.get_device()
    strides += _need_view(k, "k", shape, device)
    strides += (0, 0, 0) if v is None else _need_view(v, "v", shape, device)
    dims, pos_ptr, table_ptr = _rope_args(q, pos, rope, eps)
    _need_on(torch.bfloat16, shape[3:], device, (wq, "wq"), (wk, "wk"))
    if out is None:
        qo, ko = torch.empty(shape, dtype=q.dtype, device=q.device), torch.empty(shape, dtype=q.dtype, device=q.device)
        vo = None if v is None else torch.empty(shape, dtype=q.dtype, device=q.device)
    else:
        qo, ko, vo = out
        _need_on(torch.bfloat16, shape, device, (qo, "q_out"), (ko, "k_out"), (vo, "v_out"))
    _call("dsv_qk_norm_rope_fwd", device, dims, q.data_ptr(), k.data_ptr(), _ptr(v), _strides9(strides), _ptr(wq),
          _ptr(wk), pos_ptr, table_ptr, _ptr(qo), _ptr(ko), _ptr(vo))
    return qo, ko, vo


def dsv_qk_norm_rope_bwd_workspace(B: int, H: int, N: int, d: int) -> int:
    return _qk_norm_rope_ws(int(B), int(H), int(N), int(d))


def dsv_qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, dv_out: Optional[torch.Tensor], q: torch.Tensor,
                         k: torch.Tensor, wq: Optional[torch.Tensor], wk: Optional[torch.Tensor],
                         pos: Optional[torch.Tensor], rope: Optional[RopeTable], eps: float = 1e-6,
                         out: Optional[Tuple] = None, workspace: Optional[torch.Tensor] = None):
    """(dq, dk, dv, dwq, dwk) of dsv_qk_norm_rope_fwd: dq, dk, dv bf16 [B, H, N, d] (by default views of
    one packed [B, N, 3, H, d] gradient; `out` takes any three views with contiguous features), dwq, dwk
    fp32 [d] (None where the weight is None).  q, k are the forward's inputs; dv_out = None: no values
    (dv is None)."""
    strides = _need_view(q, "q")
    shape, device = q.shape, q.get_device()
    strides += _need_view(k, "k", shape, device)
    _need_on(torch.bfloat16, shape, device, (dq_out, "dq_out"), (dk_out, "dk_out"), (dv_out, "dv_out"))
    dims, pos_ptr, table_ptr = _rope_args(q, pos, rope, eps)
    _need_on(torch.bfloat16, shape[3:], device, (wq, "wq"), (wk, "wk"))
    B, H, N, d = shape
    if out is None:
        nt = 2 if dv_out is None else 3
        packed = torch.empty((B, N, nt, H, d), dtype=q.dtype, device=q.device)
        strides1 = (N * nt * H * d, d, nt * H * d)
        dq, dk = packed.as_strided(shape, (*strides1, 1), 0), packed.as_strided(shape, (*strides1, 1), H * d)
        dv = None if dv_out is None else packed.as_strided(shape, (*strides1, 1), 2 * H * d)
        dstrides = strides1 * 3
    else:
        dq, dk, dv = out
        dstrides = _need_view(dq, "dq", shape, device) + _need_view(dk, "dk", shape, device)
        dstrides += (0, 0, 0) if dv is None else _need_view(dv, "dv", shape, device)
    dwq = None if wq is None else torch.empty((d,), dtype=torch.float32, device=q.device)
    dwk = None if wk is None else torch.empty((d,), dtype=torch.float32, device=q.device)
    ws, nbytes, _keep = _workspace(workspace, 0 if wq is None and wk is None else _qk_norm_rope_ws(B, H, N, d), q)
    _call("dsv_qk_norm_rope_bwd", device, dims, _ptr(dq_out), _ptr(dk_out), _ptr(dv_out), q.data_ptr(),
          k.data_ptr(), _strides6(strides), _ptr(wq), _ptr(wk), pos_ptr, table_ptr, _ptr(dq), _ptr(dk), _ptr(dv),
          _strides9(dstrides), _ptr(dwq), _ptr(dwk), ws, nbytes)
    return dq, dk, dv, dwq, dwk


# ---------------------------------------------------------------- gated feed-forward

_ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}


@functools.lru_cache(maxsize=256)
def _ffn_dims(M: int, D: int, F: int, act: str):
    """(dims struct, workspace bytes of the forward, of the backward)."""
    if act not in _ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(_ACTIVATIONS)}, got {act!r}")
    dims = FfnDims(M, D, F, _ACTIVATIONS[act])
    lib = load_library()
    return dims, int(lib.dsv_ffn_gated_fwd_workspace(dims)), int(lib.dsv_ffn_gated_bwd_workspace(dims))


def _ffn_args(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act: str):
    """((dims struct, workspace bytes of the forward, of the backward), h's shape) after the checks of the inputs."""
    for t, n in ((x, "x"), (w_gate, "w_gate")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
    if x.dtype is not torch.bfloat16 or x.dim() < 2 or not x.is_contiguous() or not x.is_cuda:
        raise ValueError(f"x: need a contiguous CUDA bfloat16 [..., D] tensor with at least 2 dims, got {x.dtype} "
                         f"{tuple(x.shape)} contiguous={x.is_contiguous()} device={x.device}")
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate must be [F, D], got {tuple(w_gate.shape)}")
    D, F, device = x.shape[-1], w_gate.shape[0], x.get_device()
    _need_on(torch.bfloat16, (F, D), device, (w_gate, "w_gate"), (w_up, "w_up"))
    return _ffn_dims(x.numel() // D if D else 0, D, F, act), (*x.shape[:-1], F)


def dsv_ffn_gated_fwd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act: str = "silu",
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h [..., F] = act(x w_gate^T) * (x w_up^T) for x bf16 [..., D] and weights bf16 [F, D]
    (act: "silu" or "gelu_tanh"; see include/dsv.h)."""
    (dims, nbytes, _), shape = _ffn_args(x, w_gate, w_up, act)
    device = x.get_device()
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    else:
        _need_on(torch.bfloat16, shape, device, (out, "out"))
    ws, nbytes, _keep = _workspace(workspace, nbytes, x)
    _call("dsv_ffn_gated_fwd", device, dims, x.data_ptr(), w_gate.data_ptr(), _ptr(w_up), out.data_ptr(), ws, nbytes)
    return out


def dsv_ffn_gated_fwd_workspace(M: int, D: int, F: int) -> int:
    return _ffn_dims(int(M), int(D), int(F), "silu")[1]


def dsv_ffn_gated_bwd_workspace(M: int, D: int, F: int) -> int:
    return _ffn_dims(int(M), int(D), int(F), "silu")[2]


def dsv_ffn_gated_bwd(dh: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act: str = "silu",
                      out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None,
                      workspace: Optional[torch.Tensor] = None):
    """(dx [..., D], dw_gate [F, D], dw_up [F, D]), all bf16, for the loss gradient dh [..., F]; g and u are
    recomputed from x (the forward keeps nothing)."""
    (dims, _, nbytes), shape = _ffn_args(x, w_gate, w_up, act)
    device = x.get_device()
    _need_on(torch.bfloat16, shape, device, (dh, "dh"))
    if out is None:
        dx, dwg, dwu = torch.empty_like(x), torch.empty_like(w_gate), torch.empty_like(w_gate)
    else:
        dx, dwg, dwu = out
        _need_on(torch.bfloat16, x.shape, device, (dx, "dx"))
        _need_on(torch.bfloat16, w_gate.shape, device, (dwg, "dw_gate"), (dwu, "dw_up"))
    ws, nbytes, _keep = _workspace(workspace, nbytes, x)
    _call("dsv_ffn_gated_bwd", device, dims, _ptr(dh), x.data_ptr(), w_gate.data_ptr(), _ptr(w_up), _ptr(dx), _ptr(dwg),
          _ptr(dwu), ws, nbytes)
    return dx, dwg, dwu


def dsv_last_device_status(device: Optional[torch.device] = None) -> int:
    stream = torch.cuda.current_stream(device).cuda_stream
    return int(load_library().dsv_last_device_status(stream))


def dsv_profile_enable(on: bool = True) -> None:
    _check(load_library().dsv_profile_enable(1 if on else 0), "dsv_profile_enable")


def dsv_profile_read() -> dict:
    """{kernel name: (launches, total device ms)} since the previous read."""
    lib = load_library()
    need = int(lib.dsv_profile_read(None, 0))
    buf = ctypes.create_string_buffer(max(need, 1) + 4096)
    lib.dsv_profile_read(buf, len(buf))
    out = {}
    for line in buf.value.decode().splitlines():
        name, n, ms = line.split()
        out[name] = (int(n), float(ms))
    return out
