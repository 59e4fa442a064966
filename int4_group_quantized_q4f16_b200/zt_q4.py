"""Thin ctypes binding of ``libzt_q4.so`` (declared in ``include/zt_q4.h``).

Argument marshalling only: torch supplies device memory and the current CUDA
stream; every step of the computation runs in the library's kernels.  Importing
this module loads the library and fails loudly when it is missing -- there is
no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
# ZT_Q4_LIB names another build of the same library to load instead, e.g. the
# bounds-checked libzt_q4_checked.so beside this file
LIB_PATH = os.environ.get("ZT_Q4_LIB") or os.path.join(_PKG, "libzt_q4.so")
CHECKED_LIB_PATH = os.path.join(_PKG, "libzt_q4_checked.so")
ZT_Q4_ERR_BOUNDS = 2

ZT_OK = 0
ZT_ERR_INVALID_ARG = -1
ZT_ERR_MISALIGNED = -2
ZT_ERR_WORKSPACE = -3
ZT_ERR_LAUNCH = -4
ZT_ERR_UNSUPPORTED = -5
ZT_ERR_DEVICE = -6

_P = ctypes.c_void_p
_I = ctypes.c_int


class ZtError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        cuda = lib.zt_q4_last_cuda_error().decode() if status in (ZT_ERR_LAUNCH, ZT_ERR_DEVICE) else ""
        super().__init__(f"{what}: status {status}: {strerror(status)}" + (f" [{cuda}]" if cuda else ""))


ZT_Q4_GEMV = 0
ZT_Q4_GATE_UP_SILU = 1
ZT_Q4_LM_HEAD = 2
ZT_Q4_PASS_MAX = 192


class ZtNorm(ctypes.Structure):
    """struct zt_q4_norm of include/zt_q4.h (residual add + RMSNorm prologue)"""
    _fields_ = [("residual", ctypes.c_void_p), ("delta", ctypes.c_void_p), ("gamma", ctypes.c_void_p),
                ("residual_out", ctypes.c_void_p), ("x_out", ctypes.c_void_p), ("eps", ctypes.c_float)]


class ZtRope(ctypes.Structure):
    """struct zt_q4_rope of include/zt_q4.h (rotary position embedding epilogue)"""
    _fields_ = [("pos", ctypes.c_void_p), ("head_dim", ctypes.c_int), ("theta", ctypes.c_float)]


class ZtProj(ctypes.Structure):
    """struct zt_q4_proj of include/zt_q4.h"""
    _fields_ = [("qw", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("argmax", ctypes.c_void_p), ("kind", ctypes.c_int),
                ("N", ctypes.c_int), ("K", ctypes.c_int), ("wait", ctypes.c_int), ("ld_out", ctypes.c_int),
                ("group", ctypes.c_int), ("norm", ctypes.POINTER(ZtNorm)), ("rope", ctypes.POINTER(ZtRope))]


class ZtKv(ctypes.Structure):
    """struct zt_q4_kv of include/zt_q4.h (a paged 4-bit KV cache)"""
    _fields_ = [("pages", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("err", ctypes.c_void_p)]


class ZtKvRows(ctypes.Structure):
    """struct zt_q4_kv_rows of include/zt_q4.h (places of appended or gathered rows)"""
    _fields_ = [("seq", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("n", ctypes.c_int),
                ("page_table", ctypes.c_void_p), ("n_seqs", ctypes.c_int), ("max_pages", ctypes.c_int)]


class ZtKvRope(ctypes.Structure):
    """struct zt_q4_kv_rope of include/zt_q4.h (rotary embedding of an append)"""
    _fields_ = [("theta", ctypes.c_float), ("q", ctypes.c_void_p), ("ld_q", ctypes.c_int), ("q_heads", ctypes.c_int),
                ("q_out", ctypes.c_void_p), ("ld_q_out", ctypes.c_int), ("k_out", ctypes.c_void_p),
                ("ld_k_out", ctypes.c_int)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m int4_group_quantized_q4f16_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.zt_q4_gemv.argtypes = [_P, _P, _P, _P, _I, _I, _I, _P]
    lib.zt_q4_gate_up_silu.argtypes = [_P, _P, _P, _P, _I, _I, _I, _P]
    lib.zt_q4_lmhead_workspace_bytes.argtypes = [_I, _I, _I]
    lib.zt_q4_lmhead_workspace_bytes.restype = ctypes.c_size_t
    lib.zt_q4_lmhead_argmax.argtypes = [_P, _P, _P, _P, _P, _P, ctypes.c_size_t, _I, _I, _I, _P]
    lib.zt_q4_lmhead_argmax_noalloc.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _P]
    lib.zt_q4_lmhead_argmax_noalloc.restype = ctypes.c_int
    lib.zt_q4_pass_workspace_bytes.argtypes = [ctypes.POINTER(ZtProj), _I, _I]
    lib.zt_q4_pass_workspace_bytes.restype = ctypes.c_size_t
    lib.zt_q4_pass.argtypes = [ctypes.POINTER(ZtProj), _I, _I, _P, ctypes.c_size_t, _P]
    lib.zt_q4_pass.restype = ctypes.c_int
    lib.zt_q4_pass_errors.argtypes = [_P, _I, ctypes.POINTER(ctypes.c_uint)]
    lib.zt_q4_pass_plan.argtypes = [_I, _I, _I] + [ctypes.POINTER(_I)] * 5
    lib.zt_q4_pass_plan.restype = ctypes.c_int
    lib.zt_q4_pass_test_withhold.argtypes = [ctypes.POINTER(ZtProj), _I, _I, _P, ctypes.c_size_t, _P]
    lib.zt_q4_pass_test_withhold.restype = ctypes.c_int
    lib.zt_q4_pass_test_cut.argtypes = [ctypes.POINTER(ZtProj), _I, _I, _P, ctypes.c_size_t, _P, _I]
    lib.zt_q4_pass_test_cut.restype = ctypes.c_int
    lib.zt_q4_build_flags.argtypes = []
    lib.zt_q4_build_flags.restype = ctypes.c_int
    lib.zt_q4_pass_errors.restype = ctypes.c_int
    lib.zt_q4_dequant_f16.argtypes = [_P, _P, _P, _I, _I, _I, _P]
    lib.zt_q4_gemm_f16w.argtypes = [_P, _P, _P, _I, _I, _I, _P, ctypes.c_size_t, _P]
    lib.zt_q4_gemm_f16w_workspace_bytes.argtypes = [_I, _I, _I]
    lib.zt_q4_gemm_f16w_workspace_bytes.restype = ctypes.c_size_t
    lib.zt_q4_gemm_f16w_errors.argtypes = [_P, ctypes.POINTER(ctypes.c_uint)]
    lib.zt_q4_gemm_workspace_bytes.argtypes = [_I, _I, _I]
    lib.zt_q4_gemm_workspace_bytes.restype = ctypes.c_size_t
    lib.zt_q4_gemm.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _P, ctypes.c_size_t, _P]
    lib.zt_q4_gemm_errors.argtypes = [_P, _I, _I, ctypes.POINTER(ctypes.c_uint)]
    lib.zt_q4_gemm_gate_up_workspace_bytes.argtypes = [_I, _I, _I]
    lib.zt_q4_gemm_gate_up_workspace_bytes.restype = ctypes.c_size_t
    lib.zt_q4_gemm_gate_up_silu.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _P, ctypes.c_size_t, _P]
    lib.zt_q4_gemm_f16w_gate_up_silu.argtypes = [_P, _P, _P, _I, _I, _I, _P, ctypes.c_size_t, _P]
    for f in (lib.zt_q4_dequant_f16, lib.zt_q4_gemm_f16w, lib.zt_q4_gemm, lib.zt_q4_gemm_errors,
              lib.zt_q4_gemm_f16w_errors, lib.zt_q4_gemm_gate_up_silu, lib.zt_q4_gemm_f16w_gate_up_silu):
        f.restype = ctypes.c_int
    lib.zt_q4_pack_host.argtypes = [_P, _I, _I, _P]
    lib.zt_q4_unpack_host.argtypes = [_P, _I, _I, _P]
    lib.zt_q4_strerror.argtypes = [_I]
    lib.zt_q4_strerror.restype = ctypes.c_char_p
    lib.zt_q4_version.argtypes = []
    lib.zt_q4_last_cuda_error.argtypes = []
    lib.zt_q4_last_cuda_error.restype = ctypes.c_char_p
    lib.zt_q4_kv_page_bytes.argtypes = [_I, _I, _I]
    lib.zt_q4_kv_page_bytes.restype = ctypes.c_size_t
    lib.zt_q4_kv_append.argtypes = [ctypes.POINTER(ZtKv), ctypes.POINTER(ZtKvRows), _P, _I, _P, _I,
                                    ctypes.POINTER(ZtKvRope), _P]
    lib.zt_q4_kv_gather.argtypes = [ctypes.POINTER(ZtKv), ctypes.POINTER(ZtKvRows), _P, _I, _P, _I, _P]
    lib.zt_q4_kv_copy_pages.argtypes = [ctypes.POINTER(ZtKv), _P, _P, _I, _I, ctypes.c_size_t, _P]
    lib.zt_q4_kv_attention_workspace_bytes.argtypes = [_I, _I, _I, _I]
    lib.zt_q4_kv_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.zt_q4_kv_attention.argtypes = [ctypes.POINTER(ZtKv), _P, _I, _I, _I, _P, _P, _I, _I, ctypes.c_float, _P, _I,
                                       _P, ctypes.c_size_t, _P]
    lib.zt_q4_prompt_attention.argtypes = [_P, _I, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float,
                                           _P, _I, _P, _P]
    lib.zt_q4_prompt_attention.restype = ctypes.c_int
    lib.zt_q4_kv_errors.argtypes = [_P, ctypes.POINTER(ctypes.c_uint)]
    for f in (lib.zt_q4_kv_append, lib.zt_q4_kv_gather, lib.zt_q4_kv_copy_pages, lib.zt_q4_kv_attention,
              lib.zt_q4_kv_errors):
        f.restype = ctypes.c_int
    for f in (lib.zt_q4_gemv, lib.zt_q4_gate_up_silu, lib.zt_q4_lmhead_argmax,
              lib.zt_q4_pack_host, lib.zt_q4_unpack_host, lib.zt_q4_version):
        f.restype = ctypes.c_int
    return lib


lib = _load()


def strerror(status: int) -> str:
    return lib.zt_q4_strerror(int(status)).decode()


def version() -> Tuple[int, int]:
    v = lib.zt_q4_version()
    return v >> 16, v & 0xFFFF


def is_checked_build() -> bool:
    """True when the loaded library is the bounds-checked build (-DZT_Q4_CHECKED)."""
    return bool(lib.zt_q4_build_flags() & 1)


def _check(rc: int, what: str) -> None:
    if rc != ZT_OK:
        raise ZtError(rc, what)


# ------------------------------------------------------------ host layout --
def pack_host(q: np.ndarray) -> np.ndarray:
    """codes uint8 [N][K] (0..15) -> packed uint32 [N][K/8], low nibble first."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    N, K = q.shape
    qw = np.empty((N, K // 8), dtype=np.uint32)
    _check(lib.zt_q4_pack_host(q.ctypes.data, N, K, qw.ctypes.data), "zt_q4_pack_host")
    return qw


def unpack_host(qw: np.ndarray, K: int) -> np.ndarray:
    qw = np.ascontiguousarray(qw, dtype=np.uint32)
    N = qw.shape[0]
    q = np.empty((N, K), dtype=np.uint8)
    _check(lib.zt_q4_unpack_host(qw.ctypes.data, N, K, q.ctypes.data), "zt_q4_unpack_host")
    return q


# ---------------------------------------------------------- device calls --
def _torch():
    import torch
    return torch


def _stream_handle(stream) -> Optional[int]:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dims(qw, scales, x, rows_mult: int, group: int = 32):
    torch = _torch()
    for t, name in ((qw, "qw"), (scales, "scales"), (x, "x")):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if qw.dtype not in (torch.int32, torch.uint32):
        raise TypeError("qw must hold 32-bit words (int32 or uint32)")
    if scales.dtype != torch.float16 or x.dtype != torch.float16:
        raise TypeError("scales and x must be float16")
    x2 = x if x.dim() == 2 else x.view(1, -1)
    M, K = x2.shape
    n_rows = qw.shape[0]
    if qw.dim() != 2 or qw.shape[1] * 8 != K or K % group or scales.shape != (n_rows, K // group):
        raise ValueError(f"shape mismatch: qw {tuple(qw.shape)}, scales {tuple(scales.shape)}, x {tuple(x.shape)}")
    if n_rows % rows_mult:
        raise ValueError("gate/up weights need an even number of rows")
    return M, n_rows // rows_mult, K


def gemv(qw, scales, x, y=None, stream=None):
    """y[M][N] fp16 = dequant(qw, scales) @ x^T (torch CUDA tensors)."""
    torch = _torch()
    M, N, K = _dims(qw, scales, x, 1)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    _check(lib.zt_q4_gemv(qw.data_ptr(), scales.data_ptr(), x.data_ptr(), y.data_ptr(),
                          M, N, K, _stream_handle(stream)), "zt_q4_gemv")
    return y


def gate_up_silu(qw, scales, x, y=None, stream=None):
    """y[M][N] fp16 = SiLU(gate . x) * (up . x); qw has 2N rows, gate first."""
    torch = _torch()
    M, N, K = _dims(qw, scales, x, 2)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    _check(lib.zt_q4_gate_up_silu(qw.data_ptr(), scales.data_ptr(), x.data_ptr(), y.data_ptr(),
                                  M, N, K, _stream_handle(stream)), "zt_q4_gate_up_silu")
    return y


# ------------------------------------------------- batched prefill (M > 16) --
def _group_of(K: int, scales) -> int:
    g = K // scales.shape[1]
    if g * scales.shape[1] != K:
        raise ValueError("scales must have K / group columns")
    return g


def dequant_f16(qw, scales, w16=None, stream=None):
    """w16 fp16 [N][K] = fp16((q - 7) * s), one rounding to nearest even."""
    torch = _torch()
    N, K = qw.shape[0], qw.shape[1] * 8
    g = _group_of(K, scales)
    _dims(qw, scales, torch.empty((1, K), dtype=torch.float16, device=qw.device), 1, g)
    if w16 is None:
        w16 = torch.empty((N, K), dtype=torch.float16, device=qw.device)
    _check(lib.zt_q4_dequant_f16(qw.data_ptr(), scales.data_ptr(), w16.data_ptr(), N, K, g,
                                 _stream_handle(stream)), "zt_q4_dequant_f16")
    return w16


def gemm_f16w_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.zt_q4_gemm_f16w_workspace_bytes(M, N, K))


def gemm_f16w(w16, x, y=None, workspace=None, stream=None):
    """y fp16 [M][N] = x [M][K] @ w16^T on the tensor cores; workspace: uint8
    CUDA tensor of gemm_f16w_workspace_bytes(M, N, K) bytes (error word and
    split-K partials)."""
    torch = _torch()
    for t, name in ((w16, "w16"), (x, "x")):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.float16 or t.dim() != 2:
            raise ValueError(f"{name} must be a contiguous 2-D float16 CUDA tensor")
    (N, K), M = w16.shape, x.shape[0]
    if x.shape[1] != K:
        raise ValueError("x and w16 disagree on K")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    if workspace is None:
        workspace = torch.empty((gemm_f16w_workspace_bytes(M, N, K),), dtype=torch.uint8, device=x.device)
    _check(lib.zt_q4_gemm_f16w(w16.data_ptr(), x.data_ptr(), y.data_ptr(), M, N, K, workspace.data_ptr(),
                               workspace.numel(), _stream_handle(stream)), "zt_q4_gemm_f16w")
    return y


def gemm_f16w_errors(workspace) -> int:
    out = ctypes.c_uint(0)
    _check(lib.zt_q4_gemm_f16w_errors(workspace.data_ptr(), ctypes.byref(out)), "zt_q4_gemm_f16w_errors")
    return int(out.value)


def gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.zt_q4_gemm_workspace_bytes(M, N, K))


def gemm(qw, scales, x, y=None, workspace=None, stream=None):
    """Batched prefill: y fp16 [M][N] = x @ fp16(dequant(qw, scales))^T: the
    dequant into the workspace, then the tensor-core GEMM (and, for shapes
    split along K, the ordered sum of the partials)."""
    torch = _torch()
    N, K = qw.shape[0], qw.shape[1] * 8
    g = _group_of(K, scales)
    M, _, _ = _dims(qw, scales, x, 1, g)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    if workspace is None:
        workspace = torch.empty((gemm_workspace_bytes(M, N, K),), dtype=torch.uint8, device=x.device)
    _check(lib.zt_q4_gemm(qw.data_ptr(), scales.data_ptr(), x.data_ptr(), y.data_ptr(), M, N, K, g,
                          workspace.data_ptr(), workspace.numel(), _stream_handle(stream)), "zt_q4_gemm")
    return y


def gemm_errors(workspace, N: int, K: int) -> int:
    out = ctypes.c_uint(0)
    _check(lib.zt_q4_gemm_errors(workspace.data_ptr(), N, K, ctypes.byref(out)), "zt_q4_gemm_errors")
    return int(out.value)


def gemm_gate_up_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.zt_q4_gemm_gate_up_workspace_bytes(M, N, K))


def gemm_gate_up_silu(qw, scales, x, y=None, workspace=None, stream=None):
    """Batched fused FFN: y fp16 [M][N] = SiLU(x @ W16_gate^T) * (x @ W16_up^T),
    qw / scales with 2N rows (gate first), through the binary16 weights."""
    torch = _torch()
    two_n, K = qw.shape[0], qw.shape[1] * 8
    g = _group_of(K, scales)
    M, N, _ = _dims(qw, scales, x, 2, g)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    if workspace is None:
        workspace = torch.empty((gemm_gate_up_workspace_bytes(M, N, K),), dtype=torch.uint8, device=x.device)
    _check(lib.zt_q4_gemm_gate_up_silu(qw.data_ptr(), scales.data_ptr(), x.data_ptr(), y.data_ptr(), M, N, K, g,
                                       workspace.data_ptr(), workspace.numel(), _stream_handle(stream)),
           "zt_q4_gemm_gate_up_silu")
    return y


def gemm_f16w_gate_up_silu(w16, x, y=None, workspace=None, stream=None):
    """The fused FFN on binary16 weights w16 [2N][K] (gate rows first)."""
    torch = _torch()
    for t, name in ((w16, "w16"), (x, "x")):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.float16 or t.dim() != 2:
            raise ValueError(f"{name} must be a contiguous 2-D float16 CUDA tensor")
    (two_n, K), M = w16.shape, x.shape[0]
    if x.shape[1] != K or two_n % 2:
        raise ValueError("w16 must be [2N][K] with x [M][K]")
    N = two_n // 2
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    if workspace is None:
        workspace = torch.empty((256,), dtype=torch.uint8, device=x.device)
    _check(lib.zt_q4_gemm_f16w_gate_up_silu(w16.data_ptr(), x.data_ptr(), y.data_ptr(), M, N, K,
                                            workspace.data_ptr(), workspace.numel(), _stream_handle(stream)),
           "zt_q4_gemm_f16w_gate_up_silu")
    return y


def lmhead_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.zt_q4_lmhead_workspace_bytes(M, N, K))


def lmhead_argmax(qw, scales, x, logits=None, argmax=None, workspace=None, stream=None):
    """(logits f32 [M][N], argmax int32 [M]); workspace is a uint8 CUDA tensor."""
    torch = _torch()
    M, N, K = _dims(qw, scales, x, 1)
    if logits is None:
        logits = torch.empty((M, N), dtype=torch.float32, device=x.device)
    if argmax is None:
        argmax = torch.empty((M,), dtype=torch.int32, device=x.device)
    if workspace is None:
        workspace = torch.empty((lmhead_workspace_bytes(M, N, K),), dtype=torch.uint8, device=x.device)
    _check(lib.zt_q4_lmhead_argmax(qw.data_ptr(), scales.data_ptr(), x.data_ptr(), logits.data_ptr(),
                                   argmax.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                   M, N, K, _stream_handle(stream)), "zt_q4_lmhead_argmax")
    return logits, argmax


def lmhead_argmax_noalloc(qw, scales, x, logits=None, argmax=None, stream=None):
    """lmhead_argmax through the entry point that allocates no device memory
    (its scratch is a static array in the library; see include/zt_q4.h)."""
    torch = _torch()
    M, N, K = _dims(qw, scales, x, 1)
    if logits is None:
        logits = torch.empty((M, N), dtype=torch.float32, device=x.device)
    if argmax is None:
        argmax = torch.empty((M,), dtype=torch.int32, device=x.device)
    _check(lib.zt_q4_lmhead_argmax_noalloc(qw.data_ptr(), scales.data_ptr(), x.data_ptr(), logits.data_ptr(),
                                           argmax.data_ptr(), M, N, K, _stream_handle(stream)),
           "zt_q4_lmhead_argmax_noalloc")
    return logits, argmax


def pass_plan(M: int, K_max: int, n: int = 1) -> Tuple[int, int, int, int, int]:
    """(CTAs per SM, ring stages, k_window, column_blocks, warps per CTA) of
    the decode kernel for these shapes; k_window 0 = activations staged whole;
    column_blocks 2 = the first ceil(M/2) tokens and the rest in separate CTAs
    (no device needed)."""
    c, st, kw, cb, w = _I(0), _I(0), _I(0), _I(0), _I(0)
    _check(lib.zt_q4_pass_plan(M, K_max, n, ctypes.byref(c), ctypes.byref(st), ctypes.byref(kw), ctypes.byref(cb),
                               ctypes.byref(w)), "zt_q4_pass_plan")
    return c.value, st.value, kw.value, cb.value, w.value


class Pass:
    """A decode weight pass: a list of projections run by one persistent kernel.

    Each entry is a dict with torch CUDA tensors: kind ("gemv", "gate_up",
    "lm_head"), qw, scales, x, out (and argmax for "lm_head"), and optional
    wait (read x only after all earlier projections completed).  An optional
    "norm" dict turns on the residual add + RMSNorm prologue (x is then not
    read and may be omitted): residual, gamma, eps, and optionally delta,
    residual_out, x_out.  An optional "rope" dict (gemv only) rotates the
    output's feature pairs: pos (int32 [M] CUDA tensor), head_dim, theta.
    "ld_out" sets the output row stride (default N); "group" the k per scale
    (32, 64 or 128; scales are [rows][K / group]).  The ctypes arrays and
    the workspace are built once; run() only launches."""

    KINDS = {"gemv": ZT_Q4_GEMV, "gate_up": ZT_Q4_GATE_UP_SILU, "lm_head": ZT_Q4_LM_HEAD}

    def __init__(self, projs, workspace=None):
        torch = _torch()
        if not 1 <= len(projs) <= ZT_Q4_PASS_MAX:
            raise ValueError(f"a pass has 1..{ZT_Q4_PASS_MAX} projections")
        self._keep = projs
        arr = (ZtProj * len(projs))()
        self._norms = []
        M = None
        for i, p in enumerate(projs):
            kind = self.KINDS[p["kind"]]
            nm = p.get("norm")
            xs = p.get("x") if nm is None else nm["residual"]
            group = int(p.get("group", 32))
            m, n, k = _dims(p["qw"], p["scales"], xs, 2 if kind == ZT_Q4_GATE_UP_SILU else 1, group)
            if M is None:
                M = m
            elif m != M:
                raise ValueError("all projections of a pass share M")
            am = p.get("argmax")
            norm_ptr = None
            if nm is not None:
                def ptr(key, numel):
                    t = nm.get(key)
                    if t is None:
                        return None
                    if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.float16 or t.numel() != numel:
                        raise ValueError(f"norm {key} must be a contiguous CUDA float16 tensor of {numel} elements")
                    return t.data_ptr()
                z = ZtNorm(ptr("residual", m * k), ptr("delta", m * k), ptr("gamma", k),
                           ptr("residual_out", m * k), ptr("x_out", m * k), float(nm.get("eps", 1e-5)))
                self._norms.append(z)
                norm_ptr = ctypes.pointer(z)
            rope_ptr = None
            rp = p.get("rope")
            if rp is not None:
                pos = rp["pos"]
                if not pos.is_cuda or pos.dtype != torch.int32 or pos.numel() != m or not pos.is_contiguous():
                    raise ValueError("rope pos must be a contiguous CUDA int32 tensor with one position per token")
                z = ZtRope(pos.data_ptr(), int(rp["head_dim"]), float(rp.get("theta", 10000.0)))
                self._norms.append(z)
                rope_ptr = ctypes.pointer(z)
            x = p.get("x")
            arr[i] = ZtProj(p["qw"].data_ptr(), p["scales"].data_ptr(), x.data_ptr() if x is not None else None,
                            p["out"].data_ptr(), am.data_ptr() if am is not None else None, kind, n, k,
                            int(bool(p.get("wait", 0))), int(p.get("ld_out", 0)), group, norm_ptr, rope_ptr)
        self.arr, self.n, self.M = arr, len(projs), M
        nbytes = int(lib.zt_q4_pass_workspace_bytes(arr, self.n, M))
        if workspace is None:
            workspace = torch.empty((nbytes,), dtype=torch.uint8, device=projs[0]["out"].device)
        self.workspace = workspace

    def run(self, stream=None):
        _check(lib.zt_q4_pass(self.arr, self.n, self.M, self.workspace.data_ptr(), self.workspace.numel(),
                              _stream_handle(stream)), "zt_q4_pass")

    def run_withholding_phase0(self, stream=None):
        """Error-path test: the pass with CTA 0's phase-0 arrival withheld (see
        zt_q4_pass_test_withhold); the next phase's bounded wait runs out."""
        _check(lib.zt_q4_pass_test_withhold(self.arr, self.n, self.M, self.workspace.data_ptr(),
                                            self.workspace.numel(), _stream_handle(stream)), "zt_q4_pass_test_withhold")

    def run_with_cut_extent(self, rows: int, stream=None):
        """Checked-build test: the pass with every weight extent ``rows`` rows short (see
        zt_q4_pass_test_cut); the copies of the last rows fail their check and are skipped."""
        _check(lib.zt_q4_pass_test_cut(self.arr, self.n, self.M, self.workspace.data_ptr(),
                                       self.workspace.numel(), _stream_handle(stream), rows), "zt_q4_pass_test_cut")

    def errors(self) -> int:
        v = ctypes.c_uint(0)
        _check(lib.zt_q4_pass_errors(self.workspace.data_ptr(), self.n, ctypes.byref(v)), "zt_q4_pass_errors")
        return int(v.value)


# ----------------------------------------------- paged 4-bit KV cache --
ZT_Q4_KV_ERR_PLACE = 1
ZT_Q4_KV_ERR_WAIT = 2
ZT_Q4_KV_ERR_WORKSPACE = 4
ZT_Q4_KV_MAX_SEQS = 2048


def kv_page_bytes(page_size: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of one page of the 4-bit cache (one layer)."""
    n = int(lib.zt_q4_kv_page_bytes(page_size, kv_heads, head_dim))
    if n == 0:
        raise ValueError(f"no cache page of {page_size} tokens, {kv_heads} heads of {head_dim}: page_size is a multiple "
                         "of 16 up to 1024, head_dim 64, 96 or 128")
    return n


def kv_attention_workspace_bytes(kv_heads: int, q_heads: int, head_dim: int, tokens: int = 1) -> int:
    return int(lib.zt_q4_kv_attention_workspace_bytes(kv_heads, q_heads, head_dim, tokens))


def _on(t, device, dtype, what, dim):
    if not t.is_cuda or t.device != device or t.dtype != dtype or t.dim() != dim:
        raise ValueError(f"{what} must be a {dim}-D {dtype} CUDA tensor on {device}")


def _c_int(n, what):
    """n, which ctypes would cut off where a C int cannot hold it."""
    if n > 2**31 - 1:
        raise ValueError(f"{what} is {n}, more than a 32-bit integer holds")
    return n


def _ints(t, device, what, dim=1, numel=None):
    torch = _torch()
    _on(t, device, torch.int32, what, dim)
    if not t.is_contiguous() or (numel is not None and t.numel() != numel):
        raise ValueError(f"{what} must be contiguous" + (f" with {numel} elements" if numel is not None else ""))
    for n in t.shape:
        _c_int(n, f"a dimension of {what}")
    return t.data_ptr()


def _heads(t, device, what, rows, heads, dim):
    """(pointer, row stride) of fp16 rows [rows][heads][dim] whose heads lie side by side."""
    torch = _torch()
    _on(t, device, torch.float16, what, 3)
    if rows is None:
        rows = t.shape[0]
    if tuple(t.shape) != (rows, heads, dim):
        raise ValueError(f"{what} must be [{rows}, {heads}, {dim}], is {tuple(t.shape)}")
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim) or (rows > 1 and t.stride(0) < heads * dim):
        raise ValueError(f"the heads of a row of {what} must lie side by side, rows behind each other")
    return t.data_ptr(), _c_int(int(t.stride(0)), f"the row stride of {what}") if rows > 1 else heads * dim


def _errors(err) -> int:
    """An error word when everything launched on its device has finished (torch's streams are not ordered with the copy)."""
    v = ctypes.c_uint(0)
    _torch().cuda.synchronize(err.device)
    _check(lib.zt_q4_kv_errors(err.data_ptr(), ctypes.byref(v)), "zt_q4_kv_errors")
    return int(v.value)


class _Fill:
    """The zero-fill of buffers that this module allocated, on the stream that was current then.  The caller does not see the
    buffers, so runs on other streams are ordered behind the fill here, and the allocator is told of them: memory that is
    let go is not given to others before those runs have ended."""

    def __init__(self, device, *tensors):
        torch = _torch()
        self.tensors = tensors
        with torch.cuda.device(device):
            stream = torch.cuda.current_stream()
            self.captured = torch.cuda.is_current_stream_capturing()
            self.event = torch.cuda.Event()
            self.event.record(stream)
        # handles of the streams that come behind the fill; a captured one runs with its graph only
        self.ordered = set() if self.captured else {stream.cuda_stream}

    def order(self, stream, capturing) -> bool:
        """Makes `stream` wait for the fill; whether that holds for its later work too."""
        if stream.cuda_stream in self.ordered:
            return True
        if self.captured and not capturing:
            raise RuntimeError("a plan or cache made while a graph was captured can run in that capture only")
        for t in self.tensors:
            t.record_stream(stream)
        if capturing:
            # a fill outside the capture cannot be waited for here: torch.cuda.graph waits for the device before it begins
            if self.captured:
                stream.wait_event(self.event)
            return False
        stream.wait_event(self.event)
        self.ordered.add(stream.cuda_stream)
        return True


class _Launch:
    """A call whose arguments are checked and marshalled once; run() only launches, on the tensors' device and its
    current stream (or `stream`).  The tensors are kept alive; their contents are read at run().  A first run on another
    stream than the one that was current when the plan (or its cache) was made waits for what was filled there.  A run in a
    capture does not: begin it when that stream has been waited for (torch.cuda.graph does), and keep the plan as long as
    the graph."""

    def __init__(self, name, device, args, keep, result, fills):
        torch = _torch()
        self._fn, self._name, self._args, self._keep, self._result = getattr(lib, name), name, args, keep, result
        self._device, self._index, self._fills = device, device.index, fills
        self._ordered = set.intersection(*(f.ordered for f in fills))
        # the raw handle: building torch's Stream object takes longer than a launch
        self._current, self._raw_stream = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream

    def _order(self, handle):
        torch = _torch()
        # (an external stream of handle 0 would be another one than the default stream)
        stream = torch.cuda.ExternalStream(handle, device=self._device) if handle else torch.cuda.default_stream(self._device)
        with torch.cuda.stream(stream):
            capturing = torch.cuda.is_current_stream_capturing()
        if all([f.order(stream, capturing) for f in self._fills]):
            self._ordered.add(handle)

    def run(self, stream=None):
        if self._current() != self._index:
            with _torch().cuda.device(self._device):
                return self.run(stream)
        handle = self._raw_stream(self._index) if stream is None else _stream_handle(stream)
        if handle not in self._ordered:
            self._order(handle)
        rc = self._fn(*self._args, handle)
        if rc != ZT_OK:
            raise ZtError(rc, self._name)
        return self._result


class KvCache:
    """A paged 4-bit KV cache (layout and quantization: include/zt_q4.h) over `pages`, a uint8 CUDA tensor
    [layers, n_pages, page_bytes] (or [n_pages, page_bytes] for one layer) that the caller owns.  A device error word
    collects indices out of range; errors() reads it when the device's work has finished, clear_errors() resets it on the
    current stream."""

    def __init__(self, pages, page_size: int, kv_heads: int, head_dim: int):
        torch = _torch()
        nbytes = kv_page_bytes(page_size, kv_heads, head_dim)
        if pages.dim() == 2:
            pages = pages.unsqueeze(0)
        if not pages.is_cuda or pages.dtype != torch.uint8 or pages.dim() != 3 or not pages.is_contiguous():
            raise ValueError("pages must be a contiguous uint8 CUDA tensor [layers, n_pages, page_bytes]")
        if pages.shape[2] != nbytes or pages.shape[0] < 1 or pages.shape[1] < 1:
            raise ValueError(f"a page of {page_size} tokens has {nbytes} bytes, pages is {tuple(pages.shape)}")
        self.pages, self.device = pages, pages.device
        self.layers, self.n_pages, self.page_bytes = (int(n) for n in pages.shape)
        self.page_size, self.kv_heads, self.head_dim = page_size, kv_heads, head_dim
        self.err = torch.zeros((1,), dtype=torch.int32, device=self.device)
        self._fill = _Fill(self.device, self.err)

    @classmethod
    def empty(cls, layers: int, n_pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda"):
        """A cache on memory of its own (zeros: every place reads back as 0)."""
        torch = _torch()
        cache = cls(torch.zeros((layers, n_pages, kv_page_bytes(page_size, kv_heads, head_dim)), dtype=torch.uint8,
                                device=device), page_size, kv_heads, head_dim)
        cache._fill.tensors += (cache.pages,)
        return cache

    def _struct(self, layer: int) -> ZtKv:
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer {layer} of a cache of {self.layers}")
        return ZtKv(self.pages.data_ptr() + layer * self.n_pages * self.page_bytes, self.n_pages, self.page_size,
                    self.kv_heads, self.head_dim, self.err.data_ptr())

    def _rows(self, seq, pos, table) -> ZtKvRows:
        n = int(pos.numel())
        return ZtKvRows(_ints(seq, self.device, "seq", 1, n), _ints(pos, self.device, "pos", 1, n), n,
                        _ints(table, self.device, "table", 2), int(table.shape[0]), int(table.shape[1]))

    def errors(self) -> int:
        return _errors(self.err)

    def clear_errors(self) -> None:
        self.err.zero_()


class KvAppend(_Launch):
    """Appends rows to layer `layer` of a cache: k and v fp16 [n, kv_heads, head_dim] (rows may be strided: views into
    a QKV buffer) go to positions pos of sequences seq (int32 [n]; pos < 0 skips the row) through the page table
    int32 [n_seqs, max_pages].  With theta, k and q (fp16 [n, q_heads, head_dim], optional) are rotated first;
    run() returns (rotated q or None, rotated k), written to q_out and k_out (allocated here when not given)."""

    def __init__(self, cache: KvCache, k, v, seq, pos, table, layer: int = 0, q=None, theta=None, q_out=None, k_out=None):
        torch = _torch()
        n, dev, dim = int(pos.numel()), cache.device, cache.head_dim
        kv, rows = cache._struct(layer), cache._rows(seq, pos, table)
        kp, ld_k = _heads(k, dev, "k", n, cache.kv_heads, dim)
        vp, ld_v = _heads(v, dev, "v", n, cache.kv_heads, dim)
        rope = None
        if theta is None:
            if q is not None or q_out is not None or k_out is not None:
                raise ValueError("q, q_out and k_out belong to a rotation: give theta")
        else:
            if q is None and q_out is not None:
                raise ValueError("q_out without q")
            if k_out is None:
                k_out = torch.empty((n, cache.kv_heads, dim), dtype=torch.float16, device=dev)
            rope = ZtKvRope(float(theta))
            rope.k_out, rope.ld_k_out = _heads(k_out, dev, "k_out", n, cache.kv_heads, dim)
            if q is not None:
                rope.q_heads = int(q.shape[1]) if q.dim() == 3 else 0
                if q_out is None:
                    q_out = torch.empty((n, rope.q_heads, dim), dtype=torch.float16, device=dev)
                rope.q, rope.ld_q = _heads(q, dev, "q", n, rope.q_heads, dim)
                rope.q_out, rope.ld_q_out = _heads(q_out, dev, "q_out", n, rope.q_heads, dim)
        super().__init__("zt_q4_kv_append", dev,
                         (ctypes.byref(kv), ctypes.byref(rows), kp, ld_k, vp, ld_v,
                          ctypes.byref(rope) if rope else None),
                         (cache, k, v, seq, pos, table, q, q_out, k_out, kv, rows, rope), (q_out, k_out), (cache._fill,))


class KvGather(_Launch):
    """Reads rows of a cache back as fp16: run() returns (k, v) [n, kv_heads, head_dim], row i being position pos[i] of
    sequence seq[i] (pos < 0 leaves the row as it was)."""

    def __init__(self, cache: KvCache, seq, pos, table, layer: int = 0, k=None, v=None):
        torch = _torch()
        n, dev, dim = int(pos.numel()), cache.device, cache.head_dim
        kv, rows = cache._struct(layer), cache._rows(seq, pos, table)
        k = torch.empty((n, cache.kv_heads, dim), dtype=torch.float16, device=dev) if k is None else k
        v = torch.empty((n, cache.kv_heads, dim), dtype=torch.float16, device=dev) if v is None else v
        kp, ld_k = _heads(k, dev, "k", n, cache.kv_heads, dim)
        vp, ld_v = _heads(v, dev, "v", n, cache.kv_heads, dim)
        super().__init__("zt_q4_kv_gather", dev, (ctypes.byref(kv), ctypes.byref(rows), kp, ld_k, vp, ld_v),
                         (cache, seq, pos, table, k, v, kv, rows), (k, v), (cache._fill,))


class KvCopy(_Launch):
    """Copies page src[i] onto page dst[i] (int32 CUDA tensors) in every layer of a cache.  No page may be both a
    destination and another entry's source or destination."""

    def __init__(self, cache: KvCache, src, dst):
        n = int(src.numel())
        kv = cache._struct(0)
        super().__init__("zt_q4_kv_copy_pages", cache.device,
                         (ctypes.byref(kv), _ints(src, cache.device, "src", 1, n), _ints(dst, cache.device, "dst", 1, n), n,
                          cache.layers, cache.n_pages * cache.page_bytes), (cache, src, dst, kv), cache.pages,
                         (cache._fill,))


class KvAttention(_Launch):
    """Attention of the last tokens of each sequence over a cache that already holds them: q fp16
    [n_seqs, tokens, q_heads, head_dim] (tokens 1..16, rows may be strided), lens int32 [n_seqs] (cached tokens),
    table int32 [n_seqs, max_pages].  run() returns out, like q and contiguous when not given; a query that sees no
    token gets zeros.  scale defaults to head_dim ** -0.5.  workspace (allocated here when not given): uint8, at least
    kv_attention_workspace_bytes(...), zero-filled before its first use and left so by every call; calls that may overlap
    need workspaces of their own."""

    def __init__(self, cache: KvCache, q, lens, table, layer: int = 0, out=None, scale=None, workspace=None):
        torch = _torch()
        dev, dim = cache.device, cache.head_dim
        _on(q, dev, torch.float16, "q", 4)
        seqs, tokens, heads = (int(n) for n in q.shape[:3])
        kv = cache._struct(layer)
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float16, device=dev)
        (qp, ld_q), (op, ld_out) = (self._rows_of(t, dev, what, seqs, tokens, heads, dim)
                                    for t, what in ((q, "q"), (out, "out")))
        if int(table.shape[0]) != seqs:
            raise ValueError(f"table has {table.shape[0]} rows for {seqs} sequences")
        nbytes = kv_attention_workspace_bytes(cache.kv_heads, heads, dim, tokens)
        fills = (cache._fill,)
        if workspace is None:
            workspace = torch.zeros((max(nbytes, 16),), dtype=torch.uint8, device=dev)
            fills += (_Fill(dev, workspace),)
        _on(workspace, dev, torch.uint8, "workspace", 1)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        super().__init__("zt_q4_kv_attention", dev,
                         (ctypes.byref(kv), qp, ld_q, heads, tokens, _ints(lens, dev, "lens", 1, seqs),
                          _ints(table, dev, "table", 2), seqs, int(table.shape[1]),
                          float(dim ** -0.5 if scale is None else scale), op, ld_out, workspace.data_ptr(),
                          workspace.numel()),
                         (cache, q, lens, table, out, workspace, kv), out, fills)

    @staticmethod
    def _rows_of(t, dev, what, seqs, tokens, heads, dim):
        _on(t, dev, _torch().float16, what, 4)
        if tuple(t.shape) != (seqs, tokens, heads, dim):
            raise ValueError(f"{what} must be [{seqs}, {tokens}, {heads}, {dim}], is {tuple(t.shape)}")
        if tokens > 1 and seqs > 1 and t.stride(0) != tokens * t.stride(1):
            raise ValueError(f"the tokens of {what} must lie at one stride")
        row = t.stride(1) if tokens > 1 else t.stride(0)
        flat = t.as_strided((seqs * tokens, t.shape[2], t.shape[3]), (row, t.stride(2), t.stride(3)), t.storage_offset())
        return _heads(flat, dev, what, seqs * tokens, heads, dim)


class PromptAttention(_Launch):
    """Attention over packed prompts: q fp16 [total_q, q_heads, head_dim], k and v fp16 [total_k, kv_heads, head_dim]
    (rows may be strided: views into a QKV buffer), cu_q and cu_k int32 [n_seqs + 1] offsets of the sequences.  Causal:
    query i of a sequence with nq queries and nk keys sees the first i + 1 + nk - nq keys; a query that sees none gets
    zeros.  run() returns out, contiguous when not given.  scale defaults to head_dim ** -0.5.  errors() reads the error
    word when the device's work has finished (0 unless a bounded wait ran out)."""

    def __init__(self, q, k, v, cu_q, cu_k, causal: bool = True, out=None, scale=None):
        torch = _torch()
        if not q.is_cuda or q.dim() != 3 or k.dim() != 3:
            raise ValueError("q and k must be 3-D CUDA tensors")
        dev, (total_q, heads, dim), (total_k, kv_heads) = q.device, (int(n) for n in q.shape), (int(n) for n in k.shape[:2])
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float16, device=dev)
        (qp, ld_q), (kp, ld_k), (vp, ld_v), (op, ld_o) = (
            _heads(t, dev, what, n, h, dim) for t, what, n, h in
            ((q, "q", total_q, heads), (k, "k", total_k, kv_heads), (v, "v", total_k, kv_heads), (out, "out", total_q, heads)))
        self.err = torch.zeros((1,), dtype=torch.int32, device=dev)
        seqs = int(cu_q.numel()) - 1
        super().__init__("zt_q4_prompt_attention", dev,
                         (qp, ld_q, kp, ld_k, vp, ld_v, _ints(cu_q, dev, "cu_q"), _ints(cu_k, dev, "cu_k", 1, seqs + 1), seqs,
                          total_q, total_k, heads, kv_heads, dim, int(bool(causal)),
                          float(dim ** -0.5 if scale is None else scale), op, ld_o, self.err.data_ptr()),
                         (q, k, v, cu_q, cu_k, out), out, (_Fill(dev, self.err),))

    def errors(self) -> int:
        return _errors(self.err)
