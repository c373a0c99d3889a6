"""Thin ctypes binding of libw8a8.so, with the C entry points' names.

Argument marshalling only: each function checks dtypes/devices, allocates
outputs with torch (device memory), passes raw pointers and the current CUDA
stream to the library, and raises :class:`W8A8Error` on a non-zero status.
Every step of the computation runs in the library's CUDA kernels; there is
no CPU path.  If the library has not been built, :func:`lib` raises.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libw8a8.so")

OK, ERR_INVALID_ARG, ERR_WORKSPACE, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT = 0, -1, -2, -3, -4, -5
PATH_AUTO, PATH_TCGEN05, PATH_GEMV = 0, 1, 2

# Every function the header include/w8a8.h declares.
EXPORTS = (
    "w8a8_quant_act", "w8a8_quant_rows_f32", "w8a8_linear_workspace_size", "w8a8_linear",
    "w8a8_linear_noalloc_scratch_size", "w8a8_linear_noalloc",
    "w8a8_gemm_workspace_size", "w8a8_gemm_q", "w8a8_gemm_s32", "w8a8_moe_workspace_size",
    "w8a8_moe_forward", "w8a8_moe_set_combine", "w8a8_moe_g128_workspace_size", "w8a8_moe_g128_forward", "w8a8_mlp_workspace_size", "w8a8_mlp_forward", "fwht128_quant", "w8a8_linear_g128",
    "group128_quant", "w8a8_linear_group128", "w8a8_trunk_weight_quant", "w8a8_linear_trunk",
    "w8a8_shared_expert_workspace_size", "w8a8_shared_expert_forward",
    "w8a8_linear_epilogue", "w8a8_kv_append", "w8a8_paged_attention_workspace_size", "w8a8_paged_attention",
    "w8a8_token_logprobs",
    "w8a8_exp_proj",
    "w8a8_get_device_error", "w8a8_debug_wait_timeout", "w8a8_status_str", "w8a8_version",
)

_lib = None


class W8A8Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} ({status})")


class MoeG128Debug(ctypes.Structure):
    _fields_ = [("topk_ids", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("qx", ctypes.c_void_p), ("sx", ctypes.c_void_p), ("qa", ctypes.c_void_p),
                ("sa", ctypes.c_void_p)]


class SharedExpertDebug(ctypes.Structure):
    _fields_ = [("qx", ctypes.c_void_p), ("sx", ctypes.c_void_p), ("qa", ctypes.c_void_p), ("sa", ctypes.c_void_p)]


class MlpDebug(ctypes.Structure):
    _fields_ = [("qx", ctypes.c_void_p), ("sx", ctypes.c_void_p), ("qa", ctypes.c_void_p), ("sa", ctypes.c_void_p)]


class MoeDebug(ctypes.Structure):
    _fields_ = [("topk_ids", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("qx", ctypes.c_void_p), ("sx", ctypes.c_void_p), ("qa", ctypes.c_void_p),
                ("sa", ctypes.c_void_p)]


def lib() -> ctypes.CDLL:
    """Loads the library (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libw8a8.so not built ({LIB_PATH}); run moe_gemm_absmax_b200.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    sig = {
        "w8a8_quant_act": ([vp, i64, i64, i64, vp, vp, vp], i32),
        "w8a8_quant_rows_f32": ([vp, i64, i64, vp, vp, vp], i32),
        "w8a8_linear_workspace_size": ([i64, i64, i64], sz),
        "w8a8_linear": ([vp, vp, vp, vp, i64, i64, i64, vp, sz, vp], i32),
        "w8a8_linear_noalloc_scratch_size": ([i64, i64, i64], sz),
        "w8a8_linear_noalloc": ([vp, vp, vp, vp, i64, i64, i64, vp], i32),
        "w8a8_gemm_workspace_size": ([i64, i64, i64, i32], sz),
        "w8a8_gemm_q": ([vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, sz, vp], i32),
        "w8a8_gemm_s32": ([vp, vp, vp, i64, i64, i64, i32, vp, sz, vp], i32),
        "w8a8_moe_workspace_size": ([i64, i32, i32, i32, i32], sz),
        "w8a8_moe_set_combine": ([i32], i32),
        "w8a8_moe_forward": ([vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, vp, sz,
                              ctypes.POINTER(MoeDebug), vp], i32),
        "w8a8_moe_g128_workspace_size": ([i64, i32, i32, i32, i32], sz),
        "w8a8_moe_g128_forward": ([vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, vp, sz,
                                   ctypes.POINTER(MoeG128Debug), vp], i32),
        "w8a8_mlp_workspace_size": ([i64, i64, i64], sz),
        "w8a8_mlp_forward": ([vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, sz, ctypes.POINTER(MlpDebug), vp], i32),
        "fwht128_quant": ([vp, i64, i64, vp, vp, vp], i32),
        "w8a8_linear_g128": ([vp, vp, vp, vp, vp, i64, i64, i64, vp], i32),
        "group128_quant": ([vp, i64, i64, vp, vp, vp], i32),
        "w8a8_linear_group128": ([vp, vp, vp, vp, vp, i64, i64, i64, vp], i32),
        "w8a8_trunk_weight_quant": ([vp, i64, i64, vp, vp, vp, vp], i32),
        "w8a8_linear_trunk": ([vp, vp, vp, vp, vp, vp, i64, i64, i64, vp], i32),
        "w8a8_shared_expert_workspace_size": ([i64, i32, i32], sz),
        "w8a8_shared_expert_forward": ([vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, vp, sz,
                                        ctypes.POINTER(SharedExpertDebug), vp], i32),
        "w8a8_linear_epilogue": ([vp, i64, vp, vp, vp, i32, vp, i64, vp, i64, i64, i64, i64, vp, sz, vp], i32),
        "w8a8_kv_append": ([vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, i32, i32, i64, i32, vp], i32),
        "w8a8_paged_attention_workspace_size": ([i64, i32, i32, i32, i32, i32, i64], sz),
        "w8a8_paged_attention": ([vp, i64, vp, vp, vp, vp, vp, i64, vp, vp, i64, i32, i32, i32, i64, i32, i64, f32, vp,
                                  sz, vp], i32),
        "w8a8_token_logprobs": ([vp, i32, i64, vp, i32, vp, vp, vp, vp, i64, i64, i32, vp], i32),
        "w8a8_exp_proj": ([vp, vp, i64, vp], i32),
        "w8a8_get_device_error": ([vp, ctypes.POINTER(ctypes.c_int)], i32),
        "w8a8_debug_wait_timeout": ([i64, vp], i32),
        "w8a8_status_str": ([i32], ctypes.c_char_p),
        "w8a8_version": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def status_str(status: int) -> str:
    try:
        return lib().w8a8_status_str(int(status)).decode()
    except RuntimeError:
        return "library not loaded"


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise W8A8Error(rc, what)


def _stream(stream=None) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ quant

def quant_act(x: torch.Tensor, stream=None):
    """Per-token int8 quant of bf16 x [M,K] -> (codes int8 [M,K], scales fp32 [M]).

    x may be a row-strided view (unit column stride, row stride = ldx)."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise TypeError("x must be a 2-D bfloat16 tensor")
    M, K = x.shape
    ldx = x.stride(0) if M > 1 else K
    if x.stride(1) != 1 or ldx < K:
        raise ValueError("x rows must be contiguous (unit column stride, row stride >= K)")
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    s = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib().w8a8_quant_act(_ptr(x), M, K, ldx, _ptr(q), _ptr(s), _stream(stream)), "w8a8_quant_act")
    return q, s


def quant_rows_f32(w: torch.Tensor, stream=None):
    """Per-output-channel int8 quant of fp32 weights [N,K] -> (int8 [N,K], fp32 [N])."""
    _need(w, torch.float32, "w")
    K = w.shape[-1]
    N = w.numel() // K
    q = torch.empty(w.shape, dtype=torch.int8, device=w.device)
    s = torch.empty(w.shape[:-1], dtype=torch.float32, device=w.device)
    _check(lib().w8a8_quant_rows_f32(_ptr(w), N, K, _ptr(q), _ptr(s), _stream(stream)), "w8a8_quant_rows_f32")
    return q, s


# ------------------------------------------------------------------ dense

def linear_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().w8a8_linear_workspace_size(M, N, K))


def linear(x: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor, y: torch.Tensor | None = None,
           ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Dense W8A8 linear: bf16 x [M,K] against int8 qw [N,K] / fp32 sw [N] -> bf16 [M,N]."""
    _need(x, torch.bfloat16, "x", 2)
    _need(qw, torch.int8, "qw", 2)
    _need(sw, torch.float32, "sw", 1)
    M, K = x.shape
    N = qw.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    need = linear_workspace_size(M, N, K)
    if ws is None:
        ws = _workspace(need, x.device)
    _check(lib().w8a8_linear(_ptr(x), _ptr(qw), _ptr(sw), _ptr(y), M, N, K, _ptr(ws), ws.numel(),
                             _stream(stream)), "w8a8_linear")
    return y


NOALLOC_SCRATCH_BYTES = 4 << 20


def linear_noalloc(x: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor, y: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """The dense W8A8 linear for callers that cannot allocate device memory
    while it runs: same result as :func:`linear`, scratch kept in the
    library's static device array (at most NOALLOC_SCRATCH_BYTES), so only
    x, the weights and y are passed.  Calls that overlap on the GPU race on
    that array; the first call on a device must come before stream capture.
    (The output tensor is allocated here only when the caller passes none.)"""
    _need(x, torch.bfloat16, "x", 2)
    _need(qw, torch.int8, "qw", 2)
    _need(sw, torch.float32, "sw", 1)
    M, K = x.shape
    N = qw.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _check(lib().w8a8_linear_noalloc(_ptr(x), _ptr(qw), _ptr(sw), _ptr(y), M, N, K, _stream(stream)),
           "w8a8_linear_noalloc")
    return y


def gemm_workspace_size(M: int, N: int, K: int, path: int = PATH_AUTO) -> int:
    return int(lib().w8a8_gemm_workspace_size(M, N, K, path))


def gemm_q(qx, sx, qw, sw, path: int = PATH_AUTO, y=None, ws=None, stream=None) -> torch.Tensor:
    _need(qx, torch.int8, "qx", 2)
    _need(qw, torch.int8, "qw", 2)
    _need(sx, torch.float32, "sx", 1)
    _need(sw, torch.float32, "sw", 1)
    M, K = qx.shape
    N = qw.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=qx.device)
    if ws is None:
        ws = _workspace(gemm_workspace_size(M, N, K, path), qx.device)
    _check(lib().w8a8_gemm_q(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(y), M, N, K, path, _ptr(ws),
                             ws.numel(), _stream(stream)), "w8a8_gemm_q")
    return y


def gemm_s32(qx, qw, path: int = PATH_AUTO, acc=None, ws=None, stream=None) -> torch.Tensor:
    _need(qx, torch.int8, "qx", 2)
    _need(qw, torch.int8, "qw", 2)
    M, K = qx.shape
    N = qw.shape[0]
    if acc is None:
        acc = torch.empty((M, N), dtype=torch.int32, device=qx.device)
    if ws is None:
        ws = _workspace(gemm_workspace_size(M, N, K, path), qx.device)
    _check(lib().w8a8_gemm_s32(_ptr(qx), _ptr(qw), _ptr(acc), M, N, K, path, _ptr(ws), ws.numel(),
                               _stream(stream)), "w8a8_gemm_s32")
    return acc


# ------------------------------------------------------------------ MoE

def moe_workspace_size(T: int, E: int, H: int, I: int, topk: int) -> int:
    return int(lib().w8a8_moe_workspace_size(T, E, H, I, topk))


MOE_COMBINE_AUTO, MOE_COMBINE_EXACT = 0, 1


def moe_set_combine(mode: int) -> int:
    """Combine mode of moe_forward (process-wide); returns the previous one."""
    r = int(lib().w8a8_moe_set_combine(int(mode)))
    if r < 0:
        raise W8A8Error(r, "w8a8_moe_set_combine")
    return r


def moe_forward(x, logits, w13, s13, w2, s2, topk: int = 8, y=None, ws=None, debug: bool = False,
                stream=None):
    """Routed W8A8 MoE layer.  Returns y bf16 [T,H], or (y, debug dict) when debug."""
    _need(x, torch.bfloat16, "x", 2)
    _need(logits, torch.bfloat16, "logits", 2)
    _need(w13, torch.int8, "w13", 3)
    _need(w2, torch.int8, "w2", 3)
    _need(s13, torch.float32, "s13", 2)
    _need(s2, torch.float32, "s2", 2)
    T, H = x.shape
    E, I2, _ = w13.shape
    I = I2 // 2
    dev = x.device
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = _workspace(moe_workspace_size(T, E, H, I, topk), dev)
    dbg_t = None
    dbg_p = None
    if debug:
        dbg_t = dict(topk_ids=torch.empty((T, topk), dtype=torch.int32, device=dev),
                     topk_w=torch.empty((T, topk), dtype=torch.float32, device=dev),
                     counts=torch.empty(E, dtype=torch.int32, device=dev),
                     qx=torch.empty((T, H), dtype=torch.int8, device=dev),
                     sx=torch.empty(T, dtype=torch.float32, device=dev),
                     qa=torch.empty((T, topk, I), dtype=torch.int8, device=dev),
                     sa=torch.empty((T, topk), dtype=torch.float32, device=dev))
        dbg_p = ctypes.pointer(MoeDebug(*[v.data_ptr() for v in dbg_t.values()]))
    _check(lib().w8a8_moe_forward(_ptr(x), _ptr(logits), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), _ptr(y),
                                  T, E, H, I, topk, _ptr(ws), ws.numel(), dbg_p, _stream(stream)),
           "w8a8_moe_forward")
    return (y, dbg_t) if debug else y


# ------------------------------------------------------------------ MoE on the FWHT128 grid

def moe_g128_workspace_size(T: int, E: int, H: int, I: int, topk: int) -> int:
    return int(lib().w8a8_moe_g128_workspace_size(T, E, H, I, topk))


def moe_g128_forward(x, logits, w13, s13, w2, s2, topk: int = 8, y=None, ws=None, debug: bool = False,
                     stream=None):
    """Routed experts on the FWHT128 grid: bf16 x [T,H] (unrotated), bf16 logits [T,E];
    w13 int8 [E,2I,H] with bf16 group scales s13 [E,2I,H/128]; w2 int8 [E,H,I] with
    s2 [E,H,I/128] (rows rotated along K and group-quantized, e.g. by fwht128_quant).
    Returns y bf16 [T,H], or (y, debug dict) when debug."""
    _need(x, torch.bfloat16, "x", 2)
    _need(logits, torch.bfloat16, "logits", 2)
    _need(w13, torch.int8, "w13", 3)
    _need(w2, torch.int8, "w2", 3)
    _need(s13, torch.bfloat16, "s13", 3)
    _need(s2, torch.bfloat16, "s2", 3)
    T, H = x.shape
    E, I2, _ = w13.shape
    I = I2 // 2
    dev = x.device
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = _workspace(moe_g128_workspace_size(T, E, H, I, topk), dev)
    dbg_t = None
    dbg_p = None
    if debug:
        dbg_t = dict(topk_ids=torch.empty((T, topk), dtype=torch.int32, device=dev),
                     topk_w=torch.empty((T, topk), dtype=torch.float32, device=dev),
                     counts=torch.empty(E, dtype=torch.int32, device=dev),
                     qx=torch.empty((T, H), dtype=torch.int8, device=dev),
                     sx=torch.empty((T, H // 128), dtype=torch.bfloat16, device=dev),
                     qa=torch.empty((T, topk, I), dtype=torch.int8, device=dev),
                     sa=torch.empty((T, topk, I // 128), dtype=torch.bfloat16, device=dev))
        dbg_p = ctypes.pointer(MoeG128Debug(*[v.data_ptr() for v in dbg_t.values()]))
    _check(lib().w8a8_moe_g128_forward(_ptr(x), _ptr(logits), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), _ptr(y),
                                       T, E, H, I, topk, _ptr(ws), ws.numel(), dbg_p, _stream(stream)),
           "w8a8_moe_g128_forward")
    return (y, dbg_t) if debug else y


# ------------------------------------------------------------------ dense gated MLP block

def mlp_workspace_size(M: int, H: int, I: int) -> int:
    return int(lib().w8a8_mlp_workspace_size(M, H, I))


def mlp_forward(x, w13, s13, w2, s2, y=None, ws=None, debug: bool = False, stream=None):
    """Dense gated MLP block: bf16 x [M,H] -> gate_up (w13 int8 [2I,H], rows 2i gate /
    2i+1 up, s13 [2I]) with SiLU(gate)*up -> requant -> down (w2 int8 [H,I], s2 [H])
    -> bf16 y [M,H].  Returns y, or (y, debug dict) when debug."""
    _need(x, torch.bfloat16, "x", 2)
    _need(w13, torch.int8, "w13", 2)
    _need(w2, torch.int8, "w2", 2)
    _need(s13, torch.float32, "s13", 1)
    _need(s2, torch.float32, "s2", 1)
    M, H = x.shape
    I = w13.shape[0] // 2
    dev = x.device
    if y is None:
        y = torch.empty((M, H), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = _workspace(mlp_workspace_size(M, H, I), dev)
    dbg_t = dbg_p = None
    if debug:
        dbg_t = dict(qx=torch.empty((M, H), dtype=torch.int8, device=dev),
                     sx=torch.empty(M, dtype=torch.float32, device=dev),
                     qa=torch.empty((M, I), dtype=torch.int8, device=dev),
                     sa=torch.empty(M, dtype=torch.float32, device=dev))
        dbg_p = ctypes.pointer(MlpDebug(*[v.data_ptr() for v in dbg_t.values()]))
    _check(lib().w8a8_mlp_forward(_ptr(x), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), _ptr(y), M, H, I, _ptr(ws),
                                  ws.numel(), dbg_p, _stream(stream)), "w8a8_mlp_forward")
    return (y, dbg_t) if debug else y


# ------------------------------------------------------------------ FWHT128

def fwht128_quant(x: torch.Tensor, stream=None):
    """Rotated group-128 quant of bf16 x [M,K] -> (int8 [M,K], bf16 scales [M,K/128])."""
    _need(x, torch.bfloat16, "x", 2)
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    s = torch.empty((M, K // 128), dtype=torch.bfloat16, device=x.device)
    _check(lib().fwht128_quant(_ptr(x), M, K, _ptr(q), _ptr(s), _stream(stream)), "fwht128_quant")
    return q, s


def linear_g128(qx, sx, qw, sw, y=None, stream=None) -> torch.Tensor:
    _need(qx, torch.int8, "qx", 2)
    _need(qw, torch.int8, "qw", 2)
    _need(sx, torch.bfloat16, "sx", 2)
    _need(sw, torch.bfloat16, "sw", 2)
    M, K = qx.shape
    N = qw.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=qx.device)
    _check(lib().w8a8_linear_g128(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(y), M, N, K, _stream(stream)),
           "w8a8_linear_g128")
    return y


def group128_quant(x: torch.Tensor, stream=None):
    """Group-128 quant without the rotation (the head's grid): bf16 x [M,K] ->
    (int8 [M,K], bf16 scales [M,K/128])."""
    _need(x, torch.bfloat16, "x", 2)
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    s = torch.empty((M, K // 128), dtype=torch.bfloat16, device=x.device)
    _check(lib().group128_quant(_ptr(x), M, K, _ptr(q), _ptr(s), _stream(stream)), "group128_quant")
    return q, s


def linear_group128(qx, sx, qw, sw, y=None, stream=None) -> torch.Tensor:
    """Group-128 GEMM on the unrotated grid (no 1/128): -> bf16 y [M,N]."""
    _need(qx, torch.int8, "qx", 2)
    _need(qw, torch.int8, "qw", 2)
    _need(sx, torch.bfloat16, "sx", 2)
    _need(sw, torch.bfloat16, "sw", 2)
    M, K = qx.shape
    N = qw.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=qx.device)
    _check(lib().w8a8_linear_group128(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(y), M, N, K, _stream(stream)),
           "w8a8_linear_group128")
    return y


def trunk_weight_quant(w: torch.Tensor, stream=None):
    """The trunk's two-level format of bf16 rows [N,K] (K % 256 == 0): returns
    (codes int8 [N,K], u8 group scales [N,K/256], bf16 row scales [N])."""
    _need(w, torch.bfloat16, "w", 2)
    N, K = w.shape
    q = torch.empty((N, K), dtype=torch.int8, device=w.device)
    su8 = torch.empty((N, K // 256), dtype=torch.uint8, device=w.device)
    s2 = torch.empty(N, dtype=torch.bfloat16, device=w.device)
    _check(lib().w8a8_trunk_weight_quant(_ptr(w), N, K, _ptr(q), _ptr(su8), _ptr(s2), _stream(stream)),
           "w8a8_trunk_weight_quant")
    return q, su8, s2


def linear_trunk(qx, sx, qw, su8, s2, y=None, stream=None) -> torch.Tensor:
    """x codes + bf16 group scales (fwht128_quant) times W in the trunk format -> bf16 y [M,N]."""
    _need(qx, torch.int8, "qx", 2)
    _need(qw, torch.int8, "qw", 2)
    _need(sx, torch.bfloat16, "sx", 2)
    _need(su8, torch.uint8, "su8", 2)
    _need(s2, torch.bfloat16, "s2", 1)
    M, K = qx.shape
    N = qw.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=qx.device)
    _check(lib().w8a8_linear_trunk(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(su8), _ptr(s2), _ptr(y), M, N, K,
                                   _stream(stream)), "w8a8_linear_trunk")
    return y


def shared_expert_workspace_size(M: int, H: int, I: int) -> int:
    return int(lib().w8a8_shared_expert_workspace_size(M, H, I))


def shared_expert_forward(x, w13, u13, r13, w2, s2, y=None, ws=None, debug: bool = False, stream=None):
    """The shared expert on the rotated grid: bf16 x [M,H]; gate_up in the trunk format
    (w13 int8 [2I,H], u13 uint8 [2I,H/256], r13 bf16 [2I]); down on the group-128 grid
    (w2 int8 [H,I], s2 bf16 [H,I/128]).  Returns y bf16 [M,H], or (y, debug dict)."""
    _need(x, torch.bfloat16, "x", 2)
    _need(w13, torch.int8, "w13", 2)
    _need(u13, torch.uint8, "u13", 2)
    _need(r13, torch.bfloat16, "r13", 1)
    _need(w2, torch.int8, "w2", 2)
    _need(s2, torch.bfloat16, "s2", 2)
    M, H = x.shape
    I = w13.shape[0] // 2
    dev = x.device
    if y is None:
        y = torch.empty((M, H), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = _workspace(shared_expert_workspace_size(M, H, I), dev)
    dbg_t = dbg_p = None
    if debug:
        dbg_t = dict(qx=torch.empty((M, H), dtype=torch.int8, device=dev),
                     sx=torch.empty((M, H // 128), dtype=torch.bfloat16, device=dev),
                     qa=torch.empty((M, I), dtype=torch.int8, device=dev),
                     sa=torch.empty((M, I // 128), dtype=torch.bfloat16, device=dev))
        dbg_p = ctypes.pointer(SharedExpertDebug(*[v.data_ptr() for v in dbg_t.values()]))
    _check(lib().w8a8_shared_expert_forward(_ptr(x), _ptr(w13), _ptr(u13), _ptr(r13), _ptr(w2), _ptr(s2), _ptr(y),
                                            M, H, I, _ptr(ws), ws.numel(), dbg_p, _stream(stream)),
           "w8a8_shared_expert_forward")
    return (y, dbg_t) if debug else y


# ------------------------------------------------------------------ linear with an epilogue

ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = range(5)


def _placed(fn):
    """Runs fn with the device of its first tensor current and, where a stream is given, on that stream: what fn
    allocates then belongs to the stream that uses it, so the caching allocator cannot hand it on too early.  fn gets
    the raw stream as raw_stream; callers give stream=, and see that in the signature."""
    params = list(inspect.signature(fn).parameters.values())
    name = params[0].name
    shown = [p for p in params if p.name != "raw_stream"]
    shown.append(inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None))

    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        if not args and name not in kwargs:
            raise TypeError(f"{fn.__name__}() missing 1 required positional argument: '{name}'")
        first = args[0] if args else kwargs[name]
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        index = first.get_device()
        if stream is None and index == torch._C._cuda_getDevice():
            return fn(*args, raw_stream=_raw_stream(index), **kwargs)
        if stream is None:
            with torch.cuda.device(index):
                return fn(*args, raw_stream=_raw_stream(index), **kwargs)
        if stream.device != first.device:
            raise ValueError("stream is on another device than the tensors")
        with torch.cuda.stream(stream):
            return fn(*args, raw_stream=stream.cuda_stream, **kwargs)

    call.__signature__ = inspect.Signature(shown)
    return call


def _raw_stream(index: int) -> int:
    """cudaStream_t of the device's current stream, without a Stream object around it (3 us of a 10 us call)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _bytes(n: int, device) -> torch.Tensor:
    return torch.empty_strided((n,), (1,), dtype=torch.uint8, device=device)


def _on(t, dtype, name, shape, device):
    """Contiguous tensor of this type, shape and device; its address."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.device != device \
            or not t.is_contiguous():
        _need(t, dtype, name)
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t.data_ptr()


def _caller_ws(ws, device):
    """Address and bytes of a workspace that the caller gave."""
    if not isinstance(ws, torch.Tensor) or ws.device != device:
        raise TypeError(f"ws must be a CUDA tensor on {device}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _row_stride(t, dtype, name, device, shape=None, ndim=2) -> int:
    """Row stride of a tensor whose rows (all but the first dim) are dense."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise TypeError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    size, step = t.shape, t.stride()
    if len(size) != ndim or (shape is not None and size != shape):
        raise ValueError(f"{name} must have shape {tuple(shape) if shape is not None else f'({ndim} dims)'}, "
                         f"got {tuple(size)}")
    n = size[1] if ndim == 2 else size[1] * size[2]
    if step[-1] != 1 or (ndim == 3 and step[1] != size[2]):   # strides of a dim of size 1 do not matter
        if (size[-1] != 1 and step[-1] != 1) or (ndim == 3 and size[1] != 1 and step[1] != size[2]):
            raise ValueError(f"{name}: all but the first dim must be dense")
    return step[0] if size[0] > 1 else n


@functools.lru_cache(maxsize=1024)
def _linear_ws(M: int, N: int, K: int) -> int:
    return max(linear_workspace_size(M, N, K), 256)


@_placed
def linear_epilogue(x, qw, sw, bias=None, act: int = ACT_NONE, residual=None, y=None, ws=None, *,
                    raw_stream) -> torch.Tensor:
    """Online W8A8 linear with its epilogue: y = residual + act(linear(x) + bias), rounded to bf16 once.

    x bf16 [M,K]; qw int8 [N,K], sw fp32 [N]; bias fp32 [N]; residual and y bf16 [M,N].  x, residual and y may be
    row-strided (unit column stride, row strides a multiple of 8); y may be the residual itself.  act is one of
    ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH.  stream= as in the other calls."""
    dev = x.device
    ldx = _row_stride(x, torch.bfloat16, "x", dev)
    M, K = x.shape
    if not isinstance(qw, torch.Tensor) or qw.dim() != 2:
        raise TypeError("qw must be a 2-D CUDA tensor")
    N = qw.shape[0]
    pw, ps = _on(qw, torch.int8, "qw", (N, K), dev), _on(sw, torch.float32, "sw", (N,), dev)
    pb = None if bias is None else _on(bias, torch.float32, "bias", (N,), dev)
    ldr, pr = 0, None
    if residual is not None:
        ldr, pr = _row_stride(residual, torch.bfloat16, "residual", dev, (M, N)), residual.data_ptr()
    if y is None:
        y, ldy = torch.empty_strided((M, N), (N, 1), dtype=torch.bfloat16, device=dev), N
    else:
        ldy = _row_stride(y, torch.bfloat16, "y", dev, (M, N))
    if ws is None:
        nws = _linear_ws(M, N, K)
        ws = _bytes(nws, dev)
        pws = ws.data_ptr()
    else:
        pws, nws = _caller_ws(ws, dev)
    _check(lib().w8a8_linear_epilogue(x.data_ptr(), ldx, pw, ps, pb, act, pr, ldr, y.data_ptr(), ldy, M, N, K,
                                      pws, nws, raw_stream), "w8a8_linear_epilogue")
    return y


# ------------------------------------------------------------------ paged cache and attention

def _cache_args(k_cache, v_cache, k_scale, v_scale, device):
    """Shape (pages, Hkv, page size, D) of a paged cache, int8 with scales or bf16 without, and its addresses."""
    dtype = torch.bfloat16 if k_scale is None else torch.int8
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise TypeError("k_cache must be a 4-D CUDA tensor")
    shape = k_cache.shape
    pk, pv = _on(k_cache, dtype, "k_cache", shape, device), _on(v_cache, dtype, "v_cache", shape, device)
    if k_scale is None:
        if v_scale is not None:
            raise ValueError("k_scale and v_scale are given together or not at all")
        return shape, pk, pv, None, None
    return (shape, pk, pv, _on(k_scale, torch.float32, "k_scale", shape[:3], device),
            _on(v_scale, torch.float32, "v_scale", shape[:3], device))


@_placed
def kv_append(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None, *, raw_stream) -> None:
    """Writes the keys and values of T tokens into the paged cache, in place.

    k, v bf16 [T,Hkv,D] (token stride a multiple of 8, the rest dense); caches [pages,Hkv,page_size,D], int8 with
    scales fp32 [pages,Hkv,page_size] or bf16 without; slots int64 [T], page * page_size + position, negative to
    skip a token, distinct otherwise.  A slot past the cache is skipped and shows in get_device_error()."""
    dev = k.device
    ldk = _row_stride(k, torch.bfloat16, "k", dev, ndim=3)
    ldv = _row_stride(v, torch.bfloat16, "v", dev, k.shape, ndim=3)
    (pages, Hkv, page, D), pkc, pvc, pks, pvs = _cache_args(k_cache, v_cache, k_scale, v_scale, dev)
    T = k.shape[0]
    if k.shape[1:] != (Hkv, D):
        raise ValueError(f"k has heads {tuple(k.shape[1:])}, the cache {(Hkv, D)}")
    _check(lib().w8a8_kv_append(k.data_ptr(), ldk, v.data_ptr(), ldv, pkc, pvc, pks, pvs,
                                _on(slots, torch.int64, "slots", (T,), dev), T, Hkv, D, pages, page, raw_stream),
           "w8a8_kv_append")


def paged_attention_workspace_size(B: int, Hq: int, Hkv: int, D: int, int8: bool, page_size: int,
                                   max_pages: int) -> int:
    return int(lib().w8a8_paged_attention_workspace_size(B, Hq, Hkv, D, int8, page_size, max_pages))


_attention_ws = functools.lru_cache(maxsize=4096)(paged_attention_workspace_size)


@_placed
def paged_attention(q, k_cache, v_cache, block_table, lengths, scale: float | None = None, k_scale=None, v_scale=None,
                    y=None, ws=None, *, raw_stream) -> torch.Tensor:
    """Attention of one new token per sequence over the paged cache -> bf16 [B,Hq,D].

    q bf16 [B,Hq,D] (sequence stride a multiple of 8, the rest dense); caches as in :func:`kv_append`; block_table
    int32 [B,max_pages], lengths int32 [B] (the new token included).  scale defaults to D ** -0.5.  A sequence of
    length 0 gives zeros; absent pages and lengths past the table show in get_device_error()."""
    dev = q.device
    ldq = _row_stride(q, torch.bfloat16, "q", dev, ndim=3)
    (pages, Hkv, page, D), pkc, pvc, pks, pvs = _cache_args(k_cache, v_cache, k_scale, v_scale, dev)
    B, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError(f"q has head dim {Dq}, the cache {D}")
    ld_table = _row_stride(block_table, torch.int32, "block_table", dev)
    if block_table.shape[0] != B:
        raise ValueError("block_table must have a row per sequence")
    if y is None:
        y = torch.empty_strided((B, Hq, D), (Hq * D, D, 1), dtype=torch.bfloat16, device=dev)
        py = y.data_ptr()
    else:
        py = _on(y, torch.bfloat16, "y", (B, Hq, D), dev)
    max_pages, pws = block_table.shape[1], None
    if ws is None:
        nws = _attention_ws(B, Hq, Hkv, D, pks is not None, page, max_pages)
        if nws:
            ws = _bytes(nws, dev)
            pws = ws.data_ptr()
    else:
        pws, nws = _caller_ws(ws, dev)
    _check(lib().w8a8_paged_attention(q.data_ptr(), ldq, pkc, pvc, pks, pvs, block_table.data_ptr(), ld_table,
                                      _on(lengths, torch.int32, "lengths", (B,), dev), py, B, Hq, Hkv, D, pages, page,
                                      max_pages, D ** -0.5 if scale is None else scale, pws, nws, raw_stream),
           "w8a8_paged_attention")
    return y


# ------------------------------------------------------------------ log probabilities

@_placed
def token_logprobs(logits, tokens=None, topk: int = 0, entropy: bool = True, *, raw_stream):
    """Log probabilities from the head's logits [M,V], bf16 or fp32 (rows may be strided).

    Returns (logprob, entropy, top_ids, top_logprobs): fp32 of the shape of tokens (int32 [M] or [M,G]; NaN for a
    token outside the vocabulary), fp32 [M] in nats, int32 [M,topk] by descending logit with ties to the lower index,
    fp32 [M,topk].  None for what was not asked for."""
    dev, dtype = logits.device, logits.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError(f"logits must be torch.bfloat16 or torch.float32, got {dtype}")
    ld = _row_stride(logits, dtype, "logits", dev)
    M, V = logits.shape
    f32 = torch.float32
    G, logprob, h, ids, top = 0, None, None, None, None
    pt = pl = ph = pi = pv = None
    if tokens is not None:
        if not isinstance(tokens, torch.Tensor) or tokens.dim() not in (1, 2) or tokens.shape[0] != M:
            raise ValueError("tokens must be [M] or [M, G]")
        pt = _on(tokens, torch.int32, "tokens", tokens.shape, dev)
        G = 1 if tokens.dim() == 1 else tokens.shape[1]
        logprob = torch.empty_like(tokens, dtype=f32)
        pl = logprob.data_ptr()
    if entropy:
        h = torch.empty_strided((M,), (1,), dtype=f32, device=dev)
        ph = h.data_ptr()
    if topk > 0:
        ids = torch.empty_strided((M, topk), (topk, 1), dtype=torch.int32, device=dev)
        top = torch.empty_strided((M, topk), (topk, 1), dtype=f32, device=dev)
        pi, pv = ids.data_ptr(), top.data_ptr()
    _check(lib().w8a8_token_logprobs(logits.data_ptr(), int(dtype is f32), ld, pt, G, pl, ph, pi, pv, M, V, topk,
                                     raw_stream), "w8a8_token_logprobs")
    return logprob, h, ids, top


# ------------------------------------------------------------------ diagnostics

def exp_proj(x: torch.Tensor, stream=None) -> torch.Tensor:
    _need(x, torch.float32, "x")
    y = torch.empty_like(x)
    _check(lib().w8a8_exp_proj(_ptr(x), _ptr(y), x.numel(), _stream(stream)), "w8a8_exp_proj")
    return y


def get_device_error(stream=None):
    """Synchronizes the stream; returns (status, site) and clears the error word."""
    site = ctypes.c_int(0)
    rc = lib().w8a8_get_device_error(_stream(stream), ctypes.byref(site))
    return int(rc), int(site.value)


def debug_wait_timeout(limit_ns: int, stream=None) -> None:
    _check(lib().w8a8_debug_wait_timeout(int(limit_ns), _stream(stream)), "w8a8_debug_wait_timeout")


def version() -> str:
    return lib().w8a8_version().decode()
