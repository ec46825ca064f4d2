"""gemm_rocmfp2_mul_gb300: ROCmFP2 / HFP4G32 block-quantized GEMV and GEMM on GB300.

Thin Python binding of ``librfp2.so`` (C ABI declared in ``include/rfp2.h``).
Every function has the name of the C entry point it calls and only marshals
arguments: it takes torch CUDA tensors, allocates outputs and workspaces with
torch when the caller does not pass them, passes raw device pointers and the
current torch stream to the library, and raises :class:`RFP2Error` on a
non-zero status.  All arithmetic runs in the library's CUDA kernels; there is
no CPU or PyTorch fallback: if the library is not built or cannot be loaded,
every call raises.  Tensors have to be on the current device, where the library
launches.  Most calls go through ctypes; those of the attention operators, small
and many, through a compiled binding.

Build the library with :func:`build` (nvcc, sm_103a).
"""
from __future__ import annotations

import ctypes as C
import importlib.util
import os
import threading
from typing import Any, NamedTuple

__all__ = [
    "RFP2Error", "build", "lib", "library_path", "status_str",
    "rfp2_quantize_act", "rfp2_gemv_q8", "rfp2_gemv", "rfp2_gemv_workspace_bytes",
    "rfp2_gemv_noalloc",
    "rfp2_moe_gemv", "rfp2_moe_workspace_bytes", "rfp2_gemm", "rfp2_gemm_workspace_bytes",
    "hfp4_gemv", "hfp4_gemv_workspace_bytes", "hfp4_gemm", "hfp4_gemm_workspace_bytes",
    "rfp2_nvfp4_weight_bytes", "rfp2_to_nvfp4", "rfp2_gemm_nvfp4", "rfp2_gemm_nvfp4_workspace_bytes",
    "rfp2_gemv_batched", "rfp2_gemv_batched_workspace_bytes",
    "rfp2_pack_weights", "rfp2_pack_weights_weighted", "hfp4_pack_weights", "rfp2_validate_weights",
    "rfp2_debug_half_partials", "rfp2_debug_wait_timeout", "rfp2_row_bytes", "hfp4_row_bytes",
    "rfp2_set_weight_prefetch", "rfp2_weight_prefetch",
    "KVCache", "rfp2_rope_frequencies", "rfp2_rope", "rfp2_kv_alloc", "rfp2_kv_write", "rfp2_kv_read",
    "rfp2_attn_decode", "rfp2_attn_decode_workspace", "rfp2_attn_decode_workspace_bytes",
]

MAX_BATCH = 8
_lock = threading.Lock()
_lib = None


class RFP2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} ({status})")


def library_path() -> str:
    from . import buildlib as _b
    return _b.LIB


def build(force: bool = False) -> str:
    """Compile librfp2.so in-tree (nvcc, sm_103a)."""
    from . import buildlib as _b
    return _b.build(force=force)


_P, _I64, _I32, _SZ = C.c_void_p, C.c_int64, C.c_int, C.c_size_t
_F32, _F64 = C.c_float, C.c_double

_SIGNATURES = {
    "rfp2_status_str": (C.c_char_p, [_I32]),
    "rfp2_version": (_I32, []),
    "rfp2_quantize_act": (_I32, [_P, _I64, _I64, _P, _P, _P]),
    "rfp2_gemv_q8": (_I32, [_P, _I64, _I64, _P, _P, _I64, _P, _P, _P]),
    "rfp2_gemv_workspace_bytes": (_SZ, [_I64, _I64]),
    "rfp2_gemv": (_I32, [_P, _I64, _I64, _P, _I64, _P, _P, _SZ, _P, _P]),
    "rfp2_gemv_noalloc": (_I32, [_P, _I64, _I64, _P, _I64, _P, _P, _P]),
    "rfp2_moe_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "rfp2_moe_gemv": (_I32, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _SZ, _P, _P]),
    "rfp2_gemm_workspace_bytes": (_SZ, [_I64, _I64]),
    "rfp2_gemm": (_I32, [_P, _I64, _I64, _P, _I64, _P, _P, _SZ, _P, _P]),
    "rfp2_gemv_batched_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "rfp2_gemv_batched": (_I32, [_P, _I64, _I64, _P, _I64, _P, _P, _SZ, _P, _P]),
    "hfp4_gemm_workspace_bytes": (_SZ, [_I64, _I64]),
    "hfp4_gemm": (_I32, [_P, _I64, _I64, _P, _I64, _P, _P, _SZ, _P, _P]),
    "rfp2_nvfp4_weight_bytes": (_SZ, [_I64, _I64]),
    "rfp2_to_nvfp4": (_I32, [_P, _I64, _I64, _P, _P]),
    "rfp2_gemm_nvfp4_workspace_bytes": (_SZ, [_I64, _I64]),
    "rfp2_gemm_nvfp4": (_I32, [_P, _I64, _I64, _P, _I64, _P, _P, _SZ, _P, _P]),
    "hfp4_gemv_workspace_bytes": (_SZ, [_I64, _I64]),
    "hfp4_gemv": (_I32, [_P, _I64, _I64, _P, _I64, _P, _P, _SZ, _P, _P]),
    "rfp2_pack_weights": (_I32, [_P, _I64, _I64, _P, _P]),
    "rfp2_pack_weights_weighted": (_I32, [_P, _I64, _I64, _P, _P, _P]),
    "hfp4_pack_weights": (_I32, [_P, _I64, _I64, _P, _P, _P]),
    "rfp2_validate_weights": (_I32, [_P, _I64, _P, _P, _P]),
    "rfp2_debug_half_partials": (_I32, [_P, _I64, _I64, _P, _I64, _P, _P]),
    "rfp2_debug_wait_timeout": (_I32, [_P, _P]),
    "rfp2_set_weight_prefetch": (_I32, [_I32]),
    "rfp2_weight_prefetch": (_I32, []),
    "rfp2_rope_frequencies": (_I32, [_I64, _F64, _I32, _F64, _F64, _F64, _F64, _P, _P]),
    "rfp2_rope": (_I32, [_P, _I32, _I64, _I64, _I64, _I64, _I64, _P, _P, _I64, _F32, _I32, _P, _I64,
                         _I64, _P]),
    "rfp2_kv_write": (_I32, [_P, _P, _I32] + [_I64] * 5 + [_P, _P, _P, _I64, _F32, _I32]
                      + [_P] * 4 + [_I64] * 4 + [_P, _P]),
    "rfp2_kv_read": (_I32, [_P] * 4 + [_I64] * 4 + [_P, _I64, _I32, _P, _P, _P, _P]),
    "rfp2_attn_decode_workspace_bytes": (_SZ, [_I64] * 5),
    "rfp2_attn_decode": (_I32, [_P, _I32] + [_I64] * 7 + [_P] * 4 + [_I64] * 3
                         + [_P, _I64, _I64, _P, _F32, _I64, _F32, _P, _P, _P, _SZ, _P, _P]),
}


def lib():
    """The loaded ctypes library (raises if it is not built)."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"librfp2.so is not built ({path}); run gemm_rocmfp2_mul_gb300.build()")
            L = C.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def status_str(status: int) -> str:
    try:
        return lib().rfp2_status_str(int(status)).decode()
    except Exception:
        return f"status {status}"


# -- marshalling helpers --------------------------------------------------------

def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream():
    cuda = _torch()._C
    return C.c_void_p(cuda._cuda_getCurrentRawStream(cuda._cuda_getDevice()))


def _need(t, dtype, name, device=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current device")  # where the library launches
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _check(rc: int, what: str):
    if rc != 0:
        raise RFP2Error(rc, what)


def _empty(shape, dtype, like):
    return _torch().empty(shape, dtype=dtype, device=like.device)


def rfp2_row_bytes(K: int) -> int:
    """Packed bytes per ROCmFP2 row (10 bytes per 32 weights)."""
    return K // 32 * 10


def hfp4_row_bytes(K: int) -> int:
    """Bytes per HFP4G32 row (16-byte header + 17 bytes per 32 weights)."""
    return 16 + 17 * (K // 32)


def _workspace(ws, nbytes, like):
    torch = _torch()
    if ws is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=like.device)
    _need(ws, torch.uint8, "workspace")
    return ws


# -- entry points -----------------------------------------------------------------

def rfp2_quantize_act(x, q=None, d=None):
    """x fp32 [N, K] -> (q int8 [N, K], d fp32 [N, K/32])."""
    torch = _torch()
    _need(x, torch.float32, "x")
    N, K = x.shape
    q = _empty((N, K), torch.int8, x) if q is None else _need(q, torch.int8, "q")
    d = _empty((N, K // 32), torch.float32, x) if d is None else _need(d, torch.float32, "d")
    _check(lib().rfp2_quantize_act(_ptr(x), N, K, _ptr(q), _ptr(d), _stream()),
           "rfp2_quantize_act")
    return q, d


def rfp2_gemv_q8(W, M, K, q, d, y=None, dev_status=None):
    """ROCmFP2 GEMV on quantized activations: y fp32 [N, M]."""
    torch = _torch()
    _need(W, torch.uint8, "W")
    _need(q, torch.int8, "q")
    _need(d, torch.float32, "d")
    N = q.shape[0]
    y = _empty((N, M), torch.float32, q) if y is None else _need(y, torch.float32, "y")
    _check(lib().rfp2_gemv_q8(_ptr(W), M, K, _ptr(q), _ptr(d), N, _ptr(y), _ptr(dev_status),
                              _stream()), "rfp2_gemv_q8")
    return y


def rfp2_gemv_workspace_bytes(N: int, K: int) -> int:
    return int(lib().rfp2_gemv_workspace_bytes(N, K))


def rfp2_gemv(W, M, K, x, y=None, workspace=None, dev_status=None):
    """ROCmFP2 GEMV from fp32 activations (quantize + GEMV): y fp32 [N, M]."""
    torch = _torch()
    _need(W, torch.uint8, "W")
    _need(x, torch.float32, "x")
    N = x.shape[0]
    y = _empty((N, M), torch.float32, x) if y is None else _need(y, torch.float32, "y")
    nb = rfp2_gemv_workspace_bytes(N, K)
    ws = _workspace(workspace, nb, x)
    _check(lib().rfp2_gemv(_ptr(W), M, K, _ptr(x), N, _ptr(y), _ptr(ws), ws.numel(),
                           _ptr(dev_status), _stream()), "rfp2_gemv")
    return y


def rfp2_set_weight_prefetch(enable: bool) -> None:
    """Process-wide switch (default off): let the GEMV kernels start reading
    W before the kernel enqueued just before them has completed.  Turn it on
    only when no kernel that may still be running on the stream writes W."""
    _check(lib().rfp2_set_weight_prefetch(1 if enable else 0), "rfp2_set_weight_prefetch")


def rfp2_weight_prefetch() -> bool:
    """The current weight-prefetch setting."""
    return bool(lib().rfp2_weight_prefetch())


def rfp2_gemv_noalloc(W, M, K, x, y=None, dev_status=None):
    """rfp2_gemv for callers that cannot allocate device memory: the quantized
    activations go to scratch built into the library (N*K <= 65536; calls on
    one device must not overlap on the GPU).  y fp32 [N, M]; pass `y` to avoid
    the one torch allocation this wrapper would otherwise make."""
    torch = _torch()
    _need(W, torch.uint8, "W")
    _need(x, torch.float32, "x")
    N = x.shape[0]
    y = _empty((N, M), torch.float32, x) if y is None else _need(y, torch.float32, "y")
    _check(lib().rfp2_gemv_noalloc(_ptr(W), M, K, _ptr(x), N, _ptr(y), _ptr(dev_status),
                                   _stream()), "rfp2_gemv_noalloc")
    return y


def rfp2_moe_workspace_bytes(T: int, top_k: int, K: int) -> int:
    return int(lib().rfp2_moe_workspace_bytes(T, top_k, K))


def rfp2_moe_gemv(W, E, M, K, ids, x, y=None, workspace=None, dev_status=None):
    """MoE expert-indexed GEMV: y fp32 [T, top_k, M] = W[ids[t, j]] x_t."""
    torch = _torch()
    _need(W, torch.uint8, "W")
    _need(ids, torch.int32, "ids")
    _need(x, torch.float32, "x")
    T, top_k = ids.shape
    y = _empty((T, top_k, M), torch.float32, x) if y is None else _need(y, torch.float32, "y")
    ws = _workspace(workspace, rfp2_moe_workspace_bytes(T, top_k, K), x)
    _check(lib().rfp2_moe_gemv(_ptr(W), E, M, K, _ptr(ids), T, top_k, _ptr(x), _ptr(y), _ptr(ws),
                               ws.numel(), _ptr(dev_status), _stream()), "rfp2_moe_gemv")
    return y


def rfp2_gemm_workspace_bytes(M: int, K: int) -> int:
    return int(lib().rfp2_gemm_workspace_bytes(M, K))


def rfp2_gemm(W, M, K, X, Y=None, workspace=None, dev_status=None):
    """Prefill GEMM on tensor cores: Y fp32 [N, M] = X (bf16 [N, K]) W^T."""
    torch = _torch()
    _need(W, torch.uint8, "W")
    if X.dtype == torch.bfloat16:
        X = X.view(torch.int16)
    if X.dtype not in (torch.int16, torch.uint16):
        raise TypeError("X must be bfloat16 (or its 16-bit pattern)")
    _need(X, X.dtype, "X")
    N = X.shape[0]
    Y = _empty((N, M), torch.float32, X) if Y is None else _need(Y, torch.float32, "Y")
    ws = _workspace(workspace, rfp2_gemm_workspace_bytes(M, K), X)
    _check(lib().rfp2_gemm(_ptr(W), M, K, _ptr(X), N, _ptr(Y), _ptr(ws), ws.numel(),
                           _ptr(dev_status), _stream()), "rfp2_gemm")
    return Y


def rfp2_gemv_batched_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().rfp2_gemv_batched_workspace_bytes(M, K, N))


def rfp2_gemv_batched(W, M, K, x, y=None, workspace=None, dev_status=None):
    """ROCmFP2 GEMV on Q8_1 activations for verify batches (tensor cores):
    y fp32 [N, M] from fp32 x [N, K]."""
    torch = _torch()
    _need(W, torch.uint8, "W")
    _need(x, torch.float32, "x")
    N = x.shape[0]
    y = _empty((N, M), torch.float32, x) if y is None else _need(y, torch.float32, "y")
    ws = _workspace(workspace, rfp2_gemv_batched_workspace_bytes(M, K, N), x)
    _check(lib().rfp2_gemv_batched(_ptr(W), M, K, _ptr(x), N, _ptr(y), _ptr(ws), ws.numel(),
                                   _ptr(dev_status), _stream()), "rfp2_gemv_batched")
    return y


def hfp4_gemm_workspace_bytes(M: int, K: int) -> int:
    return int(lib().hfp4_gemm_workspace_bytes(M, K))


def hfp4_gemm(W, M, K, X, Y=None, workspace=None, dev_status=None):
    """HFP4G32 prefill GEMM on tensor cores: Y fp32 [N, M] = X (bf16 [N, K]) W^T."""
    torch = _torch()
    _need(W, torch.uint8, "W")
    if X.dtype == torch.bfloat16:
        X = X.view(torch.int16)
    if X.dtype not in (torch.int16, torch.uint16):
        raise TypeError("X must be bfloat16 (or its 16-bit pattern)")
    _need(X, X.dtype, "X")
    N = X.shape[0]
    Y = _empty((N, M), torch.float32, X) if Y is None else _need(Y, torch.float32, "Y")
    ws = _workspace(workspace, hfp4_gemm_workspace_bytes(M, K), X)
    _check(lib().hfp4_gemm(_ptr(W), M, K, _ptr(X), N, _ptr(Y), _ptr(ws), ws.numel(),
                           _ptr(dev_status), _stream()), "hfp4_gemm")
    return Y


def rfp2_nvfp4_weight_bytes(M: int, K: int) -> int:
    return int(lib().rfp2_nvfp4_weight_bytes(M, K))


def rfp2_to_nvfp4(W, M, K, out=None):
    """Exact NVFP4 image of packed ROCmFP2 weights: uint8 [rfp2_nvfp4_weight_bytes]
    (E2M1 codes [M, K/2], then scale bytes [M, K/16])."""
    torch = _torch()
    _need(W, torch.uint8, "W")
    n = rfp2_nvfp4_weight_bytes(M, K)
    out = torch.empty(n, dtype=torch.uint8, device=W.device) if out is None else _need(out, torch.uint8, "out")
    _check(lib().rfp2_to_nvfp4(_ptr(W), M, K, _ptr(out), _stream()), "rfp2_to_nvfp4")
    return out


def rfp2_gemm_nvfp4_workspace_bytes(N: int, K: int) -> int:
    return int(lib().rfp2_gemm_nvfp4_workspace_bytes(N, K))


def rfp2_gemm_nvfp4(Wnv, M, K, X, Y=None, workspace=None, dev_status=None):
    """NVFP4 prefill GEMM on the FP4 tensor cores: Y fp32 [N, M] = NVFP4(X) Wnv^T
    (X bf16 [N, K] quantized per token into the workspace)."""
    torch = _torch()
    _need(Wnv, torch.uint8, "Wnv")
    if X.dtype == torch.bfloat16:
        X = X.view(torch.int16)
    if X.dtype not in (torch.int16, torch.uint16):
        raise TypeError("X must be bfloat16 (or its 16-bit pattern)")
    _need(X, X.dtype, "X")
    N = X.shape[0]
    Y = _empty((N, M), torch.float32, X) if Y is None else _need(Y, torch.float32, "Y")
    ws = _workspace(workspace, rfp2_gemm_nvfp4_workspace_bytes(N, K), X)
    _check(lib().rfp2_gemm_nvfp4(_ptr(Wnv), M, K, _ptr(X), N, _ptr(Y), _ptr(ws), ws.numel(),
                                 _ptr(dev_status), _stream()), "rfp2_gemm_nvfp4")
    return Y


def hfp4_gemv_workspace_bytes(N: int, K: int) -> int:
    return int(lib().hfp4_gemv_workspace_bytes(N, K))


def hfp4_gemv(W, M, K, x, y=None, workspace=None, dev_status=None):
    """HFP4G32 GEMV: y fp32 [N, M]."""
    torch = _torch()
    _need(W, torch.uint8, "W")
    _need(x, torch.float32, "x")
    N = x.shape[0]
    y = _empty((N, M), torch.float32, x) if y is None else _need(y, torch.float32, "y")
    ws = _workspace(workspace, hfp4_gemv_workspace_bytes(N, K), x)
    _check(lib().hfp4_gemv(_ptr(W), M, K, _ptr(x), N, _ptr(y), _ptr(ws), ws.numel(),
                           _ptr(dev_status), _stream()), "hfp4_gemv")
    return y


def rfp2_pack_weights(W, out=None):
    """fp32 W [M, K] -> ROCmFP2 blocks uint8 [M, K/32, 10] (bit-identical to the oracle)."""
    torch = _torch()
    _need(W, torch.float32, "W")
    M, K = W.shape
    out = _empty((M, K // 32, 10), torch.uint8, W) if out is None else _need(out, torch.uint8, "out")
    _check(lib().rfp2_pack_weights(_ptr(W), M, K, _ptr(out), _stream()), "rfp2_pack_weights")
    return out


def rfp2_pack_weights_weighted(W, importance, out=None):
    """fp32 W [M, K] and importance fp32 [K] -> ROCmFP2 blocks uint8 [M, K/32, 10]
    with the importance-weighted scale search."""
    torch = _torch()
    _need(W, torch.float32, "W")
    _need(importance, torch.float32, "importance")
    M, K = W.shape
    if importance.numel() != K:
        raise ValueError("importance needs one value per column")
    out = (_empty((M, K // 32, 10), torch.uint8, W) if out is None
           else _need(out, torch.uint8, "out"))
    _check(lib().rfp2_pack_weights_weighted(_ptr(W), M, K, _ptr(importance), _ptr(out),
                                            _stream()), "rfp2_pack_weights_weighted")
    return out


def hfp4_pack_weights(W, out=None, dev_status=None):
    """fp32 W [M, K] -> HFP4G32 rows uint8 [M, 16 + 17*K/32]."""
    torch = _torch()
    _need(W, torch.float32, "W")
    M, K = W.shape
    out = (_empty((M, hfp4_row_bytes(K)), torch.uint8, W) if out is None
           else _need(out, torch.uint8, "out"))
    _check(lib().hfp4_pack_weights(_ptr(W), M, K, _ptr(out), _ptr(dev_status), _stream()),
           "hfp4_pack_weights")
    return out


def rfp2_validate_weights(W, dev_status=None):
    """Count of scale bytes >= 0x7F, as a device int64 tensor of one element."""
    torch = _torch()
    _need(W, torch.uint8, "W")
    bad = torch.zeros(1, dtype=torch.int64, device=W.device)
    _check(lib().rfp2_validate_weights(_ptr(W), W.numel() // 10, _ptr(bad), _ptr(dev_status),
                                       _stream()), "rfp2_validate_weights")
    return bad


def rfp2_debug_half_partials(W, M, K, q, partials=None):
    """int32 half sums [N, M, K/16] of the GEMV's integer path."""
    torch = _torch()
    _need(W, torch.uint8, "W")
    _need(q, torch.int8, "q")
    N = q.shape[0]
    partials = (_empty((N, M, K // 16), torch.int32, q) if partials is None
                else _need(partials, torch.int32, "partials"))
    _check(lib().rfp2_debug_half_partials(_ptr(W), M, K, _ptr(q), N, _ptr(partials), _stream()),
           "rfp2_debug_half_partials")
    return partials


def rfp2_debug_wait_timeout(dev_status):
    """Run the bounded-wait test hook: dev_status (device int32 [1]) gets
    RFP2_ETIMEOUT after the library's wait limit."""
    torch = _torch()
    _need(dev_status, torch.int32, "dev_status")
    _check(lib().rfp2_debug_wait_timeout(_ptr(dev_status), _stream()), "rfp2_debug_wait_timeout")
    return dev_status


# -- attention between the products -----------------------------------------------------
#
# A decode step makes these calls for every layer, each a few microseconds on the GPU; their
# arguments are checked and read by _rfp2_binding (csrc/binding.cpp), in less time than that.

_ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "ramp": 3}
_ROPE_INTERLEAVED, _ROPE_INVERSE = 1, 2
_ATTN_ZERO_BYTES = 4096
_native = None
_rope_function = None


class KVCache(NamedTuple):
    """A paged key-value cache in Q8 blocks: codes int8 [pages, heads, page_size, D] and scales
    fp32 [pages, heads, page_size, D/32], for keys and for values.  Calls take any such four."""
    k_codes: Any
    k_scales: Any
    v_codes: Any
    v_scales: Any


def _binding():
    """The loaded binding module (raises if it is not built)."""
    global _native
    if _native is None:
        _torch()
        lib()
        from . import buildlib as _b
        if not os.path.exists(_b.BINDING) or not _b.binding_fits():
            raise RuntimeError(f"no binding is built for {_b.binding_for()} ({_b.BINDING}); run gemm_rocmfp2_mul_gb300.build()")
        spec = importlib.util.spec_from_file_location("_rfp2_binding", _b.BINDING)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _native = module
    return _native


def rfp2_rope_frequencies(R, base=10000.0, scaling="plain", stretch=1.0, trained=4096.0, fast=32.0,
                          slow=1.0, device="cuda"):
    """Rotary frequencies for R rotated values: (inv_freq fp32 [R/2] on `device`, factor).
    scaling: "plain", "linear" (all divided by stretch), "base" (a larger base) or "ramp" (by the
    pair's turns over the `trained` length; factor = 0.1 ln(stretch) + 1)."""
    torch = _torch()
    f = torch.empty(max(R // 2, 0), dtype=torch.float32)
    factor = C.c_float()
    _check(lib().rfp2_rope_frequencies(R, base, _ROPE_SCALINGS[scaling], stretch, trained, fast, slow,
                                       f.data_ptr(), C.addressof(factor)), "rfp2_rope_frequencies")
    return f.to(device), factor.value


def rfp2_rope(x, positions, inv_freq, out=None, interleaved=False, inverse=False, factor=1.0):
    """Rotary positions: x [T, H, D] (any token and head strides) with the first 2*len(inv_freq)
    values of each head rotated by positions int32 [T]; out=x rotates in place.  inverse=True
    negates the angles (the gradient).  A gradient of x goes through the call, unless `out` is given:
    that is refused where x requires one."""
    if out is None:
        if x.requires_grad and _torch().is_grad_enabled():
            return _rope_with_gradient().apply(x, positions, inv_freq, interleaved, inverse, factor)
        out = _empty(x.shape, x.dtype, x)
    rc = (_native or _binding()).rope(
        x, positions, inv_freq, out,
        (_ROPE_INTERLEAVED if interleaved else 0) | (_ROPE_INVERSE if inverse else 0), factor)
    if rc:
        raise RFP2Error(rc, "rfp2_rope")
    return out


def _rope_with_gradient():
    """rfp2_rope as a function of autograd: the gradient turns back."""
    global _rope_function
    if _rope_function is None:
        class RotaryPositions(_torch().autograd.Function):
            @staticmethod
            def forward(ctx, x, positions, inv_freq, interleaved, inverse, factor):
                ctx.save_for_backward(positions, inv_freq)
                ctx.how = interleaved, inverse, factor
                return rfp2_rope(x, positions, inv_freq, None, interleaved, inverse, factor)

            @staticmethod
            def backward(ctx, gy):
                positions, inv_freq = ctx.saved_tensors
                interleaved, inverse, factor = ctx.how
                if gy.stride(-1) != 1:
                    gy = gy.contiguous()
                return rfp2_rope(gy, positions, inv_freq, None, interleaved, not inverse, factor), *[None] * 5

        _rope_function = RotaryPositions
    return _rope_function


def rfp2_kv_alloc(pages, heads, page_size, D, device="cuda"):
    """A zeroed KVCache of `pages` pages."""
    torch = _torch()
    return KVCache(*(torch.zeros((pages, heads, page_size, n), dtype=dtype, device=device)
                     for n, dtype in ((D, torch.int8), (D // 32, torch.float32)) * 2))


def rfp2_kv_write(cache, k, v, slots, positions=None, inv_freq=None, interleaved=False, factor=1.0,
                  dev_status=None):
    """Quantise k, v [T, heads, D] into the cache at slots int64 [T] (page * page_size + offset;
    -1 leaves a token out).  With positions and inv_freq, k is rotated on the way in.  Like the other calls
    over the cache, it has no gradient."""
    rc = (_native or _binding()).kv_write(cache, k, v, slots, positions, inv_freq,
                                          _ROPE_INTERLEAVED if interleaved else 0, factor, dev_status)
    if rc:
        raise RFP2Error(rc, "rfp2_kv_write")


def rfp2_kv_read(cache, slots, dtype=None, k=None, v=None, dev_status=None):
    """The values at slots int64 [T]: (k, v), each [T, heads, D] of `dtype` (fp32 unless given;
    or the type of the k and v passed to be filled).  A slot of -1 reads as zeros."""
    if k is None or v is None:
        torch = _torch()
        like = k if k is not None else v
        dtype = dtype or (like.dtype if like is not None else torch.float32)
        shape = (slots.numel(), cache[0].shape[1], cache[0].shape[3])
        k = _empty(shape, dtype, slots) if k is None else k
        v = _empty(shape, dtype, slots) if v is None else v
    rc = (_native or _binding()).kv_read(cache, slots, k, v, dev_status)
    if rc:
        raise RFP2Error(rc, "rfp2_kv_read")
    return k, v


def rfp2_attn_decode_workspace_bytes(B: int, nq: int, Hq: int, heads: int, D: int) -> int:
    return int(lib().rfp2_attn_decode_workspace_bytes(B, nq, Hq, heads, D))


def rfp2_attn_decode_workspace(q, heads):
    """A workspace for rfp2_attn_decode of q [B, nq, Hq, D] over `heads` key heads, its head zeroed;
    calls in one stream may share it."""
    if q.get_device() != _torch().cuda.current_device():
        raise ValueError("q must be on the current device")
    B, nq, Hq, D = q.shape
    workspace = _empty(max(rfp2_attn_decode_workspace_bytes(B, nq, Hq, heads, D), _ATTN_ZERO_BYTES),
                       _torch().uint8, q)
    workspace[:_ATTN_ZERO_BYTES].zero_()
    return workspace


def rfp2_attn_decode(q, cache, table, lens, scale=None, window=0, softcap=0.0, out=None, lse=None,
                     workspace=None, dev_status=None):
    """Attention of each sequence's newest tokens over the paged cache: q [B, nq, Hq, D], table int32
    [B, width] of pages, lens int32 [B] of keys held (the nq newest among them).  Returns out
    [B, nq, Hq, D] of q's type (out=q, contiguous, writes in place) and lse fp32 [B, nq, Hq].
    scale: D**-0.5 unless given; window: only the
    last `window` keys (0: all); softcap: scores become softcap * tanh(s / softcap) (0: as they are).
    workspace: from rfp2_attn_decode_workspace.  No sequence (B = 0) is nothing to do.  There is no gradient."""
    if out is None or lse is None or workspace is None:
        if q.dim() != 4:
            raise ValueError(f"q must have 4 dimensions, got {q.dim()}")
        out = _empty(q.shape, q.dtype, q) if out is None else out
        lse = _empty(q.shape[:3], _torch().float32, q) if lse is None else lse
        workspace = rfp2_attn_decode_workspace(q, cache[0].shape[1]) if workspace is None else workspace
    rc = (_native or _binding()).attn_decode(q, cache, table, lens, scale, window, softcap, out, lse, workspace,
                                             dev_status)
    if rc:
        raise RFP2Error(rc, "rfp2_attn_decode")
    return out, lse
