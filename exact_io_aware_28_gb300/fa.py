"""ctypes binding of libfa_gb300.so (names as in include/fa.h).

Argument marshalling only: every step of the attention path runs in the library's
CUDA kernels.  torch supplies device memory and the current stream.  If the library
has not been built, every call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_gb300.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)
FA_BF16, FA_FP32 = 0, 1

# Every symbol include/fa.h declares.
EXPORTS = ("fa_fwd", "fa_bwd", "fa_bwd_workspace_bytes", "fa_bwd_preprocess", "fa_bwd_main",
           "fa_bwd_dq_convert", "fa_bwd_noalloc", "fa_status_string", "fa_device_error",
           "fa_selftest_wait_timeout", "fa_decode_workspace_bytes", "fa_decode",
           "fa_fp8_vt_bytes", "fa_fp8_quantize_qk", "fa_fp8_quantize_v", "fa_fwd_fp8",
           "fa_fwd_dropout", "fa_bwd_dropout", "fa_bwd_main_dropout", "fa_dropout_random_bytes",
           "fa_attn_merge", "fa_grad_accumulate", "fa_grad_finish",
           "fa_paged_tables", "fa_paged_append", "fa_decode_paged_workspace_bytes",
           "fa_decode_paged", "fa_latent_fwd", "fa_latent_bwd_workspace_bytes", "fa_latent_bwd",
           "fa_latent_append", "fa_latent_decode_workspace_bytes", "fa_latent_decode",
           "fa_decode_shared_workspace_bytes", "fa_decode_shared", "fa_paged_fork",
           "fa_paged_free", "fa_paged_compact", "fa_paged_copy", "fa_rope", "fa_rope_append")

# Columns of latent attention: the latent vector, the keys' rotated part, a head's own key part
# and its values.
LATENT_RANK, LATENT_ROPE, LATENT_NOPE, LATENT_V = 512, 64, 128, 128
LATENT_ROW, LATENT_QK = LATENT_RANK + LATENT_ROPE, LATENT_NOPE + LATENT_ROPE

# Largest number of partial results fa_attn_merge accepts.
FA_MERGE_MAX_PARTS = 1024

# Largest workspace (bytes) fa_bwd_noalloc can serve from its built-in scratch array.
FA_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fa_status_string(status)}")


_lib: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m exact_io_aware_28_gb300.build` (nvcc, sm_103a)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P, F, I, P]
    lib.fa_fwd.restype = I
    lib.fa_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, P, P, F, I, P, S, P]
    lib.fa_bwd.restype = I
    lib.fa_bwd_preprocess.argtypes = [P, P, I, I, I, I, I, P, S, P]
    lib.fa_bwd_preprocess.restype = I
    lib.fa_bwd_main.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, P, P, F, I, P, S, P]
    lib.fa_bwd_main.restype = I
    lib.fa_bwd_dq_convert.argtypes = [P, I, I, I, I, F, I, P, S, P]
    lib.fa_bwd_dq_convert.restype = I
    lib.fa_bwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, P, P, F, I, P]
    lib.fa_bwd_noalloc.restype = I
    lib.fa_bwd_workspace_bytes.argtypes = [I, I, I, I]
    lib.fa_bwd_workspace_bytes.restype = S
    lib.fa_status_string.argtypes = [I]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_device_error.argtypes = [P]
    lib.fa_device_error.restype = I
    lib.fa_selftest_wait_timeout.argtypes = [ctypes.c_uint, P]
    lib.fa_selftest_wait_timeout.restype = I
    lib.fa_decode_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.fa_decode_workspace_bytes.restype = S
    lib.fa_decode.argtypes = [P, P, P, P, P, I, I, I, I, I, P, F, P, S, P]
    lib.fa_decode.restype = I
    lib.fa_fp8_vt_bytes.argtypes = [I, I, I, I]
    lib.fa_fp8_vt_bytes.restype = S
    lib.fa_fp8_quantize_qk.argtypes = [P, P, P, I, I, I, I, P]
    lib.fa_fp8_quantize_qk.restype = I
    lib.fa_fp8_quantize_v.argtypes = [P, P, P, I, I, I, I, P]
    lib.fa_fp8_quantize_v.restype = I
    lib.fa_fwd_fp8.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, P, P, F, P]
    lib.fa_fwd_fp8.restype = I
    U64, U32 = ctypes.c_ulonglong, ctypes.c_uint
    lib.fa_fwd_dropout.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P, F, I, I, U64, U32, P]
    lib.fa_fwd_dropout.restype = I
    lib.fa_bwd_dropout.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, P, P, F, I, I, U64,
                                   U32, P, S, P]
    lib.fa_bwd_dropout.restype = I
    lib.fa_bwd_main_dropout.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, P, P, F, I, I,
                                        U64, U32, P, S, P]
    lib.fa_bwd_main_dropout.restype = I
    lib.fa_dropout_random_bytes.argtypes = [P, I, I, I, U64, U32, P]
    lib.fa_dropout_random_bytes.restype = I
    L = ctypes.c_longlong
    lib.fa_attn_merge.argtypes = [P, P, I, P, P, I, I, I, I, I, P]
    lib.fa_attn_merge.restype = I
    lib.fa_grad_accumulate.argtypes = [P, P, L, I, P]
    lib.fa_grad_accumulate.restype = I
    lib.fa_grad_finish.argtypes = [P, P, L, I, P]
    lib.fa_grad_finish.restype = I
    lib.fa_paged_tables.argtypes = [P, P, P, I, P, L, I, P, P, P, I, P, I, I, I, P]
    lib.fa_paged_tables.restype = I
    lib.fa_paged_append.argtypes = [P, P, L, L, P, P, L, P, I, I, I, I, I, P]
    lib.fa_paged_append.restype = I
    lib.fa_decode_paged_workspace_bytes.argtypes = [I, I, I, I]
    lib.fa_decode_paged_workspace_bytes.restype = S
    lib.fa_decode_paged.argtypes = [P, P, P, L, P, L, I, P, P, P, I, I, I, I, I, I, F, P, S, P]
    lib.fa_decode_paged.restype = I
    lib.fa_latent_fwd.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P, F, I, P]
    lib.fa_latent_fwd.restype = I
    lib.fa_latent_bwd_workspace_bytes.argtypes = [I, I, I]
    lib.fa_latent_bwd_workspace_bytes.restype = S
    lib.fa_latent_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, P, F, I, P, S, P]
    lib.fa_latent_bwd.restype = I
    lib.fa_latent_append.argtypes = [P, P, L, L, P, L, P, I, I, I, P]
    lib.fa_latent_append.restype = I
    lib.fa_latent_decode_workspace_bytes.argtypes = [I, I]
    lib.fa_latent_decode_workspace_bytes.restype = S
    lib.fa_latent_decode.argtypes = [P, P, L, P, L, I, P, P, P, I, I, I, I, F, P, S, P]
    lib.fa_latent_decode.restype = I
    lib.fa_decode_shared_workspace_bytes.argtypes = [I, I, I, I]
    lib.fa_decode_shared_workspace_bytes.restype = S
    lib.fa_decode_shared.argtypes = [P, P, P, L, P, L, I, P, P, P, I, P, P, I, I, I, I, I, I, F, P,
                                     S, P]
    lib.fa_decode_shared.restype = I
    lib.fa_paged_fork.argtypes = [P, P, L, I, P, I, P, P, I, P, P, P, P, I, I, I, P]
    lib.fa_paged_fork.restype = I
    lib.fa_paged_free.argtypes = [P, P, L, I, P, I, P, P, P, I, I, I, P]
    lib.fa_paged_free.restype = I
    lib.fa_paged_compact.argtypes = [P, P, L, I, P, P, P, I, P, I, I, I, P]
    lib.fa_paged_compact.restype = I
    lib.fa_paged_copy.argtypes = [P, P, L, P, P, P, I, I, I, I, I, P]
    lib.fa_paged_copy.restype = I
    lib.fa_rope.argtypes = [P, P, L, L, L, L, L, L, P, L, L, I, P, P, I, I, I, I, I, I, I, I, P]
    lib.fa_rope.restype = I
    lib.fa_rope_append.argtypes = [P, P, P, L, L, L, P, L, P, P, L, P, P, L, I, P, P, I, I, I, I, I,
                                   I, I, I, P]
    lib.fa_rope_append.restype = I
    _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]):
    """Device address of ``t`` for the library (every tensor argument is device memory)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("the library takes CUDA tensors (device memory); got a "
                         f"{t.device.type} tensor")
    return ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float32:
        return FA_FP32
    raise TypeError(f"unsupported dtype {t.dtype}: bf16 or fp32")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return ctypes.c_void_p(int(stream))


def _check_dense(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous [B, H, N, d]")


def fa_status_string(status: int) -> str:
    return load().fa_status_string(int(status)).decode()


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_bytes(B, H, N, d))


def fa_device_error(stream=None) -> int:
    return int(load().fa_device_error(_stream(stream)))


def fa_selftest_wait_timeout(limit_ms: int, stream=None) -> None:
    """Launch the bounded-wait self-test; fa_device_error() then reports FA_ERR_TIMEOUT."""
    st = load().fa_selftest_wait_timeout(int(limit_ms), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_selftest_wait_timeout")


def fa_fwd(q, k, v, o, lse, causal: bool = False, blockmask=None, kv_len=None,
           scale: Optional[float] = None, stream=None) -> None:
    """O and lse for [B, H, N, d] tensors q, k, v (outputs o, lse preallocated)."""
    _check_dense(q, k, v, o, lse, blockmask, kv_len)
    B, H, N, d = q.shape
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    st = load().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, int(causal),
                       _ptr(blockmask), _ptr(kv_len), scale, _dtype_code(q), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd")


def fa_bwd(q, k, v, o, lse, do, dq, dk, dv, workspace, causal: bool = False, blockmask=None,
           kv_len=None, scale: Optional[float] = None, stream=None) -> None:
    """dq, dk, dv (preallocated) for the upstream gradient ``do``."""
    _check_dense(q, k, v, o, lse, do, dq, dk, dv, blockmask, kv_len)
    B, H, N, d = q.shape
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = load().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq),
                       _ptr(dk), _ptr(dv), B, H, N, d, int(causal), _ptr(blockmask),
                       _ptr(kv_len), scale, _dtype_code(q), _ptr(workspace), ws_bytes,
                       _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd")


def fa_bwd_preprocess(o, do, workspace, stream=None) -> None:
    B, H, N, d = o.shape
    st = load().fa_bwd_preprocess(_ptr(o), _ptr(do), B, H, N, d, _dtype_code(o),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd_preprocess")


def fa_bwd_main(q, k, v, lse, do, dq, dk, dv, workspace, causal=False, blockmask=None,
                kv_len=None, scale=None, stream=None) -> None:
    _check_dense(q, k, v, lse, do, dq, dk, dv, blockmask, kv_len)
    B, H, N, d = q.shape
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    st = load().fa_bwd_main(_ptr(q), _ptr(k), _ptr(v), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
                            _ptr(dv), B, H, N, d, int(causal), _ptr(blockmask), _ptr(kv_len),
                            scale, _dtype_code(q), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd_main")


def fa_bwd_dq_convert(dq, workspace, scale=None, stream=None) -> None:
    B, H, N, d = dq.shape
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    st = load().fa_bwd_dq_convert(_ptr(dq), B, H, N, d, scale, _dtype_code(dq), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd_dq_convert")


def fa_bwd_noalloc(q, k, v, o, lse, do, dq, dk, dv, causal: bool = False, blockmask=None,
                   kv_len=None, scale: Optional[float] = None, stream=None) -> None:
    """fa_bwd with the library's built-in scratch array instead of a workspace.

    For callers that cannot allocate device memory.  Problems whose workspace would exceed
    FA_NOALLOC_SCRATCH_BYTES are rejected; calls that overlap on the GPU share the array
    and race, so serialise them.
    """
    _check_dense(q, k, v, o, lse, do, dq, dk, dv, blockmask, kv_len)
    B, H, N, d = q.shape
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    st = load().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
                               _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, int(causal),
                               _ptr(blockmask), _ptr(kv_len), scale, _dtype_code(q),
                               _stream(stream))
    if st != FA_OK:
        need = fa_bwd_workspace_bytes(B, H, N, d)
        if st == FA_ERR_UNSUPPORTED and need > FA_NOALLOC_SCRATCH_BYTES:
            raise FaError(st, f"fa_bwd_noalloc: needs {need} bytes of scratch, the built-in "
                              f"array holds {FA_NOALLOC_SCRATCH_BYTES}")
        raise FaError(st, "fa_bwd_noalloc")


# ----------------------------------------------------------- allocating helpers

def alloc_workspace(B: int, H: int, N: int, d: int, device="cuda") -> torch.Tensor:
    n = fa_bwd_workspace_bytes(B, H, N, d)
    if n == 0:
        raise FaError(FA_ERR_INVALID_ARG, "fa_bwd_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def forward(q, k, v, causal=False, blockmask=None, kv_len=None, scale=None, stream=None):
    """Allocate O and lse with torch and run fa_fwd.  Returns (o, lse)."""
    B, H, N, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fa_fwd(q, k, v, o, lse, causal, blockmask, kv_len, scale, stream)
    return o, lse


def backward(q, k, v, o, lse, do, causal=False, blockmask=None, kv_len=None, scale=None,
             workspace=None, stream=None):
    """Allocate dQ, dK, dV (and the workspace unless given) and run fa_bwd."""
    B, H, N, d = q.shape
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = alloc_workspace(B, H, N, d, q.device)
    fa_bwd(q, k, v, o, lse, do, dq, dk, dv, workspace, causal, blockmask, kv_len, scale, stream)
    return dq, dk, dv


# ----------------------------------------------------------- decode

def fa_decode_workspace_bytes(B: int, Hq: int, Hkv: int, Lmax: int, d: int) -> int:
    return int(load().fa_decode_workspace_bytes(B, Hq, Hkv, Lmax, d))


def fa_decode(q, k, v, o, lse, workspace, cache_len=None, scale=None, stream=None):
    """q [B, Hq, d], k/v [B, Hkv, Lmax, d] bf16; o [B, Hq, d] bf16, lse [B, Hq] fp32 out."""
    _check_dense(q, k, v, o, lse, cache_len, workspace)
    B, Hq, d = q.shape
    Hkv, Lmax = k.shape[1], k.shape[2]
    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError("decode takes bf16 q, k, v")
    if scale is None:
        scale = 1.0 / (d ** 0.5)
    st = load().fa_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Lmax, d,
                          _ptr(cache_len), float(scale), _ptr(workspace),
                          workspace.numel() * workspace.element_size(), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_decode")


def decode(q, k, v, cache_len=None, scale=None, workspace=None, stream=None):
    """Allocate o, lse (and the workspace unless given) with torch and run fa_decode."""
    B, Hq, d = q.shape
    Hkv, Lmax = k.shape[1], k.shape[2]
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = fa_decode_workspace_bytes(B, Hq, Hkv, Lmax, d)
        if n == 0:
            raise FaError(FA_ERR_INVALID_ARG, "fa_decode_workspace_bytes")
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    fa_decode(q, k, v, o, lse, workspace, cache_len, scale, stream)
    return o, lse


def fa_fp8_vt_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_fp8_vt_bytes(B, H, N, d))


def _need_bf16(*ts):
    for t in ts:
        if t.dtype != torch.bfloat16:
            raise TypeError("the FP8 encoders take bf16 tensors")


def fa_fp8_quantize_qk(x, x8, scale, stream=None) -> None:
    """x bf16 [B, H, N, 128] -> x8 uint8 [B, H, N, 128], scale fp32 [B, H, ceil(N/128)]."""
    _check_dense(x, x8, scale)
    _need_bf16(x)
    B, H, N, d = x.shape
    st = load().fa_fp8_quantize_qk(_ptr(x), _ptr(x8), _ptr(scale), B, H, N, d, _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fp8_quantize_qk")


def fa_fp8_quantize_v(v, vt8, scale, stream=None) -> None:
    """v bf16 [B, H, N, 128] -> vt8 uint8 [B, H, 128, Np] (opaque key order), scale [B, H]."""
    _check_dense(v, vt8, scale)
    _need_bf16(v)
    B, H, N, d = v.shape
    st = load().fa_fp8_quantize_v(_ptr(v), _ptr(vt8), _ptr(scale), B, H, N, d, _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fp8_quantize_v")


def fa_fwd_fp8(q8, k8, vt8, q_scale, k_scale, v_scale, o, lse, causal=False, blockmask=None,
               kv_len=None, scale=None, stream=None) -> None:
    """O (bf16, preallocated) and lse of attention on e4m3-encoded inputs."""
    _check_dense(q8, k8, vt8, q_scale, k_scale, v_scale, o, lse, blockmask, kv_len)
    B, H, N, d = q8.shape
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    st = load().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(vt8), _ptr(q_scale), _ptr(k_scale),
                           _ptr(v_scale), _ptr(o), _ptr(lse), B, H, N, d, int(causal),
                           _ptr(blockmask), _ptr(kv_len), scale, _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_fp8")


def fp8_quantize_qk(x, stream=None):
    """Allocate and encode: returns (x8 uint8 [B, H, N, 128], scale fp32 [B, H, nb])."""
    B, H, N, d = x.shape
    x8 = torch.empty((B, H, N, d), dtype=torch.uint8, device=x.device)
    scale = torch.empty((B, H, (N + 127) // 128), dtype=torch.float32, device=x.device)
    fa_fp8_quantize_qk(x, x8, scale, stream)
    return x8, scale


def fp8_quantize_v(v, stream=None):
    """Allocate and encode: returns (vt8 uint8 [B, H, 128, Np], scale fp32 [B, H])."""
    B, H, N, d = v.shape
    Np = (N + 127) // 128 * 128
    vt8 = torch.empty((B, H, d, Np), dtype=torch.uint8, device=v.device)
    scale = torch.empty((B, H), dtype=torch.float32, device=v.device)
    fa_fp8_quantize_v(v, vt8, scale, stream)
    return vt8, scale


def forward_fp8(q8, k8, vt8, q_scale, k_scale, v_scale, causal=False, blockmask=None,
                kv_len=None, scale=None, stream=None):
    """Allocate o (bf16) and lse with torch and run fa_fwd_fp8."""
    B, H, N, d = q8.shape
    o = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    fa_fwd_fp8(q8, k8, vt8, q_scale, k_scale, v_scale, o, lse, causal, blockmask, kv_len,
               scale, stream)
    return o, lse


def attention_fp8(q, k, v, causal=False, blockmask=None, kv_len=None, scale=None, stream=None):
    """bf16 q, k, v -> (o, lse) with e4m3 tensor-core products: encode, then the forward."""
    q8, sq = fp8_quantize_qk(q, stream)
    k8, sk = fp8_quantize_qk(k, stream)
    vt8, sv = fp8_quantize_v(v, stream)
    return forward_fp8(q8, k8, vt8, sq, sk, sv, causal, blockmask, kv_len, scale, stream)


# ----------------------------------------------------------- dropout

def _drop_args(drop_threshold: int, seed: int, offset: int):
    t = int(drop_threshold)
    if not 0 <= t <= 255:
        raise ValueError("drop_threshold must be in [0, 255] (drop probability t / 256)")
    return t, int(seed) & (2 ** 64 - 1), int(offset) & (2 ** 32 - 1)


def fa_fwd_dropout(q, k, v, o, lse, drop_threshold: int, seed: int, offset: int = 0,
                   causal: bool = False, blockmask=None, kv_len=None,
                   scale: Optional[float] = None, stream=None) -> None:
    """fa_fwd with dropout on P: element (b, h, i, j) is dropped with probability t / 256
    (its Philox4x32-10 byte below t), kept ones are scaled by 256 / (256 - t)."""
    _check_dense(q, k, v, o, lse, blockmask, kv_len)
    B, H, N, d = q.shape
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    t, sd, off = _drop_args(drop_threshold, seed, offset)
    st = load().fa_fwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                               int(causal), _ptr(blockmask), _ptr(kv_len), scale,
                               _dtype_code(q), t, sd, off, _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_dropout")


def fa_bwd_dropout(q, k, v, o, lse, do, dq, dk, dv, workspace, drop_threshold: int, seed: int,
                   offset: int = 0, causal: bool = False, blockmask=None, kv_len=None,
                   scale: Optional[float] = None, stream=None) -> None:
    """Gradients of the dropped forward; the same (threshold, seed, offset) regenerate the
    mask."""
    _check_dense(q, k, v, o, lse, do, dq, dk, dv, blockmask, kv_len)
    B, H, N, d = q.shape
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    t, sd, off = _drop_args(drop_threshold, seed, offset)
    st = load().fa_bwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
                               _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, int(causal),
                               _ptr(blockmask), _ptr(kv_len), scale, _dtype_code(q), t, sd, off,
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd_dropout")


def fa_bwd_main_dropout(q, k, v, lse, do, dq, dk, dv, workspace, drop_threshold: int,
                        seed: int, offset: int = 0, causal=False, blockmask=None, kv_len=None,
                        scale=None, stream=None) -> None:
    _check_dense(q, k, v, lse, do, dq, dk, dv, blockmask, kv_len)
    B, H, N, d = q.shape
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    t, sd, off = _drop_args(drop_threshold, seed, offset)
    st = load().fa_bwd_main_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(lse), _ptr(do), _ptr(dq),
                                    _ptr(dk), _ptr(dv), B, H, N, d, int(causal),
                                    _ptr(blockmask), _ptr(kv_len), scale, _dtype_code(q), t, sd,
                                    off, _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd_main_dropout")


def fa_dropout_random_bytes(out, seed: int, offset: int = 0, stream=None) -> None:
    """The generator byte of every element of a [BH, n_q, n_k] uint8 tensor ``out``."""
    if out.dtype != torch.uint8 or out.dim() != 3 or not out.is_contiguous():
        raise ValueError("out must be a contiguous uint8 [BH, n_q, n_k] tensor")
    BH, n_q, n_k = out.shape
    _, sd, off = _drop_args(0, seed, offset)
    st = load().fa_dropout_random_bytes(_ptr(out), BH, n_q, n_k, sd, off, _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_dropout_random_bytes")


def forward_dropout(q, k, v, drop_threshold, seed, offset=0, causal=False, blockmask=None,
                    kv_len=None, scale=None, stream=None):
    """Allocate O and lse with torch and run fa_fwd_dropout.  Returns (o, lse)."""
    B, H, N, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fa_fwd_dropout(q, k, v, o, lse, drop_threshold, seed, offset, causal, blockmask, kv_len,
                   scale, stream)
    return o, lse


def backward_dropout(q, k, v, o, lse, do, drop_threshold, seed, offset=0, causal=False,
                     blockmask=None, kv_len=None, scale=None, workspace=None, stream=None):
    """Allocate dQ, dK, dV (and the workspace unless given) and run fa_bwd_dropout."""
    B, H, N, d = q.shape
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = alloc_workspace(B, H, N, d, q.device)
    fa_bwd_dropout(q, k, v, o, lse, do, dq, dk, dv, workspace, drop_threshold, seed, offset,
                   causal, blockmask, kv_len, scale, stream)
    return dq, dk, dv


# ----------------------------------------------------------- sequence sharding

def fa_attn_merge(o_parts, lse_parts, o, lse, stream=None) -> None:
    """Merge S partial (O, lse) results of the same rows over disjoint key sets:
    o_parts [S, B, H, N, d], lse_parts fp32 [S, B, H, N] -> o [B, H, N, d], lse [B, H, N]."""
    _check_dense(o_parts, lse_parts, o, lse)
    S, B, H, N, d = o_parts.shape
    if tuple(lse_parts.shape) != (S, B, H, N) or lse_parts.dtype != torch.float32:
        raise ValueError("lse_parts must be fp32 [S, B, H, N]")
    if o.dtype != o_parts.dtype:
        raise TypeError("o and o_parts must have the same dtype")
    st = load().fa_attn_merge(_ptr(o_parts), _ptr(lse_parts), S, _ptr(o), _ptr(lse), B, H, N, d,
                              _dtype_code(o_parts), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_attn_merge")


def fa_grad_accumulate(acc, x, stream=None) -> None:
    """acc (fp32) += x (bf16 or fp32, same number of elements)."""
    _check_dense(acc, x)
    if acc.dtype != torch.float32 or acc.numel() != x.numel():
        raise ValueError("acc must be fp32 with as many elements as x")
    st = load().fa_grad_accumulate(_ptr(acc), _ptr(x), acc.numel(), _dtype_code(x),
                                   _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_grad_accumulate")


def fa_grad_finish(out, acc, stream=None) -> None:
    """out (bf16 or fp32) = acc (fp32) rounded once."""
    _check_dense(acc, out)
    if acc.dtype != torch.float32 or acc.numel() != out.numel():
        raise ValueError("acc must be fp32 with as many elements as out")
    st = load().fa_grad_finish(_ptr(out), _ptr(acc), acc.numel(), _dtype_code(out),
                               _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_grad_finish")


# ----------------------------------------------------------- paged cache

def _same_gpu(stream, *ts) -> int:
    """Every tensor lies on the current CUDA device, where the library launches; returns the
    handle of ``stream`` (None: the device's current stream)."""
    here = ts[0].get_device()
    for t in ts:
        if t.get_device() != here or here < 0:
            bad = next((t for t in ts if not t.is_cuda), None)
            if bad is not None:
                raise ValueError("the library takes CUDA tensors (device memory); got a "
                                 f"{bad.device.type} tensor")
            raise ValueError(f"tensors on {ts[0].device} and {t.device}: one device a call")
    if here != torch._C._cuda_getDevice():     # the tensors are there: CUDA is initialised
        raise ValueError(f"tensors on {ts[0].device}, but the current device is cuda:"
                         f"{torch.cuda.current_device()}: enter torch.cuda.device(...) for them")
    if stream is None:
        # the handle alone: making a Stream object of it takes longer than the launch
        return torch._C._cuda_getCurrentRawStream(here)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _shaped(name, t, shape, dtype):
    """``t`` is dense and has the shape and type named."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _scratch(t):
    """The workspace has the bytes that it counts (an expanded tensor counts some more often)."""
    if not t.is_contiguous() and t.numel() > 1 + sum((n - 1) * st for n, st in zip(t.shape,
                                                                                t.stride())):
        raise ValueError("workspace must be contiguous: it counts bytes that it does not have")


def _rows(name, t, shape, dtype=torch.bfloat16):
    """Elements between the first index's entries of ``t``, whose other dimensions are dense (a
    slice of a larger tensor along them is taken as it is)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    st, dense, whole = t.stride(), 1, True
    for i in range(len(shape) - 1, 0, -1):
        if st[i] != dense and shape[i] != 1:
            whole = False
        dense *= shape[i]
    if not whole and not t.is_contiguous():      # (an empty tensor is, whatever its strides)
        raise ValueError(f"{name} must be dense behind its first dimension")
    return st[0] if whole and shape[0] > 1 else dense   # a single entry's stride says nothing


def _table(t, B):
    shape = t.shape
    if t.dtype is not torch.int32:
        raise TypeError("block_table must be torch.int32")
    if len(shape) != 2 or shape[0] != B or shape[1] < 1:
        raise ValueError(f"block_table must be [{B}, max_pages], not {list(shape)}")
    if t.is_contiguous():
        return shape[1]
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("block_table rows must be dense")
    return t.stride(0) if B > 1 else shape[1]   # a single row's stride says nothing


def _on_stream(stream, fn, *args, **kw):
    """A helper on a stream that was named: what it allocates belongs to that stream, and tensors made
    on another are kept until its work is done."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    if stream != torch.cuda.current_stream():
        for x in (*args, *kw.values()):
            for t in x if isinstance(x, (tuple, list)) else (x,):
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(stream)
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def fa_paged_tables(cache_len, new_len, free_pages, block_table, total_len, token_start, slots,
                    pages_taken, page_size: int, num_pages: int, stream=None) -> None:
    """Block tables and slot maps from the requests' lengths (int32 tensors throughout).

    cache_len, new_len [B], free_pages [F] in; block_table [B, max_pages] in and out; out:
    total_len [B], token_start [B + 1], slots [T], pages_taken [1].
    """
    B, i32 = cache_len.numel(), torch.int32
    F, T = free_pages.numel(), slots.numel()
    _shaped("cache_len", cache_len, (B,), i32)
    _shaped("new_len", new_len, (B,), i32)
    _shaped("free_pages", free_pages, (F,), i32)
    _shaped("total_len", total_len, (B,), i32)
    _shaped("token_start", token_start, (B + 1,), i32)
    _shaped("slots", slots, (T,), i32)
    _shaped("pages_taken", pages_taken, (1,), i32)
    stride = _table(block_table, B)
    handle = _same_gpu(stream, cache_len, new_len, free_pages, block_table, total_len,
                       token_start, slots, pages_taken)
    st = load().fa_paged_tables(cache_len.data_ptr(), new_len.data_ptr(), free_pages.data_ptr(),
                                F, block_table.data_ptr(), stride, block_table.shape[1],
                                total_len.data_ptr(), token_start.data_ptr(), slots.data_ptr(), T,
                                pages_taken.data_ptr(), B, page_size, num_pages, handle)
    if st != FA_OK:
        raise FaError(st, "fa_paged_tables")


def paged_tables(cache_len, new_len, free_pages, block_table, page_size: int, num_pages: int,
                 num_slots: int, stream=None):
    """Allocate the outputs and run fa_paged_tables; block_table is updated in place.

    Returns (total_len, token_start, slots, pages_taken); ``num_slots`` rows of slots, those
    behind the last new token -1.
    """
    if stream is not None:
        return _on_stream(stream, paged_tables, cache_len, new_len, free_pages, block_table,
                          page_size, num_pages, num_slots)
    B = cache_len.numel()
    buf = torch.empty(2 * B + 2 + num_slots, dtype=torch.int32, device=cache_len.device)
    total, start, taken, slots = buf.split((B, B + 1, 1, num_slots))
    fa_paged_tables(cache_len, new_len, free_pages, block_table, total, start, slots, taken,
                    page_size, num_pages)
    return total, start, slots, taken


def fa_paged_append(k, v, k_cache, v_cache, slots, stream=None) -> None:
    """Rows k, v [T, Hkv, d] (bf16, any stride between tokens) into slots [T] (int32) of the pools
    k_cache, v_cache [num_pages, Hkv, page_size, d] (equal strides)."""
    rows, pool = k.shape, k_cache.shape
    if len(rows) != 3 or len(pool) != 4 or pool[1] != rows[1] or pool[3] != rows[2]:
        raise ValueError("k must be [T, Hkv, d] and k_cache [num_pages, Hkv, page_size, d]; got "
                         f"{list(rows)} and {list(pool)}")
    T, Hkv, d = rows
    ks, vs = _rows("k", k, rows), _rows("v", v, rows)
    kp = _rows("k_cache", k_cache, pool)
    if kp != _rows("v_cache", v_cache, pool):
        raise ValueError("k_cache and v_cache must have the same stride between pages")
    _shaped("slots", slots, (T,), torch.int32)
    handle = _same_gpu(stream, k, v, k_cache, v_cache, slots)
    st = load().fa_paged_append(k.data_ptr(), v.data_ptr(), ks, vs, k_cache.data_ptr(),
                                v_cache.data_ptr(), kp, slots.data_ptr(), T, pool[0], Hkv,
                                pool[2], d, handle)
    if st != FA_OK:
        raise FaError(st, "fa_paged_append")


def paged_append(k, v, k_cache, v_cache, slots, stream=None) -> None:
    """fa_paged_append; on a ``stream`` that is named, the tensors' memory is kept until its work is
    done."""
    if stream is not None:
        return _on_stream(stream, paged_append, k, v, k_cache, v_cache, slots)
    fa_paged_append(k, v, k_cache, v_cache, slots)


def fa_decode_paged_workspace_bytes(B: int, Hq: int, Hkv: int, d: int) -> int:
    return int(load().fa_decode_paged_workspace_bytes(B, Hq, Hkv, d))


def alloc_decode_paged_workspace(B: int, Hq: int, Hkv: int, d: int, device="cuda"):
    n = fa_decode_paged_workspace_bytes(B, Hq, Hkv, d)
    if n == 0:
        raise FaError(FA_ERR_INVALID_ARG, "fa_decode_paged_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def fa_decode_paged(q, k, v, block_table, cache_len, o, lse, workspace, scale=None,
                    stream=None) -> None:
    """q [B, Hq, d] over the pools k, v [num_pages, Hkv, page_size, d] (bf16) through block_table
    [B, max_pages] and cache_len [B] (int32); o [B, Hq, d] bf16 and lse [B, Hq] fp32 out."""
    heads, pool = q.shape, k.shape
    if len(heads) != 3 or len(pool) != 4 or pool[3] != heads[2]:
        raise ValueError("q must be [B, Hq, d] and k [num_pages, Hkv, page_size, d]; got "
                         f"{list(heads)} and {list(pool)}")
    B, Hq, d = heads
    P, Hkv, page, _ = pool
    _shaped("q", q, heads, torch.bfloat16)
    kp = _rows("k", k, pool)
    if kp != _rows("v", v, pool):
        raise ValueError("k and v must have the same stride between pages")
    stride = _table(block_table, B)
    _shaped("cache_len", cache_len, (B,), torch.int32)
    _shaped("o", o, heads, torch.bfloat16)
    _shaped("lse", lse, (B, Hq), torch.float32)
    _scratch(workspace)
    handle = _same_gpu(stream, q, k, v, block_table, cache_len, o, lse, workspace)
    st = load().fa_decode_paged(q.data_ptr(), k.data_ptr(), v.data_ptr(), kp,
                                block_table.data_ptr(), stride, block_table.shape[1],
                                cache_len.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hkv, P,
                                page, d, 1.0 / d ** 0.5 if scale is None else scale,
                                workspace.data_ptr(), workspace.nbytes, handle)
    if st != FA_OK:
        raise FaError(st, "fa_decode_paged")


def decode_paged(q, k, v, block_table, cache_len, scale=None, workspace=None, stream=None):
    """Allocate o, lse (and the workspace unless given) and run fa_decode_paged."""
    if stream is not None:
        return _on_stream(stream, decode_paged, q, k, v, block_table, cache_len, scale, workspace)
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_decode_paged_workspace(*q.shape[:2], k.shape[1], q.shape[2], q.device)
    fa_decode_paged(q, k, v, block_table, cache_len, o, lse, workspace, scale)
    return o, lse


# ----------------------------------------------------------- shared prefixes

def fa_decode_shared_workspace_bytes(B: int, Hq: int, Hkv: int, d: int) -> int:
    return int(load().fa_decode_shared_workspace_bytes(B, Hq, Hkv, d))


def alloc_decode_shared_workspace(B: int, Hq: int, Hkv: int, d: int, device="cuda"):
    n = fa_decode_shared_workspace_bytes(B, Hq, Hkv, d)
    if n == 0:
        raise FaError(FA_ERR_INVALID_ARG, "fa_decode_shared_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _shared_inputs(q, k, v, block_table, cache_len, group_start, shared_len):
    """Checks; returns what fa_decode_shared is called with, in its order, but for the outputs."""
    heads, pool = q.shape, k.shape
    if len(heads) != 3 or len(pool) != 4 or pool[3] != heads[2]:
        raise ValueError("q must be [B, Hq, d] and k [num_pages, Hkv, page_size, d]; got "
                         f"{list(heads)} and {list(pool)}")
    B, Hq, d = heads
    P, Hkv, page, _ = pool
    groups = shared_len.numel()
    _shaped("q", q, heads, torch.bfloat16)
    kp = _rows("k", k, pool)
    if kp != _rows("v", v, pool):
        raise ValueError("k and v must have the same stride between pages")
    stride = _table(block_table, B)
    _shaped("cache_len", cache_len, (B,), torch.int32)
    _shaped("shared_len", shared_len, (groups,), torch.int32)
    _shaped("group_start", group_start, (groups + 1,), torch.int32)
    return ((q.data_ptr(), k.data_ptr(), v.data_ptr(), kp, block_table.data_ptr(), stride,
             block_table.shape[1], cache_len.data_ptr(), group_start.data_ptr(),
             shared_len.data_ptr(), groups), (B, Hq, Hkv, P, page, d))


def _shared_call(ins, sizes, o, lse, workspace, scale, handle):
    st = load().fa_decode_shared(*ins, o.data_ptr(), lse.data_ptr(), *sizes,
                                 1.0 / sizes[5] ** 0.5 if scale is None else scale,
                                 workspace.data_ptr(), workspace.nbytes, handle)
    if st != FA_OK:
        raise FaError(st, "fa_decode_shared")


def fa_decode_shared(q, k, v, block_table, cache_len, group_start, shared_len, o, lse, workspace,
                     scale=None, stream=None) -> None:
    """fa_decode_paged for groups of sequences with a prefix in common: group p are the sequences
    group_start[p] .. group_start[p + 1] - 1 (int32 [groups + 1]), whose first shared_len[p] tokens
    (int32 [groups]) are in the same pages."""
    ins, sizes = _shared_inputs(q, k, v, block_table, cache_len, group_start, shared_len)
    _shaped("o", o, q.shape, torch.bfloat16)
    _shaped("lse", lse, sizes[:2], torch.float32)
    _scratch(workspace)
    handle = _same_gpu(stream, q, k, v, block_table, cache_len, group_start, shared_len, o, lse,
                       workspace)
    _shared_call(ins, sizes, o, lse, workspace, scale, handle)


def decode_shared(q, k, v, block_table, cache_len, group_start, shared_len, scale=None,
                  workspace=None, stream=None):
    """Allocate o, lse (and the workspace unless given) and run fa_decode_shared."""
    if stream is not None:
        return _on_stream(stream, decode_shared, q, k, v, block_table, cache_len, group_start,
                          shared_len, scale, workspace)
    ins, sizes = _shared_inputs(q, k, v, block_table, cache_len, group_start, shared_len)
    if workspace is None:
        handle = _same_gpu(None, q, k, v, block_table, cache_len, group_start, shared_len)
        workspace = alloc_decode_shared_workspace(*sizes[:3], sizes[5], q.device)
    else:
        _scratch(workspace)
        handle = _same_gpu(None, q, k, v, block_table, cache_len, group_start, shared_len,
                           workspace)
    o = torch.empty_like(q)
    lse = torch.empty(sizes[:2], dtype=torch.float32, device=q.device)
    _shared_call(ins, sizes, o, lse, workspace, scale, handle)
    return o, lse


# ----------------------------------------------------------- pages

def _i32(name, t, n):
    """``t`` is dense int32 [n]; its address."""
    if t.dtype is torch.int32 and t.shape == (n,) and t.is_contiguous():
        return t.data_ptr()
    return _shaped(name, t, (n,), torch.int32)     # raises


def _lists(device, *sizes):
    """New int32 lists.  (Between launches an allocation takes 3 us of the host, a split of one 7.)"""
    return tuple([torch.empty(n, dtype=torch.int32, device=device) for n in sizes])


def _call(name, *args):
    st = getattr(load(), name)(*args)
    if st != FA_OK:
        raise FaError(st, name)


def fa_paged_fork(cache_len, block_table, free_pages, src, dst, copy_src, copy_dst, copy_rows,
                  pages_taken, page_size: int, num_pages: int, stream=None) -> None:
    """Requests dst[i] become copies of src[i] (int32 tensors throughout): cache_len [B] and
    block_table [B, max_pages] in and out, free_pages [F] in; out: what fa_paged_copy is to copy,
    copy_src, copy_dst, copy_rows [n], and pages_taken [1]."""
    B, F, n = cache_len.numel(), free_pages.numel(), src.numel()
    lens, free = _i32("cache_len", cache_len, B), _i32("free_pages", free_pages, F)
    pairs = _i32("src", src, n), _i32("dst", dst, n)
    outs = (_i32("copy_src", copy_src, n), _i32("copy_dst", copy_dst, n),
            _i32("copy_rows", copy_rows, n), _i32("pages_taken", pages_taken, 1))
    stride = _table(block_table, B)
    handle = _same_gpu(stream, cache_len, block_table, free_pages, src, dst, copy_src, copy_dst,
                       copy_rows, pages_taken)
    _call("fa_paged_fork", lens, block_table.data_ptr(), stride, block_table.shape[1], free, F,
          *pairs, n, *outs, B, page_size, num_pages, handle)


def paged_fork(cache_len, block_table, free_pages, src, dst, page_size: int, num_pages: int,
               stream=None):
    """Allocate the lists and run fa_paged_fork; cache_len and block_table are updated in place.
    Returns (copy_src, copy_dst, copy_rows, pages_taken)."""
    if stream is not None:
        return _on_stream(stream, paged_fork, cache_len, block_table, free_pages, src, dst,
                          page_size, num_pages)
    B, F, n = cache_len.numel(), free_pages.numel(), src.numel()
    lens, free = _i32("cache_len", cache_len, B), _i32("free_pages", free_pages, F)
    pairs = _i32("src", src, n), _i32("dst", dst, n)
    stride = _table(block_table, B)
    handle = _same_gpu(None, cache_len, block_table, free_pages, src, dst)
    outs = _lists(src.device, n, n, n, 1)
    _call("fa_paged_fork", lens, block_table.data_ptr(), stride, block_table.shape[1], free, F,
          *pairs, n, *[t.data_ptr() for t in outs], B, page_size, num_pages, handle)
    return outs


def fa_paged_free(cache_len, block_table, rows, refs, free_pages, n_free, page_size: int,
                  num_pages: int, stream=None) -> None:
    """Requests rows [n] end (int32 tensors throughout): cache_len [B] and block_table
    [B, max_pages] in and out; out: refs and free_pages [num_pages], n_free [1]."""
    B, n = cache_len.numel(), rows.numel()
    lens, ended = _i32("cache_len", cache_len, B), _i32("rows", rows, n)
    outs = (_i32("refs", refs, num_pages), _i32("free_pages", free_pages, num_pages),
            _i32("n_free", n_free, 1))
    stride = _table(block_table, B)
    handle = _same_gpu(stream, cache_len, block_table, rows, refs, free_pages, n_free)
    _call("fa_paged_free", lens, block_table.data_ptr(), stride, block_table.shape[1], ended, n,
          *outs, B, page_size, num_pages, handle)


def paged_free(cache_len, block_table, rows, page_size: int, num_pages: int, stream=None):
    """Allocate the outputs and run fa_paged_free; cache_len and block_table are updated in place.
    Returns (refs, free_pages, n_free)."""
    if stream is not None:
        return _on_stream(stream, paged_free, cache_len, block_table, rows, page_size, num_pages)
    B, n = cache_len.numel(), rows.numel()
    lens, ended = _i32("cache_len", cache_len, B), _i32("rows", rows, n)
    stride = _table(block_table, B)
    handle = _same_gpu(None, cache_len, block_table, rows)
    outs = _lists(cache_len.device, num_pages, num_pages, 1)
    _call("fa_paged_free", lens, block_table.data_ptr(), stride, block_table.shape[1], ended, n,
          *[t.data_ptr() for t in outs], B, page_size, num_pages, handle)
    return outs


def fa_paged_compact(cache_len, block_table, moved, copy_src, copy_dst, n_used, page_size: int,
                     num_pages: int, stream=None) -> None:
    """The pages in use move to the front of the pool (int32 tensors throughout): cache_len [B] in,
    block_table [B, max_pages] in and out; out: moved [num_pages], copy_src and copy_dst (at least
    num_pages / 2 each), n_used [1]."""
    B, n = cache_len.numel(), copy_src.numel()
    lens, new = _i32("cache_len", cache_len, B), _i32("moved", moved, num_pages)
    frm, to = _i32("copy_src", copy_src, n), _i32("copy_dst", copy_dst, n)
    used, stride = _i32("n_used", n_used, 1), _table(block_table, B)
    handle = _same_gpu(stream, cache_len, block_table, moved, copy_src, copy_dst, n_used)
    _call("fa_paged_compact", lens, block_table.data_ptr(), stride, block_table.shape[1], new, frm,
          to, n, used, B, page_size, num_pages, handle)


def paged_compact(cache_len, block_table, page_size: int, num_pages: int, stream=None):
    """Allocate the outputs and run fa_paged_compact; block_table is updated in place.
    Returns (moved, copy_src, copy_dst, n_used), the copies for paged_copy."""
    if stream is not None:
        return _on_stream(stream, paged_compact, cache_len, block_table, page_size, num_pages)
    B, n = cache_len.numel(), max(1, num_pages // 2)
    lens, stride = _i32("cache_len", cache_len, B), _table(block_table, B)
    handle = _same_gpu(None, cache_len, block_table)
    outs = _lists(cache_len.device, num_pages, n, n, 1)
    moved, frm, to, used = [t.data_ptr() for t in outs]
    _call("fa_paged_compact", lens, block_table.data_ptr(), stride, block_table.shape[1], moved, frm,
          to, n, used, B, page_size, num_pages, handle)
    return outs


def fa_paged_copy(k_cache, v_cache, copy_src, copy_dst, copy_rows=None, stream=None) -> None:
    """Pages copy_src[i] to copy_dst[i] (int32 [n]), or their first copy_rows[i] rows, in the bf16
    pools k_cache, v_cache [num_pages, Hkv, page_size, d] (v_cache may be None) or in a latent one
    [num_pages, page_size, 576]."""
    pool, n = k_cache.shape, copy_src.numel()
    if len(pool) == 3:
        stride, heads = _latent_pool(k_cache), 1
    elif len(pool) == 4:
        stride, heads = _rows("k_cache", k_cache, pool), pool[1]
    else:
        raise ValueError("k_cache must be [num_pages, Hkv, page_size, d] or a latent cache, not "
                         f"{list(pool)}")
    if v_cache is not None and _rows("v_cache", v_cache, pool) != stride:
        raise ValueError("k_cache and v_cache must have the same stride between pages")
    frm, to = _i32("copy_src", copy_src, n), _i32("copy_dst", copy_dst, n)
    rows = None if copy_rows is None else _i32("copy_rows", copy_rows, n)
    handle = _same_gpu(stream, *_given(k_cache, v_cache, copy_src, copy_dst, copy_rows))
    _call("fa_paged_copy", k_cache.data_ptr(), _at(v_cache), stride, frm, to, rows, n, pool[0],
          heads, pool[-2], pool[-1], handle)


def paged_copy(k_cache, v_cache, copy_src, copy_dst, copy_rows=None, stream=None) -> None:
    """fa_paged_copy; on a ``stream`` that is named, the tensors' memory is kept until its work is
    done."""
    if stream is not None:
        return _on_stream(stream, paged_copy, k_cache, v_cache, copy_src, copy_dst, copy_rows)
    fa_paged_copy(k_cache, v_cache, copy_src, copy_dst, copy_rows)


# ----------------------------------------------------------- rotary positions

def rope_table(rot: int, base: float = 10000.0, sections=None, frequencies=None, device="cuda"):
    """The plan of a rotation of ``rot`` channels: (turns int64 [rot / 2], axis int32 [rot / 2]).

    Pair i turns by base ** (-2 i / rot) radians a position, or by ``frequencies[i]``, on the axis
    whose part of ``sections`` (pairs of each axis, in order; default: one axis) it lies in.
    """
    pairs = rot // 2
    if frequencies is None:
        frequencies = [float(base) ** (-2.0 * i / rot) for i in range(pairs)]
    else:
        frequencies = [float(f) for f in frequencies]
    sections = [pairs] if sections is None else [int(n) for n in sections]
    if rot % 2 or len(frequencies) != pairs or sum(sections) != pairs or min(sections) < 0:
        raise ValueError(f"{pairs} pairs: as many frequencies, and sections that add up to them")
    turns = []
    for f in frequencies:
        t = f / (2.0 * math.pi)
        if not math.isfinite(t):
            raise ValueError("frequencies must be finite")
        u = round(math.fmod(t, 1.0) * 2.0 ** 64) % 2 ** 64   # modulo a full turn, all bits of t kept
        turns.append(u - 2 ** 64 if u >= 2 ** 63 else u)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    return (torch.tensor(turns, dtype=torch.int64, device=device),
            torch.tensor(axis, dtype=torch.int32, device=device))


def _plan(table):
    turns, axis = table
    pairs = turns.numel()
    _shaped("turns", turns, (pairs,), torch.int64)
    _shaped("axis", axis, (pairs,), torch.int32)
    return turns, axis, 2 * pairs


def _rope(x, y, pos, table, interleaved, inverse, stream):
    """fa_rope; y None: into a new tensor, which is returned."""
    shape = x.shape
    if len(shape) != 4:
        raise ValueError(f"x must be [B, H, N, d], not {list(shape)}")
    B, H, N, d = shape
    code, xs, ps = _dtype_code(x), x.stride(), pos.stride()
    if d > 1 and xs[3] != 1:
        raise ValueError("rows of x must be dense")
    if pos.dtype is not torch.int32:
        raise TypeError("pos must be torch.int32")
    if pos.dim() != 3 or pos.shape[1:] != (B, N) or (N > 1 and ps[2] != 1):
        raise ValueError(f"pos must be [axes, {B}, {N}], dense along the last, not "
                         f"{list(pos.shape)}")
    turns, axis, rot = _plan(table)
    if y is None:
        handle = _same_gpu(stream, x, pos, turns, axis)
        y = torch.empty(shape, dtype=x.dtype, device=x.device)
        ys = (H * N * d, N * d, d)
    else:
        ys = y.stride()
        if y.shape != shape or y.dtype != x.dtype:
            raise ValueError(f"y must be {list(shape)} of {x.dtype}, as x is")
        if d > 1 and ys[3] != 1:
            raise ValueError("rows of y must be dense")
        handle = _same_gpu(stream, x, y, pos, turns, axis)
    _call("fa_rope", x.data_ptr(), y.data_ptr(), *xs[:3], *ys[:3], pos.data_ptr(), ps[0], ps[1],
          pos.shape[0], turns.data_ptr(), axis.data_ptr(), B, H, N, d, rot, int(interleaved),
          int(inverse), code, handle)
    return y


def fa_rope(x, y, pos, table, interleaved: bool = False, inverse: bool = False,
            stream=None) -> None:
    """Rows of x [B, H, N, d] (bf16 or fp32; any strides, rows dense) turned into y by their
    positions pos int32 [axes, B, N]; ``table`` as of rope_table.  y may be x."""
    _rope(x, y, pos, table, interleaved, inverse, stream)


def rope(x, pos, table, interleaved: bool = False, out=None, stream=None):
    """Rotary positions: x [B, H, N, d] turned, into ``out`` (which may be x) or a new tensor."""
    if stream is not None:
        return _on_stream(stream, rope, x, pos, table, interleaved, out)
    return _rope(x, out, pos, table, interleaved, False, None)


def rope_backward(dy, pos, table, interleaved: bool = False, out=None, stream=None):
    """The gradient of rope: dy turned back, into ``out`` (which may be dy) or a new tensor."""
    if stream is not None:
        return _on_stream(stream, rope_backward, dy, pos, table, interleaved, out)
    return _rope(dy, out, pos, table, interleaved, True, None)


def fa_rope_append(q, k, v, pos, table, q_out, k_cache, v_cache, slots, interleaved: bool = False,
                   stream=None) -> None:
    """The rows of T new tokens: q [T, Hq, d] turned into q_out (which may be q), k [T, Hkv, d] turned
    and v as it is into slots [T] (int32) of the pools k_cache, v_cache [num_pages, Hkv, page_size,
    d]; bf16, any stride between tokens; positions pos int32 [axes, T], ``table`` as of
    rope_table."""
    rows, heads, pool = k.shape, q.shape, k_cache.shape
    if (len(rows) != 3 or len(heads) != 3 or len(pool) != 4 or pool[1] != rows[1]
            or pool[3] != rows[2] or heads[0] != rows[0] or heads[2] != rows[2]):
        raise ValueError("q must be [T, Hq, d], k [T, Hkv, d] and k_cache [num_pages, Hkv, "
                         f"page_size, d]; got {list(heads)}, {list(rows)} and {list(pool)}")
    T, Hkv, d = rows
    qs, ks, vs = _rows("q", q, heads), _rows("k", k, rows), _rows("v", v, rows)
    qo, kp = _rows("q_out", q_out, heads), _rows("k_cache", k_cache, pool)
    if kp != _rows("v_cache", v_cache, pool):
        raise ValueError("k_cache and v_cache must have the same stride between pages")
    slot = _i32("slots", slots, T)
    if pos.dtype is not torch.int32:
        raise TypeError("pos must be torch.int32")
    if pos.dim() != 2 or pos.shape[1] != T or (T > 1 and pos.stride(1) != 1):
        raise ValueError(f"pos must be [axes, {T}], dense along the last, not {list(pos.shape)}")
    turns, axis, rot = _plan(table)
    handle = _same_gpu(stream, q, k, v, pos, turns, axis, q_out, k_cache, v_cache, slots)
    _call("fa_rope_append", q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, q_out.data_ptr(),
          qo, k_cache.data_ptr(), v_cache.data_ptr(), kp, slot, pos.data_ptr(), pos.stride(0),
          pos.shape[0], turns.data_ptr(), axis.data_ptr(), T, heads[1], Hkv, pool[0], pool[2], d,
          rot, int(interleaved), handle)


def rope_append(q, k, v, pos, table, k_cache, v_cache, slots, interleaved: bool = False, out=None,
                stream=None):
    """Run fa_rope_append; returns the turned queries, in ``out`` (which may be q) or a new
    tensor."""
    if stream is not None:
        return _on_stream(stream, rope_append, q, k, v, pos, table, k_cache, v_cache, slots,
                          interleaved, out)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    fa_rope_append(q, k, v, pos, table, out, k_cache, v_cache, slots, interleaved)
    return out


# ----------------------------------------------------------- latent attention

def _latent_shapes(q, k_nope, k_rope, v, kv_len):
    if q.dim() != 4:
        raise ValueError(f"q must be [B, H, N, {LATENT_QK}], not {list(q.shape)}")
    B, H, N, _ = q.shape
    code, dt = _dtype_code(q), q.dtype
    _shaped("q", q, (B, H, N, LATENT_QK), dt)
    _shaped("k_nope", k_nope, (B, H, N, LATENT_NOPE), dt)
    _shaped("k_rope", k_rope, (B, N, LATENT_ROPE), dt)
    _shaped("v", v, (B, H, N, LATENT_V), dt)
    if kv_len is not None:
        _shaped("kv_len", kv_len, (B,), torch.int32)
    return B, H, N, code


def _given(*ts):
    return (t for t in ts if t is not None)


def _at(t):
    return None if t is None else t.data_ptr()


def fa_latent_fwd(q, k_nope, k_rope, v, o, o_acc, lse, causal: bool = False, kv_len=None,
                  scale: Optional[float] = None, stream=None) -> None:
    """Expanded latent attention: q [B, H, N, 192], k_nope [B, H, N, 128], k_rope [B, N, 64] shared
    by the heads, v [B, H, N, 128]; out o (as v), o_acc (fp32 O for the backward, or None) and
    lse fp32 [B, H, N]."""
    B, H, N, code = _latent_shapes(q, k_nope, k_rope, v, kv_len)
    _shaped("o", o, (B, H, N, LATENT_V), q.dtype)
    if o_acc is not None:
        _shaped("o_acc", o_acc, (B, H, N, LATENT_V), torch.float32)
    _shaped("lse", lse, (B, H, N), torch.float32)
    handle = _same_gpu(stream, *_given(q, k_nope, k_rope, v, o, o_acc, lse, kv_len))
    st = load().fa_latent_fwd(q.data_ptr(), k_nope.data_ptr(), k_rope.data_ptr(), v.data_ptr(),
                              o.data_ptr(), _at(o_acc), lse.data_ptr(), B, H, N, int(causal),
                              _at(kv_len), 1.0 / LATENT_QK ** 0.5 if scale is None else scale,
                              code, handle)
    if st != FA_OK:
        raise FaError(st, "fa_latent_fwd")


def latent_forward(q, k_nope, k_rope, v, causal: bool = False, kv_len=None, scale=None,
                   need_grad: bool = False, stream=None):
    """Allocate and run fa_latent_fwd.  Returns (o, lse), with ``need_grad`` (o, lse, o_acc)."""
    if stream is not None:
        return _on_stream(stream, latent_forward, q, k_nope, k_rope, v, causal, kv_len, scale,
                          need_grad)
    o, o_acc = torch.empty_like(v), None
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    if need_grad and q.dtype != torch.float32:
        o_acc = torch.empty(v.shape, dtype=torch.float32, device=q.device)
    fa_latent_fwd(q, k_nope, k_rope, v, o, o_acc, lse, causal, kv_len, scale)
    if not need_grad:
        return o, lse
    return o, lse, o if o_acc is None else o_acc   # fp32: o is its own unrounded form


def fa_latent_bwd_workspace_bytes(B: int, H: int, N: int) -> int:
    return int(load().fa_latent_bwd_workspace_bytes(B, H, N))


def alloc_latent_workspace(B: int, H: int, N: int, device="cuda") -> torch.Tensor:
    n = fa_latent_bwd_workspace_bytes(B, H, N)
    if n == 0:
        raise FaError(FA_ERR_INVALID_ARG, "fa_latent_bwd_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def fa_latent_bwd(q, k_nope, k_rope, v, o_acc, lse, do, dq, dk_nope, dk_rope, dv, workspace,
                  causal: bool = False, kv_len=None, scale: Optional[float] = None,
                  stream=None) -> None:
    """Gradients of fa_latent_fwd (preallocated) for the upstream gradient ``do``; o_acc and lse
    as the forward wrote them."""
    B, H, N, code = _latent_shapes(q, k_nope, k_rope, v, kv_len)
    _shaped("o_acc", o_acc, (B, H, N, LATENT_V), torch.float32)
    _shaped("lse", lse, (B, H, N), torch.float32)
    for name, t, like in (("do", do, v), ("dq", dq, q), ("dk_nope", dk_nope, k_nope),
                          ("dk_rope", dk_rope, k_rope), ("dv", dv, v)):
        _shaped(name, t, like.shape, q.dtype)
    _scratch(workspace)
    handle = _same_gpu(stream, *_given(q, k_nope, k_rope, v, o_acc, lse, do, dq, dk_nope, dk_rope,
                                       dv, workspace, kv_len))
    st = load().fa_latent_bwd(q.data_ptr(), k_nope.data_ptr(), k_rope.data_ptr(), v.data_ptr(),
                              o_acc.data_ptr(), lse.data_ptr(), do.data_ptr(), dq.data_ptr(),
                              dk_nope.data_ptr(), dk_rope.data_ptr(), dv.data_ptr(), B, H, N,
                              int(causal), _at(kv_len),
                              1.0 / LATENT_QK ** 0.5 if scale is None else scale, code,
                              workspace.data_ptr(), workspace.nbytes, handle)
    if st != FA_OK:
        raise FaError(st, "fa_latent_bwd")


def latent_backward(q, k_nope, k_rope, v, o_acc, lse, do, causal: bool = False, kv_len=None,
                    scale=None, workspace=None, stream=None):
    """Allocate the gradients (and the workspace unless given) and run fa_latent_bwd.
    Returns (dq, dk_nope, dk_rope, dv)."""
    if stream is not None:
        return _on_stream(stream, latent_backward, q, k_nope, k_rope, v, o_acc, lse, do, causal,
                          kv_len, scale, workspace)
    dq, dkn, dkr, dv = (torch.empty_like(t) for t in (q, k_nope, k_rope, v))
    if workspace is None:
        workspace = alloc_latent_workspace(*q.shape[:3], q.device)
    fa_latent_bwd(q, k_nope, k_rope, v, o_acc, lse, do, dq, dkn, dkr, dv, workspace, causal,
                  kv_len, scale)
    return dq, dkn, dkr, dv


def _latent_pool(cache):
    shape = cache.shape
    if len(shape) != 3 or shape[2] != LATENT_ROW:
        raise ValueError(f"cache must be [num_pages, page_size, {LATENT_ROW}], not {list(shape)}")
    return _rows("cache", cache, shape)


def fa_latent_append(c, k_rope, cache, slots, stream=None) -> None:
    """Latent rows c [T, 512] and k_rope [T, 64] (bf16, any stride between tokens) into slots [T]
    (int32) of the pool cache [num_pages, page_size, 576]."""
    T, ps = slots.numel(), _latent_pool(cache)
    cs, rs = _rows("c", c, (T, LATENT_RANK)), _rows("k_rope", k_rope, (T, LATENT_ROPE))
    _shaped("slots", slots, (T,), torch.int32)
    handle = _same_gpu(stream, c, k_rope, cache, slots)
    st = load().fa_latent_append(c.data_ptr(), k_rope.data_ptr(), cs, rs, cache.data_ptr(), ps,
                                 slots.data_ptr(), T, cache.shape[0], cache.shape[1], handle)
    if st != FA_OK:
        raise FaError(st, "fa_latent_append")


def latent_append(c, k_rope, cache, slots, stream=None) -> None:
    """fa_latent_append; on a ``stream`` that is named, the tensors' memory is kept until its work is
    done."""
    if stream is not None:
        return _on_stream(stream, latent_append, c, k_rope, cache, slots)
    fa_latent_append(c, k_rope, cache, slots)


def fa_latent_decode_workspace_bytes(B: int, H: int) -> int:
    return int(load().fa_latent_decode_workspace_bytes(B, H))


def alloc_latent_decode_workspace(B: int, H: int, device="cuda") -> torch.Tensor:
    n = fa_latent_decode_workspace_bytes(B, H)
    if n == 0:
        raise FaError(FA_ERR_INVALID_ARG, "fa_latent_decode_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def fa_latent_decode(q, cache, block_table, cache_len, o, lse, workspace, scale=None,
                     stream=None) -> None:
    """Absorbed latent decode: q [B, H, 576] over the pool cache [num_pages, page_size, 576]
    (bf16) through block_table [B, max_pages] and cache_len [B] (int32); o [B, H, 512] bf16 and
    lse [B, H] fp32 out."""
    if q.dim() != 3 or q.shape[2] != LATENT_ROW:
        raise ValueError(f"q must be [B, H, {LATENT_ROW}], not {list(q.shape)}")
    B, H, _ = q.shape
    _shaped("q", q, q.shape, torch.bfloat16)
    ps, stride = _latent_pool(cache), _table(block_table, B)
    _shaped("cache_len", cache_len, (B,), torch.int32)
    _shaped("o", o, (B, H, LATENT_RANK), torch.bfloat16)
    _shaped("lse", lse, (B, H), torch.float32)
    _scratch(workspace)
    handle = _same_gpu(stream, q, cache, block_table, cache_len, o, lse, workspace)
    st = load().fa_latent_decode(q.data_ptr(), cache.data_ptr(), ps, block_table.data_ptr(), stride,
                                 block_table.shape[1], cache_len.data_ptr(), o.data_ptr(),
                                 lse.data_ptr(), B, H, cache.shape[0], cache.shape[1],
                                 1.0 / LATENT_QK ** 0.5 if scale is None else scale,
                                 workspace.data_ptr(), workspace.nbytes, handle)
    if st != FA_OK:
        raise FaError(st, "fa_latent_decode")


def latent_decode(q, cache, block_table, cache_len, scale=None, workspace=None, stream=None):
    """Allocate o, lse (and the workspace unless given) and run fa_latent_decode."""
    if stream is not None:
        return _on_stream(stream, latent_decode, q, cache, block_table, cache_len, scale,
                          workspace)
    B, H = q.shape[:2]
    o = torch.empty((B, H, LATENT_RANK), dtype=q.dtype, device=q.device)
    lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_latent_decode_workspace(B, H, q.device)
    fa_latent_decode(q, cache, block_table, cache_len, o, lse, workspace, scale)
    return o, lse
