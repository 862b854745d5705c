"""Fused rank-sum + residual add + RMSNorm for one GB300 (sm_103a).

    reduced      = sum over ranks r of x[r]            (bf16 [T,H] each)
    residual_out = reduced + residual
    norm_out     = RMSNorm(residual_out, weight, eps)

The operator of FlagTree pull request "[TLERaw] Add NVSHMEM allreduce
RMSNorm tutorial" (Summary; Implementation sections 2-3), computed by the
hand-written CUDA kernels of ``libfarn.so``.  This module is the Python
binding of that library's C ABI (``include/farn.h``): the ``farn_*``
functions have the C names and arguments and only marshal them through
ctypes; ``forward`` is the same call for torch tensors.  Next to it stand
the operators of an expert layer and of NVFP4 projections that its outputs
go through: ``moe_route``, ``grouped_matmul`` and ``moe_combine``;
``nvfp4_quantize``, ``nvfp4_dequantize`` and ``nvfp4_matmul``;
``fp8_quantize``, ``fp8_matmul`` and ``fp8_grouped_matmul``; and those of the
attention half up to the cache, ``qk_norm_rope``, ``qk_norm_rope_cache``,
``kv_write`` and ``kv_read``.  Every
arithmetic step runs in the CUDA kernels.  There is no CPU fallback: if the library
is not built, every call raises.

A call runs on torch's current stream, or on ``stream``, and waits for no other:
its inputs have to be ready there, and to stay as they are until it has run.  What
it makes itself on a given stream (outputs that are not given, a workspace) lies in
that stream's memory; the outputs may be used on the stream that was current at the
call, once that waits for it, and dropped at any time.
"""
from __future__ import annotations

import ctypes
import os

from ._build import LIB_PATH, build_library

__all__ = [
    "FARN_MAX_W", "FarnError", "Context", "build_library", "library_path",
    "farn_create", "farn_destroy", "farn_forward", "farn_check_args",
    "farn_plan", "farn_status_string", "farn_device_status", "farn_forward_noalloc",
    "farn_forward_typed", "farn_plan_typed", "farn_forward_quant", "forward_quant",
    "farn_moe_combine", "moe_combine",
    "FARN_MAX_EXPERTS", "farn_moe_route", "moe_route",
    "farn_grouped_matmul", "grouped_matmul",
    "farn_nvfp4_quantize", "nvfp4_quantize", "farn_nvfp4_dequantize", "nvfp4_dequantize",
    "farn_nvfp4_matmul", "nvfp4_matmul",
    "farn_plan_grouped_matmul", "farn_plan_nvfp4_matmul",
    "farn_fp8_quantize", "fp8_quantize", "farn_fp8_matmul", "fp8_matmul",
    "farn_fp8_grouped_matmul", "fp8_grouped_matmul", "farn_fp8_grouped_workspace",
    "farn_plan_fp8_matmul", "farn_plan_fp8_grouped_matmul",
    "FARN_CACHE_FP8", "FARN_CACHE_NVFP4", "KvCache", "kv_cache",
    "farn_qk_norm_rope", "qk_norm_rope", "farn_qk_norm_rope_cache", "qk_norm_rope_cache",
    "farn_kv_write", "kv_write", "farn_kv_read", "kv_read",
    "FARN_BF16", "FARN_F32",
    "forward", "VARIANTS",
]

FARN_MAX_W = 32
FARN_MAX_EXPERTS = 1024
FARN_OK = 0
FARN_ERR_INVALID_ARG = -1
FARN_ERR_UNSUPPORTED = -2
FARN_ERR_ALIAS = -3
FARN_ERR_CUDA = -4
FARN_ERR_NOMEM = -5
VARIANTS = {0: "row", 1: "cluster", 2: "generic", 3: "bulk", 4: "stage", 5: "combine",
            6: "tensor", 7: "pair"}
FARN_BF16, FARN_F32 = 0, 1
FARN_CACHE_FP8, FARN_CACHE_NVFP4 = 1, 2


class KvCache(ctypes.Structure):
    """C ``farn_kv_cache``: a paged cache of keys and values, as raw device
    addresses."""
    _fields_ = [("format", ctypes.c_int), ("page_size", ctypes.c_int),
                ("n_pages", ctypes.c_int64), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("k_tensor_scale", ctypes.c_float), ("v_tensor_scale", ctypes.c_float)]


_lib = None


def library_path() -> str:
    return LIB_PATH


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built (the operator has no CPU fallback); "
                "run rank_sum_residual_gb300.build_library() on a machine with nvcc")
        lib = ctypes.CDLL(LIB_PATH)
        vp, cvp = ctypes.c_void_p, ctypes.c_void_p
        pvp = ctypes.POINTER(ctypes.c_void_p)
        i64, i32, f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_float
        lib.farn_create.argtypes = [ctypes.POINTER(ctypes.c_void_p), i32]
        lib.farn_create.restype = i32
        lib.farn_destroy.argtypes = [vp]
        lib.farn_destroy.restype = i32
        lib.farn_forward.argtypes = [vp, pvp, i32, cvp, cvp, f32, i64, i64,
                                     vp, vp, vp, vp]
        lib.farn_forward.restype = i32
        lib.farn_forward_typed.argtypes = [vp, pvp, i32, i32, cvp, cvp, f32, i64, i64,
                                           vp, vp, vp, vp]
        lib.farn_forward_typed.restype = i32
        lib.farn_forward_quant.argtypes = [vp, pvp, i32, i32, cvp, cvp, f32, i64, i64,
                                           vp, vp, vp, vp, vp, vp]
        lib.farn_forward_quant.restype = i32
        lib.farn_forward_nvfp4.argtypes = [vp, pvp, i32, i32, cvp, cvp, f32, i64, i64, f32,
                                           vp, vp, vp, vp, vp, vp]
        lib.farn_forward_nvfp4.restype = i32
        lib.farn_moe_combine.argtypes = [vp, cvp, i64, cvp, cvp, i32, cvp, cvp, f32, i64, i64,
                                         vp, vp, vp, vp]
        lib.farn_moe_combine.restype = i32
        lib.farn_moe_route.argtypes = [vp, cvp, i32, i64, i32, i32, i32, vp, vp, vp, vp, vp, vp]
        lib.farn_moe_route.restype = i32
        lib.farn_grouped_matmul.argtypes = [vp, cvp, i64, cvp, i64, cvp, i32, cvp, i64, i64, vp,
                                            vp]
        lib.farn_grouped_matmul.restype = i32
        lib.farn_nvfp4_quantize.argtypes = [vp, cvp, i64, i64, f32, vp, vp, vp]
        lib.farn_nvfp4_quantize.restype = i32
        lib.farn_nvfp4_dequantize.argtypes = [vp, cvp, cvp, i64, i64, f32, vp, vp]
        lib.farn_nvfp4_dequantize.restype = i32
        lib.farn_nvfp4_matmul.argtypes = [vp, cvp, cvp, f32, cvp, cvp, f32, i64, i64, i64, vp, vp]
        lib.farn_nvfp4_matmul.restype = i32
        pi = ctypes.POINTER(i32)
        lib.farn_plan_grouped_matmul.argtypes = [vp, cvp, i64, cvp, i64, cvp, i32, i64, i64, cvp,
                                                 pi, pi, pi]
        lib.farn_plan_grouped_matmul.restype = i32
        lib.farn_plan_nvfp4_matmul.argtypes = [vp, cvp, cvp, cvp, cvp, i64, i64, i64, cvp, pi, pi,
                                               pi]
        lib.farn_plan_nvfp4_matmul.restype = i32
        lib.farn_fp8_quantize.argtypes = [vp, cvp, i64, i64, i64, i32, vp, vp, vp]
        lib.farn_fp8_quantize.restype = i32
        lib.farn_fp8_matmul.argtypes = [vp, cvp, cvp, cvp, cvp, i64, i64, i64, vp, vp]
        lib.farn_fp8_matmul.restype = i32
        lib.farn_fp8_grouped_matmul.argtypes = [vp, cvp, cvp, i64, cvp, i64, cvp, cvp, i32, cvp,
                                                i64, i64, vp, vp, i64, vp]
        lib.farn_fp8_grouped_workspace.argtypes = [vp, i64, i32, i64, i64, ctypes.POINTER(i64)]
        lib.farn_fp8_grouped_workspace.restype = i32
        lib.farn_plan_fp8_matmul.argtypes = [vp, cvp, cvp, i64, i64, i64, cvp, pi, pi, pi]
        lib.farn_plan_fp8_matmul.restype = i32
        lib.farn_plan_fp8_grouped_matmul.argtypes = [vp, cvp, i64, cvp, i64, cvp, i32, i64, i64,
                                                     cvp, cvp, pi, pi, pi]
        lib.farn_plan_fp8_grouped_matmul.restype = i32
        lib.farn_fp8_grouped_matmul.restype = i32
        pc = vp     # a KvCache by reference: see _cache_ref
        rope = [cvp, cvp, f32, cvp, i32, pi, cvp, i32, i32]
        lib.farn_qk_norm_rope.argtypes = [vp, i64, i32, cvp, i32, i64, cvp, i32, i64, *rope, vp,
                                          i64, vp, i64, vp]
        lib.farn_qk_norm_rope.restype = i32
        lib.farn_qk_norm_rope_cache.argtypes = [vp, i64, i32, cvp, i32, i64, cvp, i64, cvp, i64,
                                                i32, *rope, vp, i64, pc, cvp, vp]
        lib.farn_qk_norm_rope_cache.restype = i32
        lib.farn_kv_write.argtypes = [vp, i64, cvp, i64, cvp, i64, pc, cvp, vp]
        lib.farn_kv_write.restype = i32
        lib.farn_kv_read.argtypes = [vp, pc, cvp, i32, i64, cvp, i64, vp, vp, vp]
        lib.farn_kv_read.restype = i32
        lib.farn_check_args.argtypes = [pvp, i32, cvp, cvp, f32, i64, i64,
                                        cvp, cvp, cvp]
        lib.farn_check_args.restype = i32
        lib.farn_plan.argtypes = [vp, i32, i64, i64, pvp, cvp, cvp, cvp, cvp,
                                  cvp, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                  ctypes.POINTER(i32)]
        lib.farn_plan.restype = i32
        lib.farn_plan_typed.argtypes = [vp, i32, i32, i32, i64, i64, pvp, cvp, cvp, cvp,
                                        cvp, cvp, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                        ctypes.POINTER(i32)]
        lib.farn_plan_typed.restype = i32
        lib.farn_plan_moe_combine.argtypes = [vp, i32, i64, i64, cvp, cvp, cvp, cvp, cvp, cvp,
                                              ctypes.POINTER(i32), ctypes.POINTER(i32)]
        lib.farn_plan_moe_combine.restype = i32
        lib.farn_forward_noalloc.argtypes = [i32, pvp, i32, cvp, cvp, f32, i64, i64,
                                             vp, vp, vp, vp, ctypes.POINTER(i32)]
        lib.farn_forward_noalloc.restype = i32
        lib.farn_device_status.argtypes = [vp, ctypes.POINTER(i32)]
        lib.farn_device_status.restype = i32
        lib.farn_status_string.argtypes = [i32]
        lib.farn_status_string.restype = ctypes.c_char_p
        _lib = lib
    return _lib


class FarnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {farn_status_string(status)} (status {status})")


def farn_status_string(status: int) -> str:
    return _load().farn_status_string(int(status)).decode()


def _ptr_array(ptrs):
    return (ctypes.c_void_p * max(1, len(ptrs)))(*[ctypes.c_void_p(int(p)) for p in ptrs])


def farn_create(device: int = 0) -> int:
    """C ``farn_create``: returns the opaque context handle (an int)."""
    h = ctypes.c_void_p()
    st = _load().farn_create(ctypes.byref(h), int(device))
    if st != FARN_OK:
        raise FarnError(st, "farn_create")
    return h.value


def farn_destroy(ctx: int) -> None:
    _load().farn_destroy(ctypes.c_void_p(ctx) if ctx else None)


def farn_forward(ctx, partials, W, residual, weight, eps, T, H,
                 reduced_out, residual_out, norm_out, stream=0) -> int:
    """C ``farn_forward`` on raw device addresses (ints); returns the status."""
    return _load().farn_forward(
        ctypes.c_void_p(ctx) if ctx else None, _ptr_array(partials), int(W),
        ctypes.c_void_p(int(residual)), ctypes.c_void_p(int(weight)), float(eps),
        int(T), int(H), ctypes.c_void_p(int(reduced_out)),
        ctypes.c_void_p(int(residual_out)), ctypes.c_void_p(int(norm_out)),
        ctypes.c_void_p(int(stream)))


def farn_forward_typed(ctx, partials, partial_dtype, W, residual, weight, eps, T, H,
                       reduced_out, residual_out, norm_out, stream=0) -> int:
    """C ``farn_forward_typed``: partials of dtype FARN_BF16 or FARN_F32."""
    return _load().farn_forward_typed(
        ctypes.c_void_p(ctx) if ctx else None, _ptr_array(partials), int(partial_dtype),
        int(W), ctypes.c_void_p(int(residual)), ctypes.c_void_p(int(weight)), float(eps),
        int(T), int(H), ctypes.c_void_p(int(reduced_out)),
        ctypes.c_void_p(int(residual_out)), ctypes.c_void_p(int(norm_out)),
        ctypes.c_void_p(int(stream)))


def farn_forward_quant(ctx, partials, partial_dtype, W, residual, weight, eps, T, H,
                       reduced_out, residual_out, norm_out, norm_q, row_scale,
                       stream=0) -> int:
    """C ``farn_forward_quant``: also writes norm_out as E4M3 bytes plus a
    per-row fp32 scale (norm_out may be 0 to skip it)."""
    return _load().farn_forward_quant(
        ctypes.c_void_p(ctx) if ctx else None, _ptr_array(partials), int(partial_dtype),
        int(W), ctypes.c_void_p(int(residual)), ctypes.c_void_p(int(weight)), float(eps),
        int(T), int(H), ctypes.c_void_p(int(reduced_out)),
        ctypes.c_void_p(int(residual_out)),
        ctypes.c_void_p(int(norm_out)) if norm_out else None,
        ctypes.c_void_p(int(norm_q)), ctypes.c_void_p(int(row_scale)),
        ctypes.c_void_p(int(stream)))


def farn_forward_nvfp4(ctx, partials, partial_dtype, W, residual, weight, eps, T, H,
                       tensor_scale, reduced_out, residual_out, norm_out, norm_fp4,
                       block_scale, stream=0) -> int:
    """C ``farn_forward_nvfp4``: also writes norm_out as NVFP4 (two E2M1
    codes per byte, one E4M3 scale per 16 elements, under tensor_scale);
    norm_out may be 0 to skip it."""
    v = lambda a: ctypes.c_void_p(int(a)) if a else None  # noqa: E731
    return _load().farn_forward_nvfp4(
        ctypes.c_void_p(ctx) if ctx else None, _ptr_array(partials), int(partial_dtype),
        int(W), v(residual), v(weight), float(eps), int(T), int(H), float(tensor_scale),
        v(reduced_out), v(residual_out), v(norm_out), v(norm_fp4), v(block_scale),
        ctypes.c_void_p(int(stream)))


def farn_moe_combine(ctx, expert_out, n_slots, index, gates, K, residual, weight, eps, T, H,
                     reduced_out, residual_out, norm_out, stream=0) -> int:
    """C ``farn_moe_combine`` on raw device addresses (ints)."""
    v = lambda a: ctypes.c_void_p(int(a)) if a else None  # noqa: E731
    return _load().farn_moe_combine(
        ctypes.c_void_p(ctx) if ctx else None, v(expert_out), int(n_slots), v(index), v(gates),
        int(K), v(residual), v(weight), float(eps), int(T), int(H), v(reduced_out),
        v(residual_out), v(norm_out), ctypes.c_void_p(int(stream)))


def _addr(a):
    return ctypes.c_void_p(int(a)) if a else None


def farn_moe_route(ctx, logits, logits_dtype, T, E, K, renormalize, experts, gates, index, rows,
                   offsets, stream=0) -> int:
    """C ``farn_moe_route`` on raw device addresses (ints)."""
    return _load().farn_moe_route(
        _addr(ctx), _addr(logits), int(logits_dtype), int(T), int(E), int(K), int(renormalize),
        _addr(experts), _addr(gates), _addr(index), _addr(rows), _addr(offsets), _addr(stream))


def farn_grouped_matmul(ctx, x, n_rows, rows, n_slots, weights, E, offsets, N, H, out,
                        stream=0) -> int:
    """C ``farn_grouped_matmul`` on raw device addresses (ints); rows 0 for
    slot s reading row s."""
    return _load().farn_grouped_matmul(
        _addr(ctx), _addr(x), int(n_rows), _addr(rows), int(n_slots), _addr(weights), int(E),
        _addr(offsets), int(N), int(H), _addr(out), _addr(stream))


def farn_nvfp4_quantize(ctx, x, T, H, tensor_scale, codes, block_scale, stream=0) -> int:
    """C ``farn_nvfp4_quantize`` on raw device addresses (ints)."""
    return _load().farn_nvfp4_quantize(
        _addr(ctx), _addr(x), int(T), int(H), float(tensor_scale), _addr(codes),
        _addr(block_scale), _addr(stream))


def farn_nvfp4_dequantize(ctx, codes, block_scale, T, H, tensor_scale, out, stream=0) -> int:
    """C ``farn_nvfp4_dequantize`` on raw device addresses (ints)."""
    return _load().farn_nvfp4_dequantize(
        _addr(ctx), _addr(codes), _addr(block_scale), int(T), int(H), float(tensor_scale),
        _addr(out), _addr(stream))


def farn_nvfp4_matmul(ctx, a_codes, a_scale, a_tensor_scale, b_codes, b_scale, b_tensor_scale,
                      T, N, H, out, stream=0) -> int:
    """C ``farn_nvfp4_matmul`` on raw device addresses (ints)."""
    return _load().farn_nvfp4_matmul(
        _addr(ctx), _addr(a_codes), _addr(a_scale), float(a_tensor_scale), _addr(b_codes),
        _addr(b_scale), float(b_tensor_scale), int(T), int(N), int(H), _addr(out),
        _addr(stream))


def farn_fp8_quantize(ctx, x, E, T, H, block_rows, codes, scales, stream=0) -> int:
    """C ``farn_fp8_quantize`` on raw device addresses (ints)."""
    return _load().farn_fp8_quantize(_addr(ctx), _addr(x), int(E), int(T), int(H),
                                     int(block_rows), _addr(codes), _addr(scales), _addr(stream))


def farn_fp8_matmul(ctx, a_codes, a_scale, b_codes, b_scale, T, N, H, out, stream=0) -> int:
    """C ``farn_fp8_matmul`` on raw device addresses (ints)."""
    return _load().farn_fp8_matmul(_addr(ctx), _addr(a_codes), _addr(a_scale), _addr(b_codes),
                                   _addr(b_scale), int(T), int(N), int(H), _addr(out),
                                   _addr(stream))


def farn_fp8_grouped_matmul(ctx, x, x_scale, n_rows, rows, n_slots, weights, w_scale, E, offsets,
                            N, H, out, workspace=0, workspace_bytes=0, stream=0) -> int:
    """C ``farn_fp8_grouped_matmul`` on raw device addresses (ints); rows 0 for
    slot s reading row s."""
    return _load().farn_fp8_grouped_matmul(
        _addr(ctx), _addr(x), _addr(x_scale), int(n_rows), _addr(rows), int(n_slots),
        _addr(weights), _addr(w_scale), int(E), _addr(offsets), int(N), int(H), _addr(out),
        _addr(workspace), int(workspace_bytes), _addr(stream))


def farn_fp8_grouped_workspace(ctx, n_slots, E, N, H) -> int:
    """C ``farn_fp8_grouped_workspace``: the bytes that a call with rows uses."""
    n = ctypes.c_int64()
    st = _load().farn_fp8_grouped_workspace(_addr(ctx), int(n_slots), int(E), int(N), int(H),
                                            ctypes.byref(n))
    if st != FARN_OK:
        raise FarnError(st, "farn_fp8_grouped_workspace")
    return n.value


def farn_plan_fp8_matmul(ctx, a_codes, b_codes, T, N, H, out):
    """C ``farn_plan_fp8_matmul``: (variant name, CTAs per tile, threads per CTA)."""
    return _plan(_load().farn_plan_fp8_matmul, "farn_plan_fp8_matmul", _addr(ctx),
                 _addr(a_codes), _addr(b_codes), int(T), int(N), int(H), _addr(out))


def farn_plan_fp8_grouped_matmul(ctx, x, n_rows, rows, n_slots, weights, E, N, H, out,
                                 workspace=0):
    """C ``farn_plan_fp8_grouped_matmul``: (variant name, CTAs per tile, threads per CTA)."""
    return _plan(_load().farn_plan_fp8_grouped_matmul, "farn_plan_fp8_grouped_matmul",
                 _addr(ctx), _addr(x), int(n_rows), _addr(rows), int(n_slots), _addr(weights),
                 int(E), int(N), int(H), _addr(out), _addr(workspace))


def _int_array(v):
    return None if v is None else (ctypes.c_int * max(1, len(v)))(*[int(x) for x in v])


def farn_qk_norm_rope(ctx, T, D, q, q_heads, q_stride, k, k_heads, k_stride, q_weight, k_weight,
                      eps, positions, axes, sections, freqs, R, interleaved, q_out, q_out_stride,
                      k_out, k_out_stride, stream=0) -> int:
    """C ``farn_qk_norm_rope`` on raw device addresses (ints); sections a
    sequence of ints or None."""
    return _load().farn_qk_norm_rope(
        _addr(ctx), int(T), int(D), _addr(q), int(q_heads), int(q_stride), _addr(k), int(k_heads),
        int(k_stride), _addr(q_weight), _addr(k_weight), float(eps), _addr(positions), int(axes),
        _int_array(sections), _addr(freqs), int(R), int(interleaved), _addr(q_out),
        int(q_out_stride), _addr(k_out), int(k_out_stride), _addr(stream))


def _cache_ref(cache):
    # the library reads a whole struct at the address
    if cache is not None and not isinstance(cache, KvCache):
        raise TypeError(f"cache must be a KvCache or None, got {type(cache).__name__}")
    return None if cache is None else ctypes.byref(cache)


def farn_qk_norm_rope_cache(ctx, T, D, q, q_heads, q_stride, k, k_stride, v, v_stride, kv_heads,
                            q_weight, k_weight, eps, positions, axes, sections, freqs, R,
                            interleaved, q_out, q_out_stride, cache, slots, stream=0) -> int:
    """C ``farn_qk_norm_rope_cache`` on raw device addresses (ints); cache a
    ``KvCache``."""
    return _load().farn_qk_norm_rope_cache(
        _addr(ctx), int(T), int(D), _addr(q), int(q_heads), int(q_stride), _addr(k),
        int(k_stride), _addr(v), int(v_stride), int(kv_heads), _addr(q_weight), _addr(k_weight),
        float(eps), _addr(positions), int(axes), _int_array(sections), _addr(freqs), int(R),
        int(interleaved), _addr(q_out), int(q_out_stride), _cache_ref(cache), _addr(slots),
        _addr(stream))


def farn_kv_write(ctx, T, k, k_stride, v, v_stride, cache, slots, stream=0) -> int:
    """C ``farn_kv_write`` on raw device addresses (ints); cache a ``KvCache``."""
    return _load().farn_kv_write(_addr(ctx), int(T), _addr(k), int(k_stride), _addr(v),
                                 int(v_stride), _cache_ref(cache), _addr(slots), _addr(stream))


def farn_kv_read(ctx, cache, table, B, width, offsets, n_tokens, k_out, v_out, stream=0) -> int:
    """C ``farn_kv_read`` on raw device addresses (ints); cache a ``KvCache``."""
    return _load().farn_kv_read(_addr(ctx), _cache_ref(cache), _addr(table), int(B), int(width),
                                _addr(offsets), int(n_tokens), _addr(k_out), _addr(v_out),
                                _addr(stream))


def farn_forward_noalloc(device, partials, W, residual, weight, eps, T, H,
                         reduced_out, residual_out, norm_out, stream=0,
                         want_status=False):
    """C ``farn_forward_noalloc`` on raw device addresses (ints), for callers
    that cannot allocate device memory: no context, nothing allocated.
    Returns (status, device status word or None); asking for the word makes
    the call wait for the kernel."""
    word = ctypes.c_int(-1)
    st = _load().farn_forward_noalloc(
        int(device), _ptr_array(partials), int(W), ctypes.c_void_p(int(residual)),
        ctypes.c_void_p(int(weight)), float(eps), int(T), int(H),
        ctypes.c_void_p(int(reduced_out)), ctypes.c_void_p(int(residual_out)),
        ctypes.c_void_p(int(norm_out)), ctypes.c_void_p(int(stream)),
        ctypes.byref(word) if want_status else None)
    return st, (word.value if want_status else None)


def farn_device_status(ctx: int) -> int:
    """C ``farn_device_status``: read and clear the device status word."""
    v = ctypes.c_int()
    st = _load().farn_device_status(ctypes.c_void_p(ctx), ctypes.byref(v))
    if st != FARN_OK:
        raise FarnError(st, "farn_device_status")
    return v.value


def farn_check_args(partials, W, residual, weight, eps, T, H, reduced_out,
                    residual_out, norm_out) -> int:
    """C ``farn_check_args``: host-only checks, addresses are only compared."""
    arr = None if partials is None else _ptr_array(partials)
    v = lambda a: ctypes.c_void_p(int(a)) if a else None  # noqa: E731
    return _load().farn_check_args(arr, int(W), v(residual), v(weight),
                                   float(eps), int(T), int(H), v(reduced_out),
                                   v(residual_out), v(norm_out))


def farn_plan(ctx, W, T, H, partials, residual, weight, reduced_out,
              residual_out, norm_out):
    """C ``farn_plan``: (variant name, CTAs per row, threads per CTA)."""
    variant, cs, thr = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    v = lambda a: ctypes.c_void_p(int(a)) if a else None  # noqa: E731
    st = _load().farn_plan(ctypes.c_void_p(ctx), int(W), int(T), int(H),
                           _ptr_array(partials), v(residual), v(weight),
                           v(reduced_out), v(residual_out), v(norm_out),
                           ctypes.byref(variant), ctypes.byref(cs),
                           ctypes.byref(thr))
    if st != FARN_OK:
        raise FarnError(st, "farn_plan")
    return VARIANTS[variant.value], cs.value, thr.value


FARN_PLAN_FP8_OUT = 1
FARN_PLAN_NVFP4_OUT = 2


def farn_plan_typed(ctx, partial_dtype, W, T, H, partials, residual, weight, reduced_out,
                    residual_out, norm_out, flags=0):
    """C ``farn_plan_typed``: (variant name, CTAs per row, threads per CTA)."""
    variant, cs, thr = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    v = lambda a: ctypes.c_void_p(int(a)) if a else None  # noqa: E731
    st = _load().farn_plan_typed(ctypes.c_void_p(ctx), int(partial_dtype), int(flags),
                                 int(W), int(T),
                                 int(H), _ptr_array(partials), v(residual), v(weight),
                                 v(reduced_out), v(residual_out), v(norm_out),
                                 ctypes.byref(variant), ctypes.byref(cs), ctypes.byref(thr))
    if st != FARN_OK:
        raise FarnError(st, "farn_plan_typed")
    return VARIANTS[variant.value], cs.value, thr.value


def farn_plan_moe_combine(ctx, K, T, H, expert_out, residual, weight, reduced_out,
                          residual_out, norm_out):
    """C ``farn_plan_moe_combine``: (variant name, threads per CTA)."""
    variant, thr = ctypes.c_int(), ctypes.c_int()
    v = lambda a: ctypes.c_void_p(int(a)) if a else None  # noqa: E731
    st = _load().farn_plan_moe_combine(ctypes.c_void_p(ctx), int(K), int(T), int(H),
                                       v(expert_out), v(residual), v(weight), v(reduced_out),
                                       v(residual_out), v(norm_out), ctypes.byref(variant),
                                       ctypes.byref(thr))
    if st != FARN_OK:
        raise FarnError(st, "farn_plan_moe_combine")
    return VARIANTS[variant.value], thr.value


def _plan(fn, name, *args):
    variant, ctas, thr = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    st = fn(*args, ctypes.byref(variant), ctypes.byref(ctas), ctypes.byref(thr))
    if st != FARN_OK:
        raise FarnError(st, name)
    return VARIANTS[variant.value], ctas.value, thr.value


def farn_plan_grouped_matmul(ctx, x, n_rows, rows, n_slots, weights, E, N, H, out):
    """C ``farn_plan_grouped_matmul``: (variant name, CTAs per tile, threads per CTA)."""
    return _plan(_load().farn_plan_grouped_matmul, "farn_plan_grouped_matmul", _addr(ctx),
                 _addr(x), int(n_rows), _addr(rows), int(n_slots), _addr(weights), int(E),
                 int(N), int(H), _addr(out))


def farn_plan_nvfp4_matmul(ctx, a_codes, a_scale, b_codes, b_scale, T, N, H, out):
    """C ``farn_plan_nvfp4_matmul``: (variant name, CTAs per tile, threads per CTA)."""
    return _plan(_load().farn_plan_nvfp4_matmul, "farn_plan_nvfp4_matmul", _addr(ctx),
                 _addr(a_codes), _addr(a_scale), _addr(b_codes), _addr(b_scale), int(T), int(N),
                 int(H), _addr(out))


class Context:
    """Owns one ``farn_ctx`` for a device (``farn_create``/``farn_destroy``)."""

    def __init__(self, device: int = 0):
        self.device = int(device)
        self.handle = farn_create(self.device)

    def close(self):
        if self.handle:
            farn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


_default_ctx: dict[int, Context] = {}


def _context_for(device_index: int) -> Context:
    c = _default_ctx.get(device_index)
    if c is None:
        c = _default_ctx[device_index] = Context(device_index)
    return c


def _check_tensor(t, name, shape, device, dtypes=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtypes = dtypes or (torch.bfloat16,)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


# ------------------------------------------------------------ torch level
class PreparedCall:
    """One operator call whose tensors were checked and whose C-ABI
    arguments were marshalled once.  Calling it launches the kernel on the
    stream given at preparation (asynchronously) and returns the outputs; a
    caller that reuses its buffers (a serving loop, a benchmark) pays only
    the C call each time.  The tensors must stay alive, in place, while the
    object is used."""

    __slots__ = ("_fn", "_args", "_name", "_keep", "outputs")

    def __init__(self, fn, args, name, outputs, keep):
        self._fn, self._args, self._name = fn, args, name
        self.outputs, self._keep = outputs, keep

    def __call__(self):
        st = self._fn(*self._args)
        if st != FARN_OK:
            raise FarnError(st, self._name)
        return self.outputs


def _vp(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _partials_checked(partials, residual, weight):
    import torch
    partials = list(partials)
    if not partials:
        raise ValueError("partials must hold at least one tensor")
    if residual.dim() != 2:
        raise ValueError("residual must be [T, H]")
    T, H = residual.shape
    dev = residual.device
    pdt = partials[0].dtype
    if pdt not in (torch.bfloat16, torch.float32):
        raise TypeError(f"partials must be bfloat16 or float32, got {pdt}")
    for r, x in enumerate(partials):
        _check_tensor(x, f"partials[{r}]", (T, H), dev, (pdt,))
    _check_tensor(residual, "residual", (T, H), dev)
    _check_tensor(weight, "weight", (H,), dev)
    return partials, T, H, dev, (FARN_F32 if pdt == torch.float32 else FARN_BF16)


def _common_args(ctx, partials, dtype, residual, weight, eps, T, H):
    return (ctypes.c_void_p(ctx.handle), _ptr_array([x.data_ptr() for x in partials]),
            ctypes.c_int(dtype), ctypes.c_int(len(partials)), _vp(residual), _vp(weight),
            ctypes.c_float(eps), ctypes.c_int64(T), ctypes.c_int64(H))


def _ctx_stream(ctx, stream, dev):
    import torch
    c = ctx if ctx is not None else _context_for(dev.index)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    return c, ctypes.c_void_p(int(s.cuda_stream))


def prepare_forward(partials, residual, weight, eps: float, out=None, ctx=None, stream=None):
    """``forward`` checked and marshalled once (see ``PreparedCall``)."""
    import torch
    partials, T, H, dev, dtype = _partials_checked(partials, residual, weight)
    if out is None:
        out = _new(stream, dev, *[((T, H), torch.bfloat16)] * 3)
    for name, t in zip(("reduced", "residual_out", "norm_out"), out):
        _check_tensor(t, name, (T, H), dev)
    c, s = _ctx_stream(ctx, stream, dev)
    args = _common_args(c, partials, dtype, residual, weight, eps, T, H) + \
        (_vp(out[0]), _vp(out[1]), _vp(out[2]), s)
    return PreparedCall(_load().farn_forward_typed, args, "farn_forward", tuple(out),
                        (partials, residual, weight, c))


def forward(partials, residual, weight, eps: float, out=None, ctx=None,
            stream=None):
    """The fused operator on torch CUDA tensors.

    partials: sequence of W tensors [T,H], all bf16 or all fp32 (fp32 partials
    are summed as fp32, see farn_forward_typed); residual [T,H] and weight
    [H] bf16; outputs bf16.
    out: optional (reduced, residual_out, norm_out) tensors to write
    (residual_out may be ``residual`` itself).  Runs asynchronously on
    ``stream`` (default: torch's current stream) and returns the outputs.
    """
    return prepare_forward(partials, residual, weight, eps, out, ctx, stream)()


def _check_quant_out(out, T, H, dev, q_shape, q_dtype, s_shape, s_dtype):
    import torch
    if len(out) != 5:
        raise ValueError("out must be (reduced, residual_out, norm_out or None, codes, scales)")
    for name, t in zip(("reduced", "residual_out"), out[:2]):
        _check_tensor(t, name, (T, H), dev)
    if out[2] is not None:
        _check_tensor(out[2], "norm_out", (T, H), dev)
    _check_tensor(out[3], "codes", q_shape, dev, (q_dtype,))
    _check_tensor(out[4], "scales", s_shape, dev, (s_dtype,))


def prepare_forward_quant(partials, residual, weight, eps: float, write_norm: bool = True,
                          out=None, ctx=None, stream=None):
    """``forward_quant`` checked and marshalled once.  out: optional
    (reduced, residual_out, norm_out or None, norm_q, row_scale)."""
    import torch
    partials, T, H, dev, dtype = _partials_checked(partials, residual, weight)
    if out is None:
        norms = [((T, H), torch.bfloat16)] * (3 if write_norm else 2)
        out = _new(stream, dev, *norms, ((T, H), torch.uint8), ((T,), torch.float32))
        if not write_norm:
            out = (*out[:2], None, *out[2:])
    _check_quant_out(out, T, H, dev, (T, H), torch.uint8, (T,), torch.float32)
    c, s = _ctx_stream(ctx, stream, dev)
    args = _common_args(c, partials, dtype, residual, weight, eps, T, H) + \
        tuple(_vp(t) for t in out) + (s,)
    return PreparedCall(_load().farn_forward_quant, args, "farn_forward_quant", tuple(out),
                        (partials, residual, weight, c))


def forward_quant(partials, residual, weight, eps: float, write_norm: bool = True,
                  ctx=None, stream=None):
    """``forward`` plus the FP8 (E4M3) copy of norm_out and its per-row
    scales.  Returns (reduced, residual_out, norm_out or None, norm_q as a
    uint8 tensor of E4M3 patterns, row_scale float32 [T])."""
    return prepare_forward_quant(partials, residual, weight, eps, write_norm,
                                 ctx=ctx, stream=stream)()


def prepare_forward_nvfp4(partials, residual, weight, eps: float, tensor_scale: float,
                          write_norm: bool = True, out=None, ctx=None, stream=None):
    """``forward_nvfp4`` checked and marshalled once.  out: optional
    (reduced, residual_out, norm_out or None, norm_fp4, block_scale)."""
    import torch
    partials, T, H, dev, dtype = _partials_checked(partials, residual, weight)
    if H % 16:
        raise ValueError(f"NVFP4 output needs H % 16 == 0, got H = {H}")
    if out is None:
        norms = [((T, H), torch.bfloat16)] * (3 if write_norm else 2)
        out = _new(stream, dev, *norms, ((T, H // 2), torch.uint8), ((T, H // 16), torch.uint8))
        if not write_norm:
            out = (*out[:2], None, *out[2:])
    _check_quant_out(out, T, H, dev, (T, H // 2), torch.uint8, (T, H // 16), torch.uint8)
    c, s = _ctx_stream(ctx, stream, dev)
    args = _common_args(c, partials, dtype, residual, weight, eps, T, H) + \
        (ctypes.c_float(tensor_scale),) + tuple(_vp(t) for t in out) + (s,)
    return PreparedCall(_load().farn_forward_nvfp4, args, "farn_forward_nvfp4", tuple(out),
                        (partials, residual, weight, c))


def forward_nvfp4(partials, residual, weight, eps: float, tensor_scale: float,
                  write_norm: bool = True, ctx=None, stream=None):
    """``forward`` plus the NVFP4 copy of norm_out.  Returns (reduced,
    residual_out, norm_out or None, norm_fp4 uint8 [T,H/2] (two E2M1 codes
    per byte, the even element in the low nibble), block_scale uint8
    [T,H/16] (E4M3 patterns)).  H must be a multiple of 16."""
    return prepare_forward_nvfp4(partials, residual, weight, eps, tensor_scale, write_norm,
                                 ctx=ctx, stream=stream)()


def prepare_moe_combine(expert_out, index, gates, residual, weight, eps: float, out=None,
                        ctx=None, stream=None):
    """``moe_combine`` checked and marshalled once."""
    import torch
    T, H = residual.shape
    dev = residual.device
    S = expert_out.shape[0]
    _check_tensor(expert_out, "expert_out", (S, H), dev)
    K = index.shape[1] if index.dim() == 2 else -1
    _check_tensor(index, "index", (T, K), dev, (torch.int32,))
    _check_tensor(gates, "gates", (T, K), dev, (torch.float32,))
    _check_tensor(residual, "residual", (T, H), dev)
    _check_tensor(weight, "weight", (H,), dev)
    if out is None:
        out = _new(stream, dev, *[((T, H), torch.bfloat16)] * 3)
    for name, t in zip(("reduced", "residual_out", "norm_out"), out):
        _check_tensor(t, name, (T, H), dev)
    c, s = _ctx_stream(ctx, stream, dev)
    args = (ctypes.c_void_p(c.handle), _vp(expert_out), ctypes.c_int64(S), _vp(index),
            _vp(gates), ctypes.c_int(K), _vp(residual), _vp(weight), ctypes.c_float(eps),
            ctypes.c_int64(T), ctypes.c_int64(H), _vp(out[0]), _vp(out[1]), _vp(out[2]), s)
    return PreparedCall(_load().farn_moe_combine, args, "farn_moe_combine", tuple(out),
                        (expert_out, index, gates, residual, weight, c))


def moe_combine(expert_out, index, gates, residual, weight, eps: float, out=None, ctx=None,
                stream=None):
    """MoE combine + residual + RMSNorm on torch CUDA tensors: expert_out bf16
    [S,H], index int32 [T,K], gates fp32 [T,K], residual bf16 [T,H], weight
    bf16 [H].  Returns (reduced, residual_out, norm_out)."""
    return prepare_moe_combine(expert_out, index, gates, residual, weight, eps, out, ctx,
                               stream)()


# The calls below check their tensors on a short path, one expression without
# calls of its own (a serving step makes several of them per layer, and their
# kernels take a few microseconds); what it turns down goes through
# _check_tensor for the message.
_torch = _current_raw_stream = None


def _load_torch():
    global _torch, _current_raw_stream
    import torch
    # the handle alone, without a Stream object around it, where torch has it
    _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _torch = torch
    return torch


def _raw_stream(stream, index):
    return _current_raw_stream(index) if stream is None else stream.cuda_stream


def _new(stream, device, *specs, returned=True):
    """New tensors, a (shape, dtype) each, for a call on `stream` to write.  On a
    given stream they come from that stream's own memory: the current stream may
    still be at work on what a free block of its own was before, and the call does
    not wait for it.  What is returned is used on the current stream, so its block
    does not go to a later call on `stream` before that use is over."""
    torch = _torch or _load_torch()
    if stream is not None:
        cuda = torch.cuda
        here = cuda.current_stream(device)
        if stream.cuda_stream != here.cuda_stream:
            return _new_elsewhere(cuda, stream, here, device, specs, returned)
    return tuple([torch.empty(s, dtype=d, device=device) for s, d in specs])


def _new_elsewhere(cuda, stream, here, device, specs, returned):
    if not isinstance(stream, cuda.Stream):
        stream = cuda.ExternalStream(stream.cuda_stream, device=device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    # cuda.stream(stream) in its place takes 6 to 8 us more per call
    index = cuda.current_device()
    cuda.set_stream(stream)
    try:
        new = tuple([_torch.empty(s, dtype=d, device=device) for s, d in specs])
    finally:
        cuda.set_stream(here)               # makes its device the current one
        cuda.set_device(index)
    if returned:
        for t in new:
            t.record_stream(here)
    return new


def _call(fn, args, name):
    st = fn(*args)
    if st != FARN_OK:
        raise FarnError(st, name)


def _moe_route_args(logits, top_k, renormalize, out, ctx, stream):
    torch = _torch or _load_torch()
    i32, f32 = torch.int32, torch.float32
    sl = logits.shape
    if len(sl) != 2:
        raise ValueError("logits must be [T, E]")
    T, E = sl
    K, index = int(top_k), logits.get_device()
    if index < 0 or not logits.is_contiguous() or logits.dtype not in (torch.bfloat16, f32):
        _check_tensor(logits, "logits", (T, E), logits.device, (torch.bfloat16, f32))
    if not 1 <= E <= FARN_MAX_EXPERTS:
        raise ValueError(f"the number of experts must be 1..{FARN_MAX_EXPERTS}, got {E}")
    if not 1 <= K <= min(E, FARN_MAX_W):
        raise ValueError(f"top_k must be 1..{min(E, FARN_MAX_W)}, got {K}")
    if out is None:
        pairs = (T, K)
        out = _new(stream, logits.device, (pairs, i32), (pairs, f32), (pairs, i32),
                   ((T * K,), i32), ((E + 1,), i32))
    else:
        out = tuple(out)
        if len(out) != 5:
            raise ValueError("out must be (experts, gates, index, rows, offsets)")
        for name, t, shape, dt in zip(("experts", "gates", "index", "rows", "offsets"), out,
                                      ((T, K), (T, K), (T, K), (T * K,), (E + 1,)),
                                      (i32, f32, i32, i32, i32)):
            _check_tensor(t, name, shape, logits.device, (dt,))
    c = ctx if ctx is not None else _context_for(index)
    if c.device != index:
        raise ValueError(f"the context is for device {c.device}, the tensors are on {index}")
    return (c.handle, logits.data_ptr(), FARN_F32 if logits.dtype is f32 else FARN_BF16, T, E, K,
            1 if renormalize else 0, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(),
            out[3].data_ptr(), out[4].data_ptr(), _raw_stream(stream, index)), out, c


def prepare_moe_route(logits, top_k: int, renormalize: bool = True, out=None, ctx=None,
                      stream=None):
    """``moe_route`` checked and marshalled once."""
    args, out, c = _moe_route_args(logits, top_k, renormalize, out, ctx, stream)
    return PreparedCall(_load().farn_moe_route, args, "farn_moe_route", out, (logits, c))


def moe_route(logits, top_k: int, renormalize: bool = True, out=None, ctx=None, stream=None):
    """The MoE router on a bf16 or fp32 tensor of logits [T,E].  Returns
    (experts int32 [T,K], gates fp32 [T,K], index int32 [T,K], rows int32
    [T*K], offsets int32 [E+1]): rows and offsets are ``grouped_matmul``'s,
    index and gates ``moe_combine``'s.  An expert masked with -inf is never
    chosen; a pair without an expert has expert -1, gate 0 and index -1."""
    args, out, _ = _moe_route_args(logits, top_k, renormalize, out, ctx, stream)
    _call(_load().farn_moe_route, args, "farn_moe_route")
    return out


def _grouped_args(x, weights, offsets, rows, out, ctx, stream):
    torch = _torch or _load_torch()
    bf, i32 = torch.bfloat16, torch.int32
    sx, sw, index = x.shape, weights.shape, x.get_device()
    if len(sx) != 2 or len(sw) != 3:
        raise ValueError("x must be [rows, H] and weights [E, N, H]")
    n_rows, H = sx
    E, N, HW = sw
    if not (HW == H and index >= 0 and weights.get_device() == index and
            offsets.get_device() == index and x.dtype is bf and weights.dtype is bf and
            offsets.dtype is i32 and offsets.shape == (E + 1,) and x.is_contiguous() and
            weights.is_contiguous() and offsets.is_contiguous()):
        dev = x.device
        _check_tensor(x, "x", (n_rows, H), dev)
        _check_tensor(weights, "weights", (E, N, H), dev)
        _check_tensor(offsets, "offsets", (E + 1,), dev, (i32,))
    S = n_rows
    if rows is not None:
        sr = rows.shape
        S = sr[0] if len(sr) == 1 else -1
        if not (S >= 0 and rows.dtype is i32 and rows.get_device() == index and
                rows.is_contiguous()):
            _check_tensor(rows, "rows", (S,), x.device, (i32,))
    if out is None:
        out, = _new(stream, x.device, ((S, N), bf))
    else:
        _check_tensor(out, "out", (S, N), x.device)
    c = ctx if ctx is not None else _context_for(index)
    if c.device != index:
        raise ValueError(f"the context is for device {c.device}, the tensors are on {index}")
    return (c.handle, x.data_ptr(), n_rows, None if rows is None else rows.data_ptr(), S,
            weights.data_ptr(), E, offsets.data_ptr(), N, H, out.data_ptr(),
            _raw_stream(stream, index)), out, c


def prepare_grouped_matmul(x, weights, offsets, rows=None, out=None, ctx=None, stream=None):
    """``grouped_matmul`` checked and marshalled once."""
    args, out, c = _grouped_args(x, weights, offsets, rows, out, ctx, stream)
    return PreparedCall(_load().farn_grouped_matmul, args, "farn_grouped_matmul", out,
                        (x, weights, offsets, rows, c))


def grouped_matmul(x, weights, offsets, rows=None, out=None, ctx=None, stream=None):
    """The experts' products on torch CUDA tensors: x bf16 [n,H], weights bf16
    [E,N,H], offsets int32 [E+1] (expert e has the slots offsets[e] ..
    offsets[e+1]-1), rows int32 [S] (the row of x that a slot reads; None:
    slot s reads row s).  Returns out bf16 [S,N], ``moe_combine``'s
    expert_out; slots that no expert has are left as they were."""
    args, out, _ = _grouped_args(x, weights, offsets, rows, out, ctx, stream)
    _call(_load().farn_grouped_matmul, args, "farn_grouped_matmul")
    return out


def _nvfp4_shape(codes, scales, name):
    torch = _torch or _load_torch()
    sc = codes.shape
    if len(sc) != 2:
        raise ValueError(f"{name} must be [rows, H/2]")
    T, half = sc
    if half % 8:
        raise ValueError(f"NVFP4 needs H % 16 == 0, got H = {half * 2}")
    u8, index = torch.uint8, codes.get_device()
    if not (index >= 0 and scales.get_device() == index and codes.dtype is u8 and
            scales.dtype is u8 and scales.shape == (T, half // 8) and codes.is_contiguous() and
            scales.is_contiguous()):
        _check_tensor(codes, name, (T, half), codes.device, (u8,))
        _check_tensor(scales, name + " scales", (T, half // 8), codes.device, (u8,))
    return T, half * 2, index


def _quantize_args(x, tensor_scale, out, ctx, stream):
    torch = _torch or _load_torch()
    u8 = torch.uint8
    sx, index = x.shape, x.get_device()
    if len(sx) != 2:
        raise ValueError("x must be [T, H]")
    T, H = sx
    if not (index >= 0 and x.dtype is torch.bfloat16 and x.is_contiguous()):
        _check_tensor(x, "x", (T, H), x.device)
    if H % 16:
        raise ValueError(f"NVFP4 needs H % 16 == 0, got H = {H}")
    if out is None:
        out = _new(stream, x.device, ((T, H // 2), u8), ((T, H // 16), u8))
    else:
        out = tuple(out)
        if len(out) != 2:
            raise ValueError("out must be (codes, scales)")
        _check_tensor(out[0], "codes", (T, H // 2), x.device, (u8,))
        _check_tensor(out[1], "scales", (T, H // 16), x.device, (u8,))
    c = ctx if ctx is not None else _context_for(index)
    if c.device != index:
        raise ValueError(f"the context is for device {c.device}, the tensors are on {index}")
    return (c.handle, x.data_ptr(), T, H, tensor_scale, out[0].data_ptr(), out[1].data_ptr(),
            _raw_stream(stream, index)), out, c


def prepare_nvfp4_quantize(x, tensor_scale: float, out=None, ctx=None, stream=None):
    """``nvfp4_quantize`` checked and marshalled once."""
    args, out, c = _quantize_args(x, tensor_scale, out, ctx, stream)
    return PreparedCall(_load().farn_nvfp4_quantize, args, "farn_nvfp4_quantize", out, (x, c))


def nvfp4_quantize(x, tensor_scale: float, out=None, ctx=None, stream=None):
    """NVFP4 codes of a bf16 tensor [T,H], in ``forward_nvfp4``'s format.
    Returns (codes uint8 [T,H/2], block_scale uint8 [T,H/16]); H must be a
    multiple of 16."""
    args, out, _ = _quantize_args(x, tensor_scale, out, ctx, stream)
    _call(_load().farn_nvfp4_quantize, args, "farn_nvfp4_quantize")
    return out


def _dequantize_args(codes, block_scale, tensor_scale, out, ctx, stream):
    torch = _torch or _load_torch()
    T, H, index = _nvfp4_shape(codes, block_scale, "codes")
    if out is None:
        out, = _new(stream, codes.device, ((T, H), torch.bfloat16))
    else:
        _check_tensor(out, "out", (T, H), codes.device)
    c = ctx if ctx is not None else _context_for(index)
    if c.device != index:
        raise ValueError(f"the context is for device {c.device}, the tensors are on {index}")
    return (c.handle, codes.data_ptr(), block_scale.data_ptr(), T, H, tensor_scale,
            out.data_ptr(), _raw_stream(stream, index)), out, c


def prepare_nvfp4_dequantize(codes, block_scale, tensor_scale: float, out=None, ctx=None,
                             stream=None):
    """``nvfp4_dequantize`` checked and marshalled once."""
    args, out, c = _dequantize_args(codes, block_scale, tensor_scale, out, ctx, stream)
    return PreparedCall(_load().farn_nvfp4_dequantize, args, "farn_nvfp4_dequantize", out,
                        (codes, block_scale, c))


def nvfp4_dequantize(codes, block_scale, tensor_scale: float, out=None, ctx=None, stream=None):
    """The values of NVFP4 codes and block scales, as a bf16 tensor [T,H]."""
    args, out, _ = _dequantize_args(codes, block_scale, tensor_scale, out, ctx, stream)
    _call(_load().farn_nvfp4_dequantize, args, "farn_nvfp4_dequantize")
    return out


def _nvfp4_matmul_args(a_codes, a_scale, a_tensor_scale, b_codes, b_scale, b_tensor_scale, out,
                       ctx, stream):
    torch = _torch or _load_torch()
    u8, bf = torch.uint8, torch.bfloat16
    index = a_codes.get_device()
    sa, sb = a_codes.shape, b_codes.shape
    half = sa[-1] if sa else 0
    if not (len(sa) == 2 and len(sb) == 2 and half % 8 == 0 and sb[1] == half and index >= 0 and
            b_codes.get_device() == index and a_scale.get_device() == index and
            b_scale.get_device() == index and a_codes.dtype is u8 and b_codes.dtype is u8 and
            a_scale.dtype is u8 and b_scale.dtype is u8 and
            a_scale.shape == (sa[0], half // 8) and b_scale.shape == (sb[0], half // 8) and
            a_codes.is_contiguous() and b_codes.is_contiguous() and a_scale.is_contiguous() and
            b_scale.is_contiguous()):
        _, H, _ = _nvfp4_shape(a_codes, a_scale, "a_codes")
        _, HB, index_b = _nvfp4_shape(b_codes, b_scale, "b_codes")
        if HB != H:
            raise ValueError(f"a and b must have the same H, got {H} and {HB}")
        if index_b != index:
            raise ValueError(f"b_codes must be on {a_codes.device}, got {b_codes.device}")
    T, N = sa[0], sb[0]
    if out is None:
        out, = _new(stream, a_codes.device, ((T, N), bf))
    else:
        _check_tensor(out, "out", (T, N), a_codes.device)
    c = ctx if ctx is not None else _context_for(index)
    if c.device != index:
        raise ValueError(f"the context is for device {c.device}, the tensors are on {index}")
    return (c.handle, a_codes.data_ptr(), a_scale.data_ptr(), a_tensor_scale,
            b_codes.data_ptr(), b_scale.data_ptr(), b_tensor_scale, T, N, half * 2,
            out.data_ptr(), _raw_stream(stream, index)), out, c


def prepare_nvfp4_matmul(a_codes, a_scale, a_tensor_scale: float, b_codes, b_scale,
                         b_tensor_scale: float, out=None, ctx=None, stream=None):
    """``nvfp4_matmul`` checked and marshalled once."""
    args, out, c = _nvfp4_matmul_args(a_codes, a_scale, a_tensor_scale, b_codes, b_scale,
                                      b_tensor_scale, out, ctx, stream)
    return PreparedCall(_load().farn_nvfp4_matmul, args, "farn_nvfp4_matmul", out,
                        (a_codes, a_scale, b_codes, b_scale, c))


def nvfp4_matmul(a_codes, a_scale, a_tensor_scale: float, b_codes, b_scale,
                 b_tensor_scale: float, out=None, ctx=None, stream=None):
    """The product of two NVFP4 tensors, a [T,H] and b [N,H] (as
    ``forward_nvfp4`` and ``nvfp4_quantize`` give them), in bf16 [T,N]."""
    args, out, _ = _nvfp4_matmul_args(a_codes, a_scale, a_tensor_scale, b_codes, b_scale,
                                      b_tensor_scale, out, ctx, stream)
    _call(_load().farn_nvfp4_matmul, args, "farn_nvfp4_matmul")
    return out


def _context_of(ctx, index):
    c = ctx if ctx is not None else _context_for(index)
    if c.device != index:
        raise ValueError(f"the context is for device {c.device}, the tensors are on {index}")
    return c


def _fp8_quantize_args(x, block_rows, out, ctx, stream):
    torch = _torch or _load_torch()
    sx, index = x.shape, x.get_device()
    if len(sx) not in (2, 3):
        raise ValueError("x must be [T, H] or [E, T, H]")
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows must be 1 or 128, got {block_rows}")
    if not (index >= 0 and x.dtype is torch.bfloat16 and x.is_contiguous()):
        _check_tensor(x, "x", sx, x.device)
    T, H = sx[-2:]
    if H < 1:
        raise ValueError("x must have at least one column")
    shape = (*sx[:-2], -(-T // block_rows), -(-H // 128))
    if out is None:
        out = _new(stream, x.device, (sx, torch.uint8), (shape, torch.float32))
    else:
        out = tuple(out)
        if len(out) != 2:
            raise ValueError("out must be (codes, scales)")
        _check_tensor(out[0], "codes", sx, x.device, (torch.uint8,))
        _check_tensor(out[1], "scales", shape, x.device, (torch.float32,))
    c = _context_of(ctx, index)
    return (c.handle, x.data_ptr(), sx[0] if len(sx) == 3 else 1, T, H, block_rows,
            out[0].data_ptr(), out[1].data_ptr(), _raw_stream(stream, index)), out, c


def prepare_fp8_quantize(x, block_rows: int = 1, out=None, ctx=None, stream=None):
    """``fp8_quantize`` checked and marshalled once."""
    args, out, c = _fp8_quantize_args(x, block_rows, out, ctx, stream)
    return PreparedCall(_load().farn_fp8_quantize, args, "farn_fp8_quantize", out, (x, c))


def fp8_quantize(x, block_rows: int = 1, out=None, ctx=None, stream=None):
    """E4M3 codes and fp32 scales of a bf16 tensor [T,H] or [E,T,H], in blocks
    of 128 elements of a row (block_rows 1: activations) or of 128 rows by 128
    columns (block_rows 128: weights).  Returns (codes uint8 of x's shape,
    scales fp32 [..,ceil(T/block_rows),ceil(H/128)]): the operands of
    ``fp8_matmul`` and ``fp8_grouped_matmul``."""
    args, out, _ = _fp8_quantize_args(x, block_rows, out, ctx, stream)
    _call((_lib or _load()).farn_fp8_quantize, args, "farn_fp8_quantize")
    return out


def _fp8_matmul_args(a_codes, a_scale, b_codes, b_scale, out, ctx, stream):
    torch = _torch or _load_torch()
    u8, f32 = torch.uint8, torch.float32
    index = a_codes.get_device()
    sa, sb = a_codes.shape, b_codes.shape
    if len(sa) != 2 or len(sb) != 2:
        raise ValueError("a_codes must be [T, H] and b_codes [N, H]")
    T, H = sa
    N = sb[0]
    HB, NB = -(-H // 128), -(-N // 128)
    if not (sb[1] == H and index >= 0 and b_codes.get_device() == index and
            a_scale.get_device() == index and b_scale.get_device() == index and
            a_codes.dtype is u8 and b_codes.dtype is u8 and a_scale.dtype is f32 and
            b_scale.dtype is f32 and a_scale.shape == (T, HB) and b_scale.shape == (NB, HB) and
            a_codes.is_contiguous() and b_codes.is_contiguous() and a_scale.is_contiguous() and
            b_scale.is_contiguous()):
        dev = a_codes.device
        _check_tensor(a_codes, "a_codes", (T, H), dev, (u8,))
        _check_tensor(b_codes, "b_codes", (N, H), dev, (u8,))
        _check_tensor(a_scale, "a_scale", (T, HB), dev, (f32,))
        _check_tensor(b_scale, "b_scale", (NB, HB), dev, (f32,))
    if out is None:
        out, = _new(stream, a_codes.device, ((T, N), torch.bfloat16))
    else:
        _check_tensor(out, "out", (T, N), a_codes.device)
    c = _context_of(ctx, index)
    return (c.handle, a_codes.data_ptr(), a_scale.data_ptr(), b_codes.data_ptr(),
            b_scale.data_ptr(), T, N, H, out.data_ptr(), _raw_stream(stream, index)), out, c


def prepare_fp8_matmul(a_codes, a_scale, b_codes, b_scale, out=None, ctx=None, stream=None):
    """``fp8_matmul`` checked and marshalled once."""
    args, out, c = _fp8_matmul_args(a_codes, a_scale, b_codes, b_scale, out, ctx, stream)
    return PreparedCall(_load().farn_fp8_matmul, args, "farn_fp8_matmul", out,
                        (a_codes, a_scale, b_codes, b_scale, c))


def fp8_matmul(a_codes, a_scale, b_codes, b_scale, out=None, ctx=None, stream=None):
    """The product of two E4M3 tensors with block scales, a [T,H] (scales
    [T,ceil(H/128)]) and b [N,H] (scales [ceil(N/128),ceil(H/128)]), as
    ``fp8_quantize`` gives them with block_rows 1 and 128, in bf16 [T,N]."""
    args, out, _ = _fp8_matmul_args(a_codes, a_scale, b_codes, b_scale, out, ctx, stream)
    _call((_lib or _load()).farn_fp8_matmul, args, "farn_fp8_matmul")
    return out


def _fp8_grouped_args(x, x_scale, weights, w_scale, offsets, rows, out, workspace, ctx, stream):
    torch = _torch or _load_torch()
    u8, i32, f32 = torch.uint8, torch.int32, torch.float32
    sx, sw, index = x.shape, weights.shape, x.get_device()
    if len(sx) != 2 or len(sw) != 3:
        raise ValueError("x must be [rows, H] and weights [E, N, H]")
    n_rows, H = sx
    E, N, HW = sw
    HB, NB = -(-H // 128), -(-N // 128)
    if not (HW == H and index >= 0 and weights.get_device() == index and
            x_scale.get_device() == index and w_scale.get_device() == index and
            offsets.get_device() == index and x.dtype is u8 and weights.dtype is u8 and
            x_scale.dtype is f32 and w_scale.dtype is f32 and offsets.dtype is i32 and
            x_scale.shape == (n_rows, HB) and w_scale.shape == (E, NB, HB) and
            offsets.shape == (E + 1,) and x.is_contiguous() and weights.is_contiguous() and
            x_scale.is_contiguous() and w_scale.is_contiguous() and offsets.is_contiguous()):
        dev = x.device
        _check_tensor(x, "x", (n_rows, H), dev, (u8,))
        _check_tensor(x_scale, "x_scale", (n_rows, HB), dev, (f32,))
        _check_tensor(weights, "weights", (E, N, H), dev, (u8,))
        _check_tensor(w_scale, "w_scale", (E, NB, HB), dev, (f32,))
        _check_tensor(offsets, "offsets", (E + 1,), dev, (i32,))
    S = n_rows
    if rows is not None:
        sr = rows.shape
        S = sr[0] if len(sr) == 1 else -1
        if not (S >= 0 and rows.dtype is i32 and rows.get_device() == index and
                rows.is_contiguous()):
            _check_tensor(rows, "rows", (S,), x.device, (i32,))
    if out is None:
        out, = _new(stream, x.device, ((S, N), torch.bfloat16))
    else:
        _check_tensor(out, "out", (S, N), x.device)
    c = _context_of(ctx, index)
    if workspace is not None:
        _check_tensor(workspace, "workspace", workspace.shape, x.device, (u8,))
    elif rows is not None:
        n = ctypes.c_int64()            # stays 0 where the call itself will be refused
        (_lib or _load()).farn_fp8_grouped_workspace(c.handle, S, E, N, H, ctypes.byref(n))
        if n.value:
            workspace, = _new(stream, x.device, (n.value, u8), returned=False)
    return (c.handle, x.data_ptr(), x_scale.data_ptr(), n_rows,
            None if rows is None else rows.data_ptr(), S, weights.data_ptr(), w_scale.data_ptr(),
            E, offsets.data_ptr(), N, H, out.data_ptr(),
            None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel(),
            _raw_stream(stream, index)), out, (c, workspace)


def prepare_fp8_grouped_matmul(x, x_scale, weights, w_scale, offsets, rows=None, out=None,
                               workspace=None, ctx=None, stream=None):
    """``fp8_grouped_matmul`` checked and marshalled once; the call keeps its
    workspace."""
    args, out, c = _fp8_grouped_args(x, x_scale, weights, w_scale, offsets, rows, out, workspace,
                                     ctx, stream)
    return PreparedCall(_load().farn_fp8_grouped_matmul, args, "farn_fp8_grouped_matmul", out,
                        (x, x_scale, weights, w_scale, offsets, rows, c))


def fp8_grouped_matmul(x, x_scale, weights, w_scale, offsets, rows=None, out=None,
                       workspace=None, ctx=None, stream=None):
    """``grouped_matmul`` on E4M3 codes with block scales: x uint8 [n,H] with
    x_scale fp32 [n,ceil(H/128)], weights uint8 [E,N,H] with w_scale fp32
    [E,ceil(N/128),ceil(H/128)], as ``fp8_quantize`` gives them with block_rows
    1 and 128.  A long call with rows lays them side by side in a workspace
    (uint8; ``farn_fp8_grouped_workspace`` bytes), which is taken from torch if
    none is given.  Returns out bf16 [S,N]."""
    args, out, _ = _fp8_grouped_args(x, x_scale, weights, w_scale, offsets, rows, out, workspace,
                                     ctx, stream)
    _call((_lib or _load()).farn_fp8_grouped_matmul, args, "farn_fp8_grouped_matmul")
    return out


def kv_cache(n_pages: int, page_size: int, heads: int, head_dim: int, format: str = "fp8",
             device="cuda"):
    """The tensors of an empty paged cache of keys and values: (k_codes,
    v_codes, k_scale, v_scale).  "fp8": codes uint8
    [n_pages,page_size,heads,head_dim] and scales fp32
    [n_pages,page_size,heads]; "nvfp4": codes uint8 [..,head_dim/2] and scales
    uint8 [..,head_dim/16], as ``nvfp4_quantize`` gives them.  Zeros: every
    slot reads as 0."""
    torch = _torch or _load_torch()
    base = (int(n_pages), int(page_size), int(heads))
    D = int(head_dim)
    if format == "fp8":
        shapes, dt = ((*base, D), base), torch.float32
    elif format == "nvfp4":
        if D % 16:
            raise ValueError(f"NVFP4 needs head_dim % 16 == 0, got {D}")
        shapes, dt = ((*base, D // 2), (*base, D // 16)), torch.uint8
    else:
        raise ValueError(f'format must be "fp8" or "nvfp4", got {format!r}')
    new = lambda s, d: torch.zeros(s, dtype=d, device=device)  # noqa: E731
    return (new(shapes[0], torch.uint8), new(shapes[0], torch.uint8), new(shapes[1], dt),
            new(shapes[1], dt))


def _cache_args(cache, tensor_scales, index, dev):
    """The C struct of a cache's four tensors."""
    kc, vc, ks, vs = cache
    u8, sc, ss = _torch.uint8, kc.shape, ks.shape
    kind = ks.dtype
    if len(sc) != 4:
        raise ValueError("the cache's codes must be [n_pages, page_size, heads, ..]")
    P, page, H, D = sc
    if kind is _torch.float32:
        format, gk, gv = FARN_CACHE_FP8, 1.0, 1.0
        fits = ss == sc[:3]
    else:
        format = FARN_CACHE_NVFP4
        D *= 2
        if D % 16:
            raise ValueError(f"NVFP4 needs head_dim % 16 == 0, got {D}")
        if tensor_scales is None:
            raise ValueError("an NVFP4 cache needs tensor_scales (keys', values')")
        gk, gv = tensor_scales
        fits = kind is u8 and ss == (P, page, H, D // 16)
    if not (fits and vs.dtype is kind and kc.dtype is u8 and vc.dtype is u8 and vc.shape == sc and
            vs.shape == ss and kc.get_device() == index and vc.get_device() == index and
            ks.get_device() == index and vs.get_device() == index and kc.is_contiguous() and
            vc.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        shape = tuple(sc[:3]) if format == FARN_CACHE_FP8 else (P, page, H, D // 16)
        for t, name, want, dt in ((kc, "k_codes", sc, u8), (vc, "v_codes", sc, u8),
                                  (ks, "k_scale", shape, kind), (vs, "v_scale", shape, kind)):
            _check_tensor(t, "the cache's " + name, want, dev,
                          (dt if dt is _torch.float32 else u8,))
    return KvCache(format, page, P, H, D, kc.data_ptr(), vc.data_ptr(), ks.data_ptr(),
                   vs.data_ptr(), gk, gv)


def _check_heads(x, name, index, dev, T, heads, D):
    """What the short checks of [T, heads, D] turned down: heads contiguous
    within a token, tokens anywhere behind each other."""
    if not isinstance(x, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dim() != 3:
        raise ValueError(f"{name} must be [T, heads, D]")
    if x.dtype is not _torch.bfloat16:
        raise TypeError(f"{name} must be {_torch.bfloat16}, got {x.dtype}")
    if not x.is_cuda or x.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {x.device}")
    if tuple(x.shape) != (T, heads, D):
        raise ValueError(f"{name} must have shape {(T, heads, D)}, got {tuple(x.shape)}")
    st = x.stride()
    if (D > 1 and st[2] != 1) or (heads > 1 and st[1] != D):
        raise ValueError(f"{name}'s heads must lie one after the other within a token")


def _token_stride(x, name, index, dev, T, heads, D):
    """The stride of the tokens of a tensor [T, heads, D]."""
    st = x.stride()
    if not (len(st) == 3 and st[2] == 1 and st[1] == D and x.dtype is _torch.bfloat16 and
            x.get_device() == index and index >= 0 and x.shape == (T, heads, D)):
        _check_heads(x, name, index, dev, T, heads, D)
    return st[0] if T > 1 else heads * D


def _heads_shape(x, name):
    sx = x.shape
    if len(sx) != 3:
        raise ValueError(f"{name} must be [T, heads, D]")
    return sx


def _check_rope(positions, freqs, sections, T, D, dev):
    """What the short checks of a rotation turned down."""
    i32, f32 = _torch.int32, _torch.float32
    R = 2 * freqs.shape[0] if freqs.dim() == 1 else -1
    if not 0 < R <= D:
        raise ValueError(f"freqs must be [R / 2] for R in 2..{D}, got {tuple(freqs.shape)}")
    if positions is None or positions.dim() not in (1, 2) or positions.shape[-1] != T:
        raise ValueError(f"positions must be [T] or [axes, T] for T = {T}")
    axes = positions.shape[0] if positions.dim() == 2 else 1
    if not 1 <= axes <= 4:
        raise ValueError(f"positions must have 1..4 axes, got {axes}")
    _check_tensor(positions, "positions", positions.shape, dev, (i32,))
    _check_tensor(freqs, "freqs", (R // 2,), dev, (f32,))
    if axes > 1 and sections is None:
        raise ValueError("positions of several axes need sections")
    if sections is not None and (len(sections) != axes or min(sections) < 0 or
                                 sum(sections) != R // 2):
        raise ValueError(f"sections must be {axes} counts of pairs with the sum {R // 2}, got "
                         f"{tuple(sections)}")


_section_arrays = tuple(ctypes.c_int * n for n in range(5))


def _rope_args(positions, freqs, sections, T, D, index, dev):
    """(positions, axes, sections, freqs, R) as the C call takes them."""
    if freqs is None:
        return None, 0, None, None, 0
    half = freqs.shape[0] if freqs.dim() == 1 else 0
    sp = positions.shape if positions is not None else ()
    axes = sp[0] if len(sp) == 2 else 1
    if not (0 < half <= D // 2 and sp and sp[-1] == T and 1 <= axes <= 4 and len(sp) <= 2 and
            positions.dtype is _torch.int32 and freqs.dtype is _torch.float32 and
            positions.get_device() == index and freqs.get_device() == index and
            positions.is_contiguous() and freqs.is_contiguous() and
            (axes == 1 if sections is None else len(sections) == axes and
             sum(sections) == half and min(sections) >= 0)):
        _check_rope(positions, freqs, sections, T, D, dev)
    pairs = (half,) if sections is None else sections
    return positions.data_ptr(), axes, _section_arrays[axes](*pairs), freqs.data_ptr(), 2 * half


def _weight_arg(w, name, D, index, dev):
    if w is None:
        return None
    if not (w.get_device() == index and w.dtype is _torch.bfloat16 and w.shape == (D,) and
            w.is_contiguous()):
        _check_tensor(w, name, (D,), dev)
    return w.data_ptr()


def _qk_args(q, k, q_weight, k_weight, eps, positions, freqs, sections, interleaved, out, ctx,
             stream):
    torch = _torch or _load_torch()
    index, dev, bf = q.get_device(), q.device, torch.bfloat16
    T, HQ, D = _heads_shape(q, "q")
    HK = _heads_shape(k, "k")[1]
    q_stride = _token_stride(q, "q", index, dev, T, HQ, D)
    k_stride = _token_stride(k, "k", index, dev, T, HK, D)
    pos, axes, sect, fr, R = _rope_args(positions, freqs, sections, T, D, index, dev)
    if out is None:
        out = _new(stream, dev, ((T, HQ, D), bf), ((T, HK, D), bf))
        qs, ks = HQ * D, HK * D
    else:
        out = tuple(out)
        if len(out) != 2:
            raise ValueError("out must be (q, k)")
        qs = _token_stride(out[0], "the output of q", index, dev, T, HQ, D)
        ks = _token_stride(out[1], "the output of k", index, dev, T, HK, D)
    c = _context_of(ctx, index)
    return (c.handle, T, D, q.data_ptr(), HQ, q_stride, k.data_ptr(), HK, k_stride,
            _weight_arg(q_weight, "q_weight", D, index, dev),
            _weight_arg(k_weight, "k_weight", D, index, dev), eps, pos, axes, sect, fr, R,
            1 if interleaved else 0, out[0].data_ptr(), qs, out[1].data_ptr(), ks,
            _raw_stream(stream, index)), out, c


def prepare_qk_norm_rope(q, k, q_weight, k_weight, eps: float, positions=None, freqs=None,
                         sections=None, interleaved: bool = False, out=None, ctx=None,
                         stream=None):
    """``qk_norm_rope`` checked and marshalled once."""
    args, out, c = _qk_args(q, k, q_weight, k_weight, eps, positions, freqs, sections,
                            interleaved, out, ctx, stream)
    return PreparedCall(_load().farn_qk_norm_rope, args, "farn_qk_norm_rope", out,
                        (q, k, q_weight, k_weight, positions, freqs, c))


def qk_norm_rope(q, k, q_weight, k_weight, eps: float, positions=None, freqs=None, sections=None,
                 interleaved: bool = False, out=None, ctx=None, stream=None):
    """RMSNorm of every query and key head and its rotation by position, in one
    pass: q bf16 [T,HQ,D], k bf16 [T,HK,D] (heads contiguous within a token;
    tokens may lie further apart, as in a projection's output), weights bf16
    [D] (None: no norm), positions int32 [T] or [axes,T], freqs fp32 [R/2]
    (radians per position; None: no rotation), sections the number of pairs
    that turn by each axis.  Pairs are (j, j + R/2), or neighbours with
    `interleaved`.  out may be (q, k) themselves.  Returns (q, k)."""
    args, out, _ = _qk_args(q, k, q_weight, k_weight, eps, positions, freqs, sections,
                            interleaved, out, ctx, stream)
    _call((_lib or _load()).farn_qk_norm_rope, args, "farn_qk_norm_rope")
    return out


def _slots_arg(slots, T, index, dev):
    if not (slots.get_device() == index and slots.dtype is _torch.int32 and
            slots.shape == (T,) and slots.is_contiguous()):
        _check_tensor(slots, "slots", (T,), dev, (_torch.int32,))
    return slots.data_ptr()


def _cache_of(cache, tensor_scales, index, dev, HK, D):
    store = _cache_args(cache, tensor_scales, index, dev)
    if store.heads != HK or store.head_dim != D:
        raise ValueError(f"the cache has {store.heads} heads of {store.head_dim}, k has {HK} of "
                         f"{D}")
    return store


def _qk_cache_args(q, k, v, q_weight, k_weight, eps, positions, freqs, cache, slots,
                   tensor_scales, sections, interleaved, out, ctx, stream):
    torch = _torch or _load_torch()
    index, dev = q.get_device(), q.device
    T, HQ, D = _heads_shape(q, "q")
    HK = _heads_shape(k, "k")[1]
    q_stride = _token_stride(q, "q", index, dev, T, HQ, D)
    k_stride = _token_stride(k, "k", index, dev, T, HK, D)
    v_stride = _token_stride(v, "v", index, dev, T, HK, D)
    pos, axes, sect, fr, R = _rope_args(positions, freqs, sections, T, D, index, dev)
    slots_at = _slots_arg(slots, T, index, dev)
    store = _cache_of(cache, tensor_scales, index, dev, HK, D)
    if out is None:
        out, = _new(stream, dev, ((T, HQ, D), torch.bfloat16))
        qs = HQ * D
    else:
        qs = _token_stride(out, "the output of q", index, dev, T, HQ, D)
    c = _context_of(ctx, index)
    return (c.handle, T, D, q.data_ptr(), HQ, q_stride, k.data_ptr(), k_stride, v.data_ptr(),
            v_stride, HK, _weight_arg(q_weight, "q_weight", D, index, dev),
            _weight_arg(k_weight, "k_weight", D, index, dev), eps, pos, axes, sect, fr, R,
            1 if interleaved else 0, out.data_ptr(), qs, ctypes.byref(store), slots_at,
            _raw_stream(stream, index)), out, c


def prepare_qk_norm_rope_cache(q, k, v, q_weight, k_weight, eps: float, positions, freqs, cache,
                               slots, tensor_scales=None, sections=None,
                               interleaved: bool = False, out=None, ctx=None, stream=None):
    """``qk_norm_rope_cache`` checked and marshalled once."""
    args, out, c = _qk_cache_args(q, k, v, q_weight, k_weight, eps, positions, freqs, cache,
                                  slots, tensor_scales, sections, interleaved, out, ctx, stream)
    return PreparedCall(_load().farn_qk_norm_rope_cache, args, "farn_qk_norm_rope_cache", out,
                        (q, k, v, q_weight, k_weight, positions, freqs, cache, slots, c))


def qk_norm_rope_cache(q, k, v, q_weight, k_weight, eps: float, positions, freqs, cache, slots,
                       tensor_scales=None, sections=None, interleaved: bool = False, out=None,
                       ctx=None, stream=None):
    """``qk_norm_rope`` with keys and values going into a cache (the four
    tensors of ``kv_cache``): token t's keys, normed and rotated, and its values
    v bf16 [T,HK,D], as they are, to slot slots[t] (int32 [T]; one outside the
    cache is skipped, and no two may be the same).  tensor_scales: the keys' and
    the values' of an NVFP4 cache.  Returns q."""
    args, out, _ = _qk_cache_args(q, k, v, q_weight, k_weight, eps, positions, freqs, cache,
                                  slots, tensor_scales, sections, interleaved, out, ctx, stream)
    _call((_lib or _load()).farn_qk_norm_rope_cache, args, "farn_qk_norm_rope_cache")
    return out


def _kv_write_args(k, v, cache, slots, tensor_scales, ctx, stream):
    _torch or _load_torch()
    index, dev = k.get_device(), k.device
    T, HK, D = _heads_shape(k, "k")
    k_stride = _token_stride(k, "k", index, dev, T, HK, D)
    v_stride = _token_stride(v, "v", index, dev, T, HK, D)
    slots_at = _slots_arg(slots, T, index, dev)
    store = _cache_of(cache, tensor_scales, index, dev, HK, D)
    c = _context_of(ctx, index)
    return (c.handle, T, k.data_ptr(), k_stride, v.data_ptr(), v_stride, ctypes.byref(store),
            slots_at, _raw_stream(stream, index)), c


def prepare_kv_write(k, v, cache, slots, tensor_scales=None, ctx=None, stream=None):
    """``kv_write`` checked and marshalled once; the call returns the cache."""
    args, c = _kv_write_args(k, v, cache, slots, tensor_scales, ctx, stream)
    return PreparedCall(_load().farn_kv_write, args, "farn_kv_write", cache, (k, v, slots, c))


def kv_write(k, v, cache, slots, tensor_scales=None, ctx=None, stream=None):
    """Keys and values, bf16 [T,heads,head_dim], quantised into slots[t] of a
    cache as they are; slots and tensor_scales as for ``qk_norm_rope_cache``.
    Returns the cache."""
    args, _ = _kv_write_args(k, v, cache, slots, tensor_scales, ctx, stream)
    _call((_lib or _load()).farn_kv_write, args, "farn_kv_write")
    return cache


def _kv_read_args(cache, table, offsets, n_tokens, tensor_scales, out, ctx, stream):
    torch = _torch or _load_torch()
    i32 = torch.int32
    index, dev = cache[0].get_device(), cache[0].device
    if index < 0:
        _check_tensor(cache[0], "the cache's k_codes", cache[0].shape, dev, (torch.uint8,))
    store = _cache_args(cache, tensor_scales, index, dev)
    st = table.shape
    if len(st) != 2:
        raise ValueError("table must be [B, width]")
    B, width = st
    n = int(n_tokens)
    if n < 0:
        raise ValueError(f"n_tokens must not be negative, got {n}")
    if not (table.get_device() == index and offsets.get_device() == index and
            table.dtype is i32 and offsets.dtype is i32 and offsets.shape == (B + 1,) and
            table.is_contiguous() and offsets.is_contiguous()):
        _check_tensor(table, "table", (B, width), dev, (i32,))
        _check_tensor(offsets, "offsets", (B + 1,), dev, (i32,))
    shape = (n, store.heads, store.head_dim)
    if out is None:
        out = _new(stream, dev, (shape, torch.bfloat16), (shape, torch.bfloat16))
    else:
        out = tuple(out)
        if len(out) != 2:
            raise ValueError("out must be (k, v)")
        _check_tensor(out[0], "the output of k", shape, dev)
        _check_tensor(out[1], "the output of v", shape, dev)
    c = _context_of(ctx, index)
    return (c.handle, ctypes.byref(store), table.data_ptr(), B, width, offsets.data_ptr(), n,
            out[0].data_ptr(), out[1].data_ptr(), _raw_stream(stream, index)), out, c


def prepare_kv_read(cache, table, offsets, n_tokens: int, tensor_scales=None, out=None, ctx=None,
                    stream=None):
    """``kv_read`` checked and marshalled once."""
    args, out, c = _kv_read_args(cache, table, offsets, n_tokens, tensor_scales, out, ctx, stream)
    return PreparedCall(_load().farn_kv_read, args, "farn_kv_read", out,
                        (cache, table, offsets, c))


def kv_read(cache, table, offsets, n_tokens: int, tensor_scales=None, out=None, ctx=None,
            stream=None):
    """The contexts of B sequences back from a cache, in bf16, one after the
    other: table int32 [B,width] holds each sequence's pages, offsets int32
    [B+1] its first output token.  Returns (k, v), bf16
    [n_tokens,heads,head_dim]; a page outside the cache reads as zeros, and
    tokens that no sequence has are left as they were."""
    args, out, _ = _kv_read_args(cache, table, offsets, n_tokens, tensor_scales, out, ctx, stream)
    _call((_lib or _load()).farn_kv_read, args, "farn_kv_read")
    return out
