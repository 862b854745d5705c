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
``nvfp4_quantize``, ``nvfp4_dequantize`` and ``nvfp4_matmul``.  Every
arithmetic step runs in the CUDA kernels.  There is no CPU fallback: if the library
is not built, every call raises.
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
        out = tuple(torch.empty((T, H), dtype=torch.bfloat16, device=dev) for _ in range(3))
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
        out = (torch.empty((T, H), dtype=torch.bfloat16, device=dev),
               torch.empty((T, H), dtype=torch.bfloat16, device=dev),
               torch.empty((T, H), dtype=torch.bfloat16, device=dev) if write_norm else None,
               torch.empty((T, H), dtype=torch.uint8, device=dev),
               torch.empty((T,), dtype=torch.float32, device=dev))
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
        out = (torch.empty((T, H), dtype=torch.bfloat16, device=dev),
               torch.empty((T, H), dtype=torch.bfloat16, device=dev),
               torch.empty((T, H), dtype=torch.bfloat16, device=dev) if write_norm else None,
               torch.empty((T, H // 2), dtype=torch.uint8, device=dev),
               torch.empty((T, H // 16), dtype=torch.uint8, device=dev))
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
        out = tuple(torch.empty((T, H), dtype=torch.bfloat16, device=dev) for _ in range(3))
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
        dev = logits.device
        pairs = (T, K)
        out = (torch.empty(pairs, dtype=i32, device=dev),
               torch.empty(pairs, dtype=f32, device=dev),
               torch.empty(pairs, dtype=i32, device=dev),
               torch.empty((T * K,), dtype=i32, device=dev),
               torch.empty((E + 1,), dtype=i32, device=dev))
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
        out = torch.empty((S, N), dtype=bf, device=x.device)
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
        dev = x.device
        out = (torch.empty((T, H // 2), dtype=u8, device=dev),
               torch.empty((T, H // 16), dtype=u8, device=dev))
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
        out = torch.empty((T, H), dtype=torch.bfloat16, device=codes.device)
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
        out = torch.empty((T, N), dtype=bf, device=a_codes.device)
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
