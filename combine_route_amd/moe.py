"""Python binding of include/moe.h: the layer operators around the dispatch
and the combine. As the rest of the package it only marshals arguments: every
tensor is checked to be a contiguous device tensor of the right element type
and shape, all on one device, before a pointer reaches the library, and the
call runs on that device, on the given stream or torch's current one there.
"""
import contextlib
import ctypes
from typing import Optional

import torch

from . import (_F32, _I32, _TORCH, EP_BF16, EP_FP16, EP_FP8_E4M3, EpConfig, _check, _dev,
               _sizes, _stream, load)

MOE_FP32 = 3
MOE_EPILOGUE_ROWS, MOE_EPILOGUE_SWIGLU = 0, 1
MOE_EXPORTED = ("moe_rms_norm", "moe_grouped_gemm", "moe_combine_backward",
                "moe_dispatch_backward")

_DTYPE_CODE = {torch.bfloat16: EP_BF16, torch.float16: EP_FP16}
_CODES = (torch.uint8, torch.float8_e4m3fn)


class MoeRmsNormArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in (
        "x", "residual", "residual_out", "weight", "out", "codes", "scales", "row_counts")] +
        [("rows", ctypes.c_int64), ("group_rows", ctypes.c_int64), ("hidden", ctypes.c_int32),
         ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("eps", ctypes.c_float)])


class MoeGroupedGemmArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in (
        "a", "a_scales", "b", "b_scales", "counts", "out", "out_scales")] +
        [(n, ctypes.c_int32) for n in ("groups", "cap", "n", "k", "out_dtype", "epilogue")])


class MoeCombineBackwardArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "grad_out", "indices", "weights", "packed_y", "grad_packed_y", "grad_weights")]


class MoeDispatchBackwardArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("grad_packed_x", "grad_x")]


def _declare(lib):
    """Argument types of the moe_ functions, once a library."""
    if getattr(lib, "_moe_declared", False):
        return lib
    V = ctypes.c_void_p
    lib.moe_rms_norm.argtypes = [ctypes.POINTER(MoeRmsNormArgs), V]
    lib.moe_grouped_gemm.argtypes = [ctypes.POINTER(MoeGroupedGemmArgs), V]
    lib.moe_combine_backward.argtypes = [V, ctypes.POINTER(MoeCombineBackwardArgs), V]
    lib.moe_dispatch_backward.argtypes = [V, ctypes.POINTER(MoeDispatchBackwardArgs), V]
    for name in MOE_EXPORTED:
        getattr(lib, name).restype = ctypes.c_int
    lib._moe_declared = True
    return lib


def _lib():
    return _declare(load())


def _shaped(t: Optional[torch.Tensor], name: str, shape, dtypes):
    """Address of a tensor that has exactly this shape; None stays None."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    nbytes = t.numel() * t.element_size() if isinstance(t, torch.Tensor) else 0
    return _dev(t, name, nbytes, dtypes)


def _device_of(**tensors) -> int:
    """The one device all of a call's tensors are on."""
    index = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be on the GPU, not {t.device}")
        if index is None:
            index = t.device.index
        elif t.device.index != index:
            raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{index}")
    return index


def _call(fn, index, stream, *args):
    """One library call with `index` the current device."""
    other = torch.cuda.current_device() != index
    with torch.cuda.device(index) if other else contextlib.nullcontext():
        _check(fn, getattr(_lib(), fn)(*args, _stream(stream, index)))


def moe_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float,
                 out: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                 residual_out: Optional[torch.Tensor] = None,
                 codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                 counts: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_rms_norm() (include/moe.h): RMS norm of x's rows [..., H] (bf16 or
    fp16) times weight [H] (x's type or float32), after the residual's
    addition. residual_out (default: residual, in place) gets x + residual;
    out the normed rows in x's type; codes [..., H] and scales [..., H / 128]
    the same rows as E4M3 with a scale per 128 elements. counts: an int32
    tensor of one count per leading index of x ([G, R, H] rows with counts
    [G]); only the first counts[g] rows of group g are read and written."""
    index = _device_of(x=x, weight=weight, out=out, residual=residual, residual_out=residual_out,
                       codes=codes, scales=scales, counts=counts)
    dtype = _DTYPE_CODE.get(x.dtype)
    if dtype is None:
        raise ValueError(f"x must be bf16 or fp16, not {x.dtype}")
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("x must have rows of at least one element")
    H = x.shape[-1]
    rows = x.numel() // H
    if residual is not None and residual_out is None:
        residual_out = residual
    same = (x.dtype,)
    group = 0
    if counts is not None:
        if x.dim() < 2 or x.shape[0] == 0:
            raise ValueError("counts needs rows of shape [G, ..., H] with G >= 1")
        group = max(1, rows // x.shape[0])
    a = MoeRmsNormArgs(
        _shaped(x, "x", x.shape, same), _shaped(residual, "residual", x.shape, same),
        _shaped(residual_out, "residual_out", x.shape, same),
        _shaped(weight, "weight", (H,), (x.dtype, torch.float32)),
        _shaped(out, "out", x.shape, same), _shaped(codes, "codes", x.shape, _CODES),
        _shaped(scales, "scales", x.shape[:-1] + (H // 128,), _F32),
        _shaped(counts, "counts", x.shape[:1], _I32), rows, group, H, dtype,
        MOE_FP32 if weight.dtype == torch.float32 else dtype, eps)
    _call("moe_rms_norm", index, stream, ctypes.byref(a))


def _product_args(a, a_scales, b, b_scales, counts):
    """Checked sizes and addresses of a grouped product's inputs."""
    for t, name in ((a, "a"), (b, "b")):
        if t.dim() != 3:
            raise ValueError(f"{name} must have 3 dimensions, not {t.dim()}")
    groups, cap, k = a.shape
    n = b.shape[1]
    blocks = -(-k // 128)
    return (groups, cap, n, k), (
        _shaped(a, "a", (groups, cap, k), _CODES),
        _shaped(a_scales, "a_scales", (groups, cap, blocks), _F32),
        _shaped(b, "b", (groups, n, k), _CODES),
        _shaped(b_scales, "b_scales", (groups, -(-n // 128), blocks), _F32),
        _shaped(counts, "counts", (groups,), _I32))


def moe_grouped_gemm(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor,
                     b_scales: torch.Tensor, out: torch.Tensor,
                     counts: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_grouped_gemm() (include/moe.h) to bf16 / fp16 rows: a [G, cap, K]
    E4M3 rows with a_scales [G, cap, K / 128], b [G, N, K] E4M3 weights with
    b_scales [G, ceil(N / 128), K / 128]; out [G, cap, N]. counts: int32 [G]
    rows of each group (default: cap)."""
    index = _device_of(a=a, a_scales=a_scales, b=b, b_scales=b_scales, out=out, counts=counts)
    (groups, cap, n, k), ptrs = _product_args(a, a_scales, b, b_scales, counts)
    dtype = _DTYPE_CODE.get(out.dtype)
    if dtype is None:
        raise ValueError(f"out must be bf16 or fp16, not {out.dtype}")
    args = MoeGroupedGemmArgs(*ptrs, _shaped(out, "out", (groups, cap, n), None), None, groups,
                              cap, n, k, dtype, MOE_EPILOGUE_ROWS)
    _call("moe_grouped_gemm", index, stream, ctypes.byref(args))


def moe_grouped_gemm_swiglu(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor,
                            b_scales: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                            counts: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_grouped_gemm() (include/moe.h) with MOE_EPILOGUE_SWIGLU: b [G, 2 I,
    K] holds each expert's I gate rows, then its I up rows; codes [G, cap, I]
    and scales [G, cap, I / 128] get silu(gate) * up as E4M3."""
    index = _device_of(a=a, a_scales=a_scales, b=b, b_scales=b_scales, codes=codes, scales=scales,
                       counts=counts)
    (groups, cap, n, k), ptrs = _product_args(a, a_scales, b, b_scales, counts)
    args = MoeGroupedGemmArgs(*ptrs, _shaped(codes, "codes", (groups, cap, n // 2), _CODES),
                              _shaped(scales, "scales", (groups, cap, n // 256), _F32), groups,
                              cap, n, k, EP_FP8_E4M3, MOE_EPILOGUE_SWIGLU)
    _call("moe_grouped_gemm", index, stream, ctypes.byref(args))


def _packed_shape(cfg: EpConfig, cap: int):
    return (cfg.world_size, cfg.num_experts_per_rank, cap, cfg.hidden_dim)


def moe_combine_backward(eplan: int, cfg: EpConfig, cap: int, grad_out, indices, weights, packed_y,
                         grad_packed_y, grad_weights, stream=None) -> None:
    """moe_combine_backward(); tensors as in include/moe.h."""
    index = _device_of(grad_out=grad_out, indices=indices, weights=weights, packed_y=packed_y,
                       grad_packed_y=grad_packed_y, grad_weights=grad_weights)
    W, M, k, _, _, _ = _sizes(cfg)
    rows, slots = (W, M, cfg.hidden_dim), (W, M, k)
    packed, dt = _packed_shape(cfg, cap), (_TORCH[cfg.combine_dtype],)
    a = MoeCombineBackwardArgs(
        _shaped(grad_out, "grad_out", rows, dt), _shaped(indices, "indices", slots, _I32),
        _shaped(weights, "weights", slots, _F32), _shaped(packed_y, "packed_y", packed, dt),
        _shaped(grad_packed_y, "grad_packed_y", packed, dt),
        _shaped(grad_weights, "grad_weights", slots, _F32))
    _call("moe_combine_backward", index, stream, eplan, ctypes.byref(a))


def moe_dispatch_backward(eplan: int, cfg: EpConfig, cap: int, grad_packed_x, grad_x,
                          stream=None) -> None:
    """moe_dispatch_backward(); tensors as in include/moe.h."""
    index = _device_of(grad_packed_x=grad_packed_x, grad_x=grad_x)
    W, M, _, _, _, _ = _sizes(cfg)
    dt = (_TORCH[cfg.combine_dtype],)
    a = MoeDispatchBackwardArgs(
        _shaped(grad_packed_x, "grad_packed_x", _packed_shape(cfg, cap), dt),
        _shaped(grad_x, "grad_x", (W, M, cfg.hidden_dim), dt))
    _call("moe_dispatch_backward", index, stream, eplan, ctypes.byref(a))
