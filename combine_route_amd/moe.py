"""Python binding of include/moe.h: the layer operators around the dispatch
and the combine. As the rest of the package it only marshals arguments: every
tensor is checked to be a contiguous device tensor of the right element type
and shape, all on one device, before a pointer reaches the library, and the
call runs on that device, on the given stream or torch's current one there.
"""
import ctypes
from typing import Optional

import torch

from . import (_F32, _I32, _TORCH, EP_BF16, EP_FP16, EP_FP8_E4M3, EpConfig, _check, _stream,
               load)

MOE_FP32 = 3
MOE_EPILOGUE_ROWS, MOE_EPILOGUE_SWIGLU = 0, 1
MOE_EXPORTED = ("moe_rms_norm", "moe_grouped_gemm", "moe_combine_backward",
                "moe_dispatch_backward")

_DTYPE_CODE = {torch.bfloat16: EP_BF16, torch.float16: EP_FP16}
_ROWS = (torch.bfloat16, torch.float16)
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


_fns = {}


def _lib():
    """The library with its moe_ functions declared."""
    if not _fns:
        lib = _declare(load())
        # all at once: another thread may be looking
        _fns.update({name: getattr(lib, name) for name in MOE_EXPORTED})
    return load()


def _refuse(t, name, shape, dtypes, index):
    """Says what is wrong with a tensor that _ptr does not accept."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU, not {t.device}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def _ptr(t: Optional[torch.Tensor], name: str, shape, dtypes, index: int):
    """Address of a contiguous tensor of exactly this shape, one of these
    element types and on device `index` (CPU tensors are on -1); None stays
    None."""
    if t is None:
        return None
    try:
        if (t.get_device() == index and t.shape == shape and t.dtype in dtypes and
                t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, shape, dtypes, index)


def _index_of(t, name: str) -> int:
    """The device a call runs on: its first tensor's."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, not {t.device}")
    return t.get_device()


def _call(fn, index, stream, *args):
    """One library call with `index` the current device, on the given stream
    or torch's current one there."""
    if not _fns:
        _lib()
    if isinstance(stream, torch.cuda.Stream) and stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    if torch.cuda.current_device() == index:
        rc = _fns[fn](*args, _stream(stream, index))
    else:
        with torch.cuda.device(index):
            rc = _fns[fn](*args, _stream(stream, index))
    if rc:
        _check(fn, rc)


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
    index = _index_of(x, "x")
    _index_of(weight, "weight")
    dtype = _DTYPE_CODE.get(x.dtype)
    if dtype is None:
        raise ValueError(f"x must be bf16 or fp16, not {x.dtype}")
    shape = x.shape
    H = shape[-1] if shape else 0
    if H == 0:
        raise ValueError("x must have rows of at least one element")
    rows = x.numel() // H
    if residual is not None and residual_out is None:
        residual_out = residual
    same = (x.dtype,)
    group = 0
    if counts is not None:
        if len(shape) < 2 or shape[0] == 0:
            raise ValueError("counts needs rows of shape [G, ..., H] with G >= 1")
        group = max(1, rows // shape[0])
    a = MoeRmsNormArgs(
        _ptr(x, "x", shape, same, index), _ptr(residual, "residual", shape, same, index),
        _ptr(residual_out, "residual_out", shape, same, index),
        _ptr(weight, "weight", (H,), (x.dtype, torch.float32), index),
        _ptr(out, "out", shape, same, index), _ptr(codes, "codes", shape, _CODES, index),
        _ptr(scales, "scales", shape[:-1] + (H // 128,), _F32, index),
        _ptr(counts, "counts", shape[:1], _I32, index), rows, group, H, dtype,
        dtype if weight.dtype == x.dtype else MOE_FP32, eps)
    _call("moe_rms_norm", index, stream, ctypes.byref(a))


def _product_args(a, a_scales, b, b_scales, counts):
    """Device, checked sizes and addresses of a grouped product's inputs."""
    index = _index_of(a, "a")
    _index_of(b, "b")
    for t, name in ((a, "a"), (b, "b")):
        if t.dim() != 3:
            raise ValueError(f"{name} must have 3 dimensions, not {t.dim()}")
    groups, cap, k = a.shape
    n = b.shape[1]
    blocks = -(-k // 128)
    return index, (groups, cap, n, k), (
        _ptr(a, "a", a.shape, _CODES, index),
        _ptr(a_scales, "a_scales", (groups, cap, blocks), _F32, index),
        _ptr(b, "b", (groups, n, k), _CODES, index),
        _ptr(b_scales, "b_scales", (groups, -(-n // 128), blocks), _F32, index),
        _ptr(counts, "counts", (groups,), _I32, index))


def moe_grouped_gemm(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor,
                     b_scales: torch.Tensor, out: torch.Tensor,
                     counts: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_grouped_gemm() (include/moe.h) to bf16 / fp16 rows: a [G, cap, K]
    E4M3 rows with a_scales [G, cap, K / 128], b [G, N, K] E4M3 weights with
    b_scales [G, ceil(N / 128), K / 128]; out [G, cap, N]. counts: int32 [G]
    rows of each group (default: cap). Sums are FP32's but for the matrix
    instruction's first step: of 8 neighbouring products each is cut to a
    multiple of 2^(E - 13), E the eight's largest sum of exponents (1.3e-5 of
    an ordinary row's norm, more where large products of one eight cancel)."""
    index, (groups, cap, n, k), ptrs = _product_args(a, a_scales, b, b_scales, counts)
    _index_of(out, "out")
    args = MoeGroupedGemmArgs(*ptrs, _ptr(out, "out", (groups, cap, n), _ROWS, index), None,
                              groups, cap, n, k, _DTYPE_CODE[out.dtype], MOE_EPILOGUE_ROWS)
    _call("moe_grouped_gemm", index, stream, ctypes.byref(args))


def moe_grouped_gemm_swiglu(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor,
                            b_scales: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                            counts: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_grouped_gemm() (include/moe.h) with MOE_EPILOGUE_SWIGLU: b [G, 2 I,
    K] holds each expert's I gate rows, then its I up rows; codes [G, cap, I]
    and scales [G, cap, I / 128] get silu(gate) * up as E4M3. Every sum is in
    FP32."""
    index, (groups, cap, n, k), ptrs = _product_args(a, a_scales, b, b_scales, counts)
    args = MoeGroupedGemmArgs(*ptrs, _ptr(codes, "codes", (groups, cap, n // 2), _CODES, index),
                              _ptr(scales, "scales", (groups, cap, n // 256), _F32, index),
                              groups, cap, n, k, EP_FP8_E4M3, MOE_EPILOGUE_SWIGLU)
    _call("moe_grouped_gemm", index, stream, ctypes.byref(args))


def moe_combine_backward(eplan: int, cfg: EpConfig, cap: int, grad_out, indices, weights, packed_y,
                         grad_packed_y, grad_weights, stream=None) -> None:
    """moe_combine_backward(); tensors as in include/moe.h."""
    index = _index_of(grad_out, "grad_out")
    W, M, k, H = (cfg.world_size, cfg.max_num_inp_token_per_rank, cfg.num_experts_per_token,
                  cfg.hidden_dim)
    slots, packed = (W, M, k), (W, cfg.num_experts_per_rank, cap, H)
    dt = (_TORCH[cfg.combine_dtype],)
    a = MoeCombineBackwardArgs(
        _ptr(grad_out, "grad_out", (W, M, H), dt, index),
        _ptr(indices, "indices", slots, _I32, index), _ptr(weights, "weights", slots, _F32, index),
        _ptr(packed_y, "packed_y", packed, dt, index),
        _ptr(grad_packed_y, "grad_packed_y", packed, dt, index),
        _ptr(grad_weights, "grad_weights", slots, _F32, index))
    _call("moe_combine_backward", index, stream, eplan, ctypes.byref(a))


def moe_dispatch_backward(eplan: int, cfg: EpConfig, cap: int, grad_packed_x, grad_x,
                          stream=None) -> None:
    """moe_dispatch_backward(); tensors as in include/moe.h."""
    index = _index_of(grad_packed_x, "grad_packed_x")
    W, H = cfg.world_size, cfg.hidden_dim
    dt = (_TORCH[cfg.combine_dtype],)
    a = MoeDispatchBackwardArgs(
        _ptr(grad_packed_x, "grad_packed_x", (W, cfg.num_experts_per_rank, cap, H), dt, index),
        _ptr(grad_x, "grad_x", (W, cfg.max_num_inp_token_per_rank, H), dt, index))
    _call("moe_dispatch_backward", index, stream, eplan, ctypes.byref(a))
