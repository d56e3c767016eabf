"""Python binding of include/moe_block.h: the operators of a whole MoE block.
As moe.py it only marshals arguments: every tensor is checked to be a
contiguous device tensor of the right element type and shape, all on one
device, before a pointer reaches the library, and the call runs on that device,
on the given stream or torch's current one there.
"""
import ctypes
from typing import Optional

import torch

from . import _F32, _I32, EP_ERR_ARG, EP_FP8_E4M3, EpError, _check, _stream, ep_last_error, load
from .moe import (_CODES, _DTYPE_CODE, _ROWS, MOE_EPILOGUE_ROWS, MOE_EPILOGUE_SWIGLU, MOE_FP32,
                  _index_of, _ptr)

MOE_INT8 = 4
BLOCK_EXPORTED = ("moe_block_norm", "moe_block_norm_backward",
                  "moe_block_norm_backward_workspace_bytes", "moe_quantize_int8",
                  "moe_grouped_gemm_int8", "moe_few_tokens", "moe_few_tokens_workspace_bytes")

_INT8 = (torch.int8,)


class MoeBlockNormArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in (
        "y", "residual", "residual_out", "post_weight", "gate", "pre_weight", "out", "codes",
        "scales", "row_counts")] +
        [(n, ctypes.c_int64) for n in ("rows", "group_rows", "gate_rows")] +
        [(n, ctypes.c_int32) for n in ("hidden", "dtype", "weight_dtype", "codes_dtype")] +
        [("residual_scale", ctypes.c_float), ("eps", ctypes.c_float)])


class MoeBlockNormBackwardArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in (
        "y", "h", "grad_h", "grad_out", "post_weight", "gate", "pre_weight", "grad_y",
        "grad_residual", "grad_post_weight", "grad_gate", "grad_pre_weight", "workspace",
        "row_counts")] +
        [(n, ctypes.c_int64) for n in ("workspace_bytes", "rows", "group_rows", "gate_rows")] +
        [(n, ctypes.c_int32) for n in ("hidden", "dtype", "weight_dtype")] +
        [("residual_scale", ctypes.c_float), ("eps", ctypes.c_float)])


class MoeQuantizeInt8Args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("rows", "codes", "scales", "row_counts")] +
                [("n_rows", ctypes.c_int64), ("group_rows", ctypes.c_int64),
                 ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32)])


class MoeGroupedGemmInt8Args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("a", "a_scales", "b", "b_scales", "counts",
                                                "out")] +
                [(n, ctypes.c_int32) for n in ("groups", "cap", "n", "k", "out_dtype",
                                               "epilogue")])


class MoeFewTokensArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in (
        "x", "indices", "weights", "gate_up", "gate_up_scales", "down", "down_scales", "out",
        "workspace")] + [("workspace_bytes", ctypes.c_int64)] +
        [(n, ctypes.c_int32) for n in ("tokens", "topk", "experts", "hidden", "inter", "dtype",
                                       "weight_dtype")])


def _declare(lib):
    """The functions of include/moe_block.h by name, with their types."""
    V, P = ctypes.c_void_p, ctypes.POINTER
    lib.moe_block_norm.argtypes = [P(MoeBlockNormArgs), V]
    lib.moe_block_norm_backward.argtypes = [P(MoeBlockNormBackwardArgs), V]
    lib.moe_block_norm_backward_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int32,
                                                            ctypes.c_int64]
    lib.moe_quantize_int8.argtypes = [P(MoeQuantizeInt8Args), V]
    lib.moe_grouped_gemm_int8.argtypes = [P(MoeGroupedGemmInt8Args), V]
    lib.moe_few_tokens.argtypes = [P(MoeFewTokensArgs), V]
    lib.moe_few_tokens_workspace_bytes.argtypes = [ctypes.c_int32] * 4
    fns = {name: getattr(lib, name) for name in BLOCK_EXPORTED}
    for name, fn in fns.items():
        fn.restype = ctypes.c_size_t if name.endswith("_bytes") else ctypes.c_int
    return fns


_fns = {}


def _fn(name):
    if not _fns:
        _fns.update(_declare(load()))  # all at once: another thread may be looking
    return _fns[name]


def _call(name, index, stream, args):
    """One library call with `index` the current device, on the given stream
    or torch's current one there."""
    fn = _fn(name)
    if isinstance(stream, torch.cuda.Stream) and stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    if torch.cuda.current_device() == index:
        rc = fn(ctypes.byref(args), _stream(stream, index))
    else:
        with torch.cuda.device(index):
            rc = fn(ctypes.byref(args), _stream(stream, index))
    if rc:
        _check(name, rc)


def _workspace_bytes(name, *sizes):
    n = _fn(name)(*sizes)
    if n == 0:
        raise EpError(name, EP_ERR_ARG, ep_last_error())
    return n


def _torch_stream(stream, index):
    """A call's stream as torch's object; None stays None (the current one)."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    # (torch's ExternalStream takes handle 0, the default stream, for none)
    handle, device = int(stream), torch.device("cuda", index)
    return (torch.cuda.ExternalStream(handle, device=device) if handle
            else torch.cuda.default_stream(device))


def _workspace(given, nbytes, index, stream):
    """The given workspace, or a new one that torch's allocator owns on the
    call's stream."""
    if given is not None:
        if not isinstance(given, torch.Tensor):
            raise TypeError("workspace must be a torch.Tensor")
        if not given.is_cuda or given.get_device() != index:
            raise ValueError(f"workspace is on {given.device}, the other tensors on cuda:{index}")
        if not given.is_contiguous():
            raise ValueError("workspace must be contiguous")
        have = given.numel() * given.element_size()
        if have < nbytes:
            raise ValueError(f"workspace holds {have} bytes; this call needs {nbytes}")
        return given
    with torch.cuda.stream(_torch_stream(stream, index)):
        return torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))


def _rows_of(t, name):
    """Device, shape, row length, number of rows and dtype code of rows [..., H]."""
    index = _index_of(t, name)
    dtype = _DTYPE_CODE.get(t.dtype)
    if dtype is None:
        raise ValueError(f"{name} must be bf16 or fp16, not {t.dtype}")
    shape = t.shape
    H = shape[-1] if shape else 0
    if H == 0:
        raise ValueError(f"{name} must have rows of at least one element")
    return index, shape, H, t.numel() // H, dtype


def _groups(counts, shape, rows):
    """Rows of each group that counts has one value for."""
    if counts is None:
        return 0
    if len(shape) < 2 or shape[0] == 0:
        raise ValueError("counts needs rows of shape [G, ..., H] with G >= 1")
    return max(1, rows // shape[0])


def _weights(weights, shape, H, rows, x_dtype, dtype, index):
    """Addresses of the post weight, gate and pre weight, rows a gate, and the
    weights' type, which they share."""
    post, gate, pre = weights
    some = post if post is not None else gate if gate is not None else pre
    wt = x_dtype if some is None else getattr(some, "dtype", x_dtype)
    if wt is not x_dtype and wt is not torch.float32:
        raise ValueError(f"weights must be {x_dtype} or torch.float32, not {wt}")
    gate_rows, gate_shape = 0, (H,)
    if gate is not None and isinstance(gate, torch.Tensor) and gate.dim() != 1:
        if len(shape) < 2 or shape[0] == 0:
            raise ValueError("a gate [G, H] needs rows of shape [G, ..., H] with G >= 1")
        gate_shape, gate_rows = (shape[0], H), rows // shape[0]
    return (_ptr(post, "post_weight", (H,), (wt,), index),
            _ptr(gate, "gate", gate_shape, (wt,), index),
            _ptr(pre, "pre_weight", (H,), (wt,), index), gate_rows,
            dtype if wt == x_dtype else MOE_FP32)


def moe_block_norm(y: torch.Tensor, residual: torch.Tensor, pre_weight: Optional[torch.Tensor],
                   eps: float, out: Optional[torch.Tensor] = None,
                   residual_out: Optional[torch.Tensor] = None,
                   post_weight: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                   codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                   counts: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_block_norm() (include/moe_block.h): h = residual_scale * residual +
    gate * norm(y) * post_weight to residual_out (default: residual, in place),
    and norm(h) * pre_weight to out in y's type and / or to codes [..., H] with
    scales: E4M3 codes (float8_e4m3fn or uint8) with scales [..., H / 128], or
    int8 codes with scales [...], one a row. y, residual: rows [..., H], bf16 or
    fp16. post_weight None: no norm of y. gate: [H], or [G, H] for rows [G, ...,
    H]. pre_weight None (without out and codes): h alone. The weights share a
    type, y's or float32. counts: int32, one count per leading index of y; only
    the first counts[g] rows of group g are read and written."""
    index, shape, H, rows, dtype = _rows_of(y, "y")
    _index_of(residual, "residual")
    if residual_out is None:
        residual_out = residual
    same = (y.dtype,)
    post_p, gate_p, pre_p, gate_rows, wt = _weights((post_weight, gate, pre_weight), shape, H,
                                                    rows, y.dtype, dtype, index)
    group = _groups(counts, shape, rows)
    int8 = isinstance(codes, torch.Tensor) and codes.dtype == torch.int8
    a = MoeBlockNormArgs(
        _ptr(y, "y", shape, same, index), _ptr(residual, "residual", shape, same, index),
        _ptr(residual_out, "residual_out", shape, same, index), post_p, gate_p, pre_p,
        _ptr(out, "out", shape, same, index),
        _ptr(codes, "codes", shape, _INT8 if int8 else _CODES + _INT8, index),
        _ptr(scales, "scales", shape[:-1] + (() if int8 else (H // 128,)), _F32, index),
        _ptr(counts, "counts", shape[:1], _I32, index), rows, group, gate_rows, H, dtype, wt,
        MOE_INT8 if int8 else EP_FP8_E4M3, residual_scale, eps)
    _call("moe_block_norm", index, stream, a)


def moe_block_norm_backward_workspace_bytes(rows: int, hidden: int, groups: int = 1) -> int:
    """Bytes of workspace that moe_block_norm_backward needs for rows of this
    many groups (the gates of a gate [G, H], or the counts; else 1); enough for
    calls on these rows in other groups, or none, too."""
    return _workspace_bytes("moe_block_norm_backward_workspace_bytes", rows, hidden, groups)


def moe_block_norm_backward(y: torch.Tensor, h: Optional[torch.Tensor], eps: float,
                            grad_y: torch.Tensor, grad_out: Optional[torch.Tensor] = None,
                            grad_h: Optional[torch.Tensor] = None,
                            grad_residual: Optional[torch.Tensor] = None,
                            pre_weight: Optional[torch.Tensor] = None,
                            post_weight: Optional[torch.Tensor] = None,
                            gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                            grad_pre_weight: Optional[torch.Tensor] = None,
                            grad_post_weight: Optional[torch.Tensor] = None,
                            grad_gate: Optional[torch.Tensor] = None,
                            counts: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_block_norm_backward() (include/moe_block.h): gradients of
    moe_block_norm from its y, the h it left in residual_out, and the gradients
    of its two results, grad_out (of out, codes' rounding taken as the identity)
    and grad_h (of residual_out); either may be None. Writes grad_y and, each
    if given, grad_residual, and in float32 grad_post_weight [H], grad_gate (the
    gate's shape) and grad_pre_weight [H], which are zeros if y has no rows.
    workspace: any tensor of moe_block_norm_backward_workspace_bytes bytes that
    no other call uses at the same time; None makes a new one."""
    index, shape, H, rows, dtype = _rows_of(y, "y")
    _index_of(grad_y, "grad_y")
    same = (y.dtype,)
    post_p, gate_p, pre_p, gate_rows, wt = _weights((post_weight, gate, pre_weight), shape, H,
                                                    rows, y.dtype, dtype, index)
    group = _groups(counts, shape, rows)
    gate_shape = gate.shape if isinstance(gate, torch.Tensor) else (H,)
    ws, nbytes = None, 0
    if rows and (grad_pre_weight is not None or grad_post_weight is not None or
                 grad_gate is not None):
        nbytes = moe_block_norm_backward_workspace_bytes(
            rows, H, shape[0] if gate_rows or counts is not None else 1)
        ws = _workspace(workspace, nbytes, index, stream)
    a = MoeBlockNormBackwardArgs(
        _ptr(y, "y", shape, same, index), _ptr(h, "h", shape, same, index),
        _ptr(grad_h, "grad_h", shape, same, index),
        _ptr(grad_out, "grad_out", shape, same, index), post_p, gate_p, pre_p,
        _ptr(grad_y, "grad_y", shape, same, index),
        _ptr(grad_residual, "grad_residual", shape, same, index),
        _ptr(grad_post_weight, "grad_post_weight", (H,), _F32, index),
        _ptr(grad_gate, "grad_gate", gate_shape, _F32, index),
        _ptr(grad_pre_weight, "grad_pre_weight", (H,), _F32, index),
        None if ws is None else ws.data_ptr(), _ptr(counts, "counts", shape[:1], _I32, index),
        nbytes, rows, group, gate_rows, H, dtype, wt, residual_scale, eps)
    _call("moe_block_norm_backward", index, stream, a)
    if rows == 0:  # the library writes nothing: these are sums over no rows
        with torch.cuda.stream(_torch_stream(stream, index)):
            for t in (grad_pre_weight, grad_post_weight, grad_gate):
                if t is not None:
                    t.zero_()


def moe_quantize_int8(rows: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                      counts: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_quantize_int8() (include/moe_block.h): rows [..., H] (bf16 or fp16) to
    codes [..., H] (int8) and scales [...] (float32, one a row). counts: int32,
    one count per leading index of rows; only the first counts[g] rows of group
    g are read and written."""
    index, shape, H, n_rows, dtype = _rows_of(rows, "rows")
    _index_of(codes, "codes")
    _index_of(scales, "scales")
    group = _groups(counts, shape, n_rows)
    a = MoeQuantizeInt8Args(
        _ptr(rows, "rows", shape, (rows.dtype,), index), _ptr(codes, "codes", shape, _INT8, index),
        _ptr(scales, "scales", shape[:-1], _F32, index),
        _ptr(counts, "counts", shape[:1], _I32, index), n_rows, group, H, dtype)
    _call("moe_quantize_int8", index, stream, a)


def _product(a, a_scales, b, b_scales, out, counts, stream, epilogue):
    index = _index_of(a, "a")
    _index_of(b, "b")
    _index_of(out, "out")
    for t, name in ((a, "a"), (b, "b")):
        if t.dim() != 3:
            raise ValueError(f"{name} must have 3 dimensions, not {t.dim()}")
    groups, cap, k = a.shape
    n = b.shape[1]
    width = n // 2 if epilogue == MOE_EPILOGUE_SWIGLU else n
    args = MoeGroupedGemmInt8Args(
        _ptr(a, "a", a.shape, _INT8, index), _ptr(a_scales, "a_scales", (groups, cap), _F32, index),
        _ptr(b, "b", (groups, n, k), _INT8, index),
        _ptr(b_scales, "b_scales", (groups, n), _F32, index),
        _ptr(counts, "counts", (groups,), _I32, index),
        _ptr(out, "out", (groups, cap, width), _ROWS, index), groups, cap, n, k,
        _DTYPE_CODE[out.dtype], epilogue)
    _call("moe_grouped_gemm_int8", index, stream, args)


def moe_grouped_gemm_int8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor,
                          b_scales: torch.Tensor, out: torch.Tensor,
                          counts: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_grouped_gemm_int8() (include/moe_block.h) to bf16 / fp16 rows: a [G,
    cap, K] int8 rows with a_scales [G, cap], b [G, N, K] int8 weights with
    b_scales [G, N]; out [G, cap, N]. counts: int32 [G] rows of each group
    (default: cap). Sums are exact, in 32-bit integers."""
    _product(a, a_scales, b, b_scales, out, counts, stream, MOE_EPILOGUE_ROWS)


def moe_grouped_gemm_int8_swiglu(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor,
                                 b_scales: torch.Tensor, out: torch.Tensor,
                                 counts: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_grouped_gemm_int8() with MOE_EPILOGUE_SWIGLU: b [G, 2 I, K] holds each
    expert's I gate rows, then its I up rows; out [G, cap, I] (bf16 or fp16)
    gets silu(gate) * up, which moe_quantize_int8 makes the next product's rows
    of."""
    _product(a, a_scales, b, b_scales, out, counts, stream, MOE_EPILOGUE_SWIGLU)


def moe_few_tokens_workspace_bytes(tokens: int, topk: int, hidden: int, inter: int) -> int:
    """Bytes of workspace that moe_few_tokens needs."""
    return _workspace_bytes("moe_few_tokens_workspace_bytes", tokens, topk, hidden, inter)


def moe_few_tokens(x: torch.Tensor, indices: torch.Tensor, weights: Optional[torch.Tensor],
                   gate_up: torch.Tensor, gate_up_scales: torch.Tensor, down: torch.Tensor,
                   down_scales: torch.Tensor, out: torch.Tensor,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_few_tokens() (include/moe_block.h): the experts of a whole layer for up
    to 64 tokens, without a dispatch. x [..., H] (bf16 or fp16) and out of its
    shape and type; indices and weights (or None: 1 each) [..., k] of the same
    leading sizes; gate_up [E, 2 I, H] and down [E, H, I] as expert_mlp's (E4M3,
    scales [E, 2 I / 128, H / 128] and [E, H / 128, I / 128]) or expert_mlp_int8's
    (int8, scales [E, 2 I] and [E, H]). workspace: any tensor of
    moe_few_tokens_workspace_bytes bytes that no other call uses at the same
    time; None makes a new one."""
    index, shape, H, tokens, dtype = _rows_of(x, "x")
    for t, name in ((indices, "indices"), (gate_up, "gate_up"), (down, "down"),
                    (gate_up_scales, "gate_up_scales"), (down_scales, "down_scales"),
                    (out, "out")):
        _index_of(t, name)
    for t, name in ((gate_up, "gate_up"), (down, "down")):
        if t.dim() != 3:
            raise ValueError(f"{name} must have 3 dimensions, not {t.dim()}")
    if indices.dim() == 0:
        raise ValueError("indices must have slots")
    topk = indices.shape[-1]
    E, inter = down.shape[0], down.shape[2]
    int8 = gate_up.dtype == torch.int8
    codes = _INT8 if int8 else _CODES
    scales = (((E, 2 * inter), (E, H)) if int8 else
              ((E, 2 * inter // 128, H // 128), (E, H // 128, inter // 128)))
    slots = shape[:-1] + (topk,)
    ws, nbytes = None, 0
    if tokens:
        nbytes = moe_few_tokens_workspace_bytes(tokens, topk, H, inter)
        ws = _workspace(workspace, nbytes, index, stream)
    a = MoeFewTokensArgs(
        _ptr(x, "x", shape, (x.dtype,), index), _ptr(indices, "indices", slots, _I32, index),
        _ptr(weights, "weights", slots, _F32, index),
        _ptr(gate_up, "gate_up", (E, 2 * inter, H), codes, index),
        _ptr(gate_up_scales, "gate_up_scales", scales[0], _F32, index),
        _ptr(down, "down", (E, H, inter), codes, index),
        _ptr(down_scales, "down_scales", scales[1], _F32, index),
        _ptr(out, "out", shape, (x.dtype,), index), None if ws is None else ws.data_ptr(), nbytes,
        tokens, topk, E, H, inter, dtype, MOE_INT8 if int8 else EP_FP8_E4M3)
    _call("moe_few_tokens", index, stream, a)
