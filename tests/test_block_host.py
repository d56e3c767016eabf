"""Host-side checks of include/moe_block.h (no GPU needed, no kernel is
launched): every function is exported, and every bad argument is refused with
its code and a message that names it, before anything is enqueued. Pointers
are fake addresses that are never dereferenced."""
import ctypes
import math
import os
import re

import pytest
import torch

import combine_route_amd as cra
from combine_route_amd import block, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F1000000000             # 16-byte aligned device-looking address


@pytest.fixture(scope="module")
def fn():
    if not os.path.exists(cra.LIB_PATH):
        import combine_route_amd.build as b
        b.build()
    return block._fn


def test_exports_every_declared_function(fn):
    with open(os.path.join(ROOT, "include", "moe_block.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = re.findall(r"\b(?:int|size_t) (moe_\w+)\s*\(", text)
    assert sorted(names) == sorted(block.BLOCK_EXPORTED)
    for n in names:
        assert fn(n) is not None and hasattr(cra, n.replace("_ex", ""))


NORM = dict(y=FAKE, residual=FAKE, residual_out=FAKE, post_weight=FAKE, gate=FAKE,
            pre_weight=FAKE, out=FAKE, codes=FAKE, scales=FAKE, row_counts=FAKE, rows=64,
            group_rows=16, gate_rows=16, hidden=256, dtype=cra.EP_BF16, weight_dtype=cra.EP_BF16,
            codes_dtype=cra.EP_FP8_E4M3, residual_scale=1.0, eps=1e-6)

COMMON = [
    (dict(y=None), cra.EP_ERR_NULL, "args.y"),
    (dict(y=FAKE + 8), cra.EP_ERR_ALIGN, "args.y"),
    (dict(post_weight=FAKE + 4), cra.EP_ERR_ALIGN, "post_weight"),
    (dict(gate=FAKE + 4), cra.EP_ERR_ALIGN, "gate"),
    (dict(pre_weight=FAKE + 4), cra.EP_ERR_ALIGN, "pre_weight"),
    (dict(row_counts=FAKE + 2), cra.EP_ERR_ALIGN, "row_counts"),
    (dict(rows=-1), cra.EP_ERR_ARG, "rows"),
    (dict(group_rows=0), cra.EP_ERR_ARG, "group_rows"),
    (dict(group_rows=7), cra.EP_ERR_ARG, "group_rows"),
    (dict(gate_rows=-1), cra.EP_ERR_ARG, "gate_rows"),
    (dict(gate_rows=48), cra.EP_ERR_ARG, "gate_rows"),
    (dict(hidden=0), cra.EP_ERR_ARG, "hidden"),
    (dict(hidden=12), cra.EP_ERR_ARG, "hidden"),
    (dict(hidden=32768 + 128), cra.EP_ERR_SIZE, "hidden"),
    (dict(dtype=cra.EP_FP8_E4M3), cra.EP_ERR_ARG, "dtype"),
    (dict(weight_dtype=cra.EP_FP16), cra.EP_ERR_ARG, "weight_dtype"),
    (dict(eps=-1.0), cra.EP_ERR_ARG, "eps"),
    (dict(eps=math.nan), cra.EP_ERR_ARG, "eps"),
    (dict(eps=math.inf), cra.EP_ERR_ARG, "eps"),
    (dict(residual_scale=math.nan), cra.EP_ERR_ARG, "residual_scale"),
    (dict(residual_scale=math.inf), cra.EP_ERR_ARG, "residual_scale"),
]


@pytest.mark.parametrize("change,code,word", COMMON + [
    (dict(residual=None), cra.EP_ERR_NULL, "residual"),
    (dict(residual_out=None), cra.EP_ERR_NULL, "residual_out"),
    (dict(pre_weight=None), cra.EP_ERR_ARG, "pre_weight"),
    (dict(out=None, codes=None, scales=None), cra.EP_ERR_ARG, "pre_weight"),
    (dict(codes=None), cra.EP_ERR_ARG, "scales"),
    (dict(scales=None), cra.EP_ERR_ARG, "codes"),
    (dict(codes_dtype=cra.EP_BF16), cra.EP_ERR_ARG, "codes_dtype"),
    (dict(hidden=136), cra.EP_ERR_ARG, "multiple of 128"),
    (dict(residual=FAKE + 2), cra.EP_ERR_ALIGN, "residual"),
    (dict(residual_out=FAKE + 2), cra.EP_ERR_ALIGN, "residual_out"),
    (dict(out=FAKE + 8), cra.EP_ERR_ALIGN, "out"),
    (dict(codes=FAKE + 8), cra.EP_ERR_ALIGN, "codes"),
    (dict(scales=FAKE + 2), cra.EP_ERR_ALIGN, "scales"),
    (dict(rows=1 << 27, group_rows=1 << 20), cra.EP_ERR_SIZE, "rows"),
])
def test_block_norm_refuses(fn, change, code, word):
    a = block.MoeBlockNormArgs(**dict(NORM, **change))
    assert fn("moe_block_norm")(ctypes.byref(a), None) == code
    assert word in cra.ep_last_error()


BACKWARD = {k: v for k, v in NORM.items() if k not in (
    "residual", "residual_out", "out", "codes", "scales", "codes_dtype")}
BACKWARD.update(h=FAKE, grad_h=FAKE, grad_out=FAKE, grad_y=FAKE, grad_residual=FAKE,
                grad_post_weight=FAKE, grad_gate=FAKE, grad_pre_weight=FAKE, workspace=FAKE,
                workspace_bytes=1 << 40)


@pytest.mark.parametrize("change,code,word", COMMON + [
    (dict(h=None), cra.EP_ERR_NULL, "args.h"),
    (dict(grad_y=None), cra.EP_ERR_NULL, "grad_y"),
    (dict(workspace=None), cra.EP_ERR_NULL, "workspace"),
    (dict(grad_out=None), cra.EP_ERR_ARG, "grad_out"),
    (dict(pre_weight=None), cra.EP_ERR_ARG, "pre_weight"),
    (dict(grad_h=None, grad_out=None, pre_weight=None, grad_pre_weight=None), cra.EP_ERR_NULL,
     "grad_h"),
    (dict(post_weight=None), cra.EP_ERR_ARG, "grad_post_weight"),
    (dict(gate=None), cra.EP_ERR_ARG, "grad_gate"),
    (dict(grad_out=None, pre_weight=None), cra.EP_ERR_ARG, "grad_pre_weight"),
    (dict(gate_rows=8), cra.EP_ERR_ARG, "gate_rows"),
    (dict(workspace_bytes=4 * 16 * 256 * 12 - 1), cra.EP_ERR_SIZE, "workspace_bytes"),
] + [(dict({n: FAKE + 8}), cra.EP_ERR_ALIGN, n) for n in (
    "h", "grad_h", "grad_out", "grad_y", "grad_residual", "grad_post_weight", "grad_gate",
    "grad_pre_weight", "workspace")])
def test_block_norm_backward_refuses(fn, change, code, word):
    a = block.MoeBlockNormBackwardArgs(**dict(BACKWARD, **change))
    assert fn("moe_block_norm_backward")(ctypes.byref(a), None) == code
    assert word in cra.ep_last_error()


QUANT = dict(rows=FAKE, codes=FAKE, scales=FAKE, row_counts=FAKE, n_rows=64, group_rows=16,
             hidden=256, dtype=cra.EP_BF16)


@pytest.mark.parametrize("change,code,word", [
    (dict(rows=None), cra.EP_ERR_NULL, "rows"),
    (dict(codes=None), cra.EP_ERR_NULL, "codes"),
    (dict(scales=None), cra.EP_ERR_NULL, "scales"),
    (dict(rows=FAKE + 8), cra.EP_ERR_ALIGN, "rows"),
    (dict(codes=FAKE + 8), cra.EP_ERR_ALIGN, "codes"),
    (dict(scales=FAKE + 2), cra.EP_ERR_ALIGN, "scales"),
    (dict(row_counts=FAKE + 1), cra.EP_ERR_ALIGN, "row_counts"),
    (dict(n_rows=-1), cra.EP_ERR_ARG, "n_rows"),
    (dict(group_rows=0), cra.EP_ERR_ARG, "group_rows"),
    (dict(group_rows=7), cra.EP_ERR_ARG, "group_rows"),
    (dict(hidden=0), cra.EP_ERR_ARG, "hidden"),
    (dict(hidden=12), cra.EP_ERR_ARG, "hidden"),
    (dict(hidden=65536 + 8), cra.EP_ERR_SIZE, "hidden"),
    (dict(dtype=block.MOE_INT8), cra.EP_ERR_ARG, "dtype"),
    (dict(n_rows=1 << 27, group_rows=1 << 20), cra.EP_ERR_SIZE, "n_rows"),
])
def test_quantize_int8_refuses(fn, change, code, word):
    a = block.MoeQuantizeInt8Args(**dict(QUANT, **change))
    assert fn("moe_quantize_int8")(ctypes.byref(a), None) == code
    assert word in cra.ep_last_error()


GEMM = dict(a=FAKE, a_scales=FAKE, b=FAKE, b_scales=FAKE, counts=FAKE, out=FAKE, groups=4, cap=16,
            n=256, k=128, out_dtype=cra.EP_BF16, epilogue=cra.MOE_EPILOGUE_ROWS)


@pytest.mark.parametrize("change,code,word", [
    (dict(epilogue=2), cra.EP_ERR_ARG, "epilogue"),
    (dict(out_dtype=cra.EP_FP8_E4M3), cra.EP_ERR_ARG, "out_dtype"),
    (dict(out_dtype=block.MOE_INT8, epilogue=cra.MOE_EPILOGUE_SWIGLU), cra.EP_ERR_ARG,
     "out_dtype"),
    (dict(groups=-1), cra.EP_ERR_ARG, "groups"),
    (dict(cap=-1), cra.EP_ERR_ARG, "cap"),
    (dict(k=0), cra.EP_ERR_ARG, "args.k"),
    (dict(k=24), cra.EP_ERR_ARG, "args.k"),
    (dict(k=65536 + 16), cra.EP_ERR_SIZE, "args.k"),
    (dict(n=0), cra.EP_ERR_ARG, "args.n"),
    (dict(n=12), cra.EP_ERR_ARG, "args.n"),
    (dict(n=24, epilogue=cra.MOE_EPILOGUE_SWIGLU), cra.EP_ERR_ARG, "args.n"),
    (dict(n=(1 << 20) + 16), cra.EP_ERR_SIZE, "args.n"),
    (dict(groups=(1 << 20) + 1), cra.EP_ERR_SIZE, "groups"),
    (dict(groups=1 << 20, cap=1 << 11), cra.EP_ERR_SIZE, "cap"),
] + [(dict({p: None}), cra.EP_ERR_NULL, p) for p in ("a", "a_scales", "b", "b_scales", "out")] +
    [(dict({p: FAKE + 8}), cra.EP_ERR_ALIGN, p) for p in ("a", "b", "out")] +
    [(dict({p: FAKE + 2}), cra.EP_ERR_ALIGN, p) for p in ("a_scales", "b_scales", "counts")])
def test_grouped_gemm_int8_refuses(fn, change, code, word):
    a = block.MoeGroupedGemmInt8Args(**dict(GEMM, **change))
    assert fn("moe_grouped_gemm_int8")(ctypes.byref(a), None) == code
    assert word in cra.ep_last_error()


FEW = dict(x=FAKE, indices=FAKE, weights=FAKE, gate_up=FAKE, gate_up_scales=FAKE, down=FAKE,
           down_scales=FAKE, out=FAKE, workspace=FAKE, workspace_bytes=1 << 40, tokens=4, topk=2,
           experts=8, hidden=256, inter=128, dtype=cra.EP_BF16, weight_dtype=cra.EP_FP8_E4M3)


@pytest.mark.parametrize("change,code,word", [
    (dict(dtype=cra.EP_FP8_E4M3), cra.EP_ERR_ARG, "args.dtype"),
    (dict(weight_dtype=cra.EP_BF16), cra.EP_ERR_ARG, "weight_dtype"),
    (dict(hidden=0), cra.EP_ERR_ARG, "hidden"),
    (dict(hidden=192), cra.EP_ERR_ARG, "hidden"),
    (dict(hidden=200, weight_dtype=block.MOE_INT8), cra.EP_ERR_ARG, "hidden"),
    (dict(inter=64), cra.EP_ERR_ARG, "inter"),
    (dict(inter=8, weight_dtype=block.MOE_INT8), cra.EP_ERR_ARG, "inter"),
    (dict(tokens=-1), cra.EP_ERR_ARG, "tokens"),
    (dict(topk=0), cra.EP_ERR_ARG, "topk"),
    (dict(experts=0), cra.EP_ERR_ARG, "experts"),
    (dict(tokens=65), cra.EP_ERR_SIZE, "tokens"),
    (dict(topk=65), cra.EP_ERR_SIZE, "topk"),
    (dict(tokens=64, topk=17), cra.EP_ERR_SIZE, "slots"),
    (dict(experts=65537), cra.EP_ERR_SIZE, "experts"),
    (dict(hidden=65536 + 128), cra.EP_ERR_SIZE, "hidden"),
    (dict(inter=65536 + 128), cra.EP_ERR_SIZE, "inter"),
    (dict(workspace_bytes=4 * 4 * 2 * 128 - 1), cra.EP_ERR_SIZE, "workspace_bytes"),
] + [(dict({p: None}), cra.EP_ERR_NULL, p) for p in (
    "x", "indices", "gate_up", "gate_up_scales", "down", "down_scales", "out", "workspace")] +
    [(dict({p: FAKE + 8}), cra.EP_ERR_ALIGN, p) for p in ("x", "gate_up", "down", "out",
                                                         "workspace")] +
    [(dict({p: FAKE + 2}), cra.EP_ERR_ALIGN, p) for p in ("indices", "weights", "gate_up_scales",
                                                         "down_scales")])
def test_few_tokens_refuses(fn, change, code, word):
    a = block.MoeFewTokensArgs(**dict(FEW, **change))
    assert fn("moe_few_tokens")(ctypes.byref(a), None) == code
    assert word in cra.ep_last_error()


def test_few_tokens_workspace_bytes(fn):
    size = cra.moe_few_tokens_workspace_bytes
    assert size(4, 2, 256, 128) == 4 * 8 * 128
    assert size(64, 16, 16, 65536) == 4 * 1024 * 65536
    for bad in ((0, 2, 256, 128), (65, 2, 256, 128), (64, 17, 256, 128), (4, 65, 256, 128),
                (4, 2, 24, 128), (4, 2, 256, 8), (4, 2, 256, 65552)):
        with pytest.raises(cra.EpError):
            size(*bad)


def test_calls_without_rows_are_no_work(fn):
    a = block.MoeBlockNormArgs(**dict(NORM, rows=0, y=None, residual=None))
    assert fn("moe_block_norm")(ctypes.byref(a), None) == cra.EP_OK
    a = block.MoeBlockNormBackwardArgs(**dict(BACKWARD, rows=0, y=None, workspace=None))
    assert fn("moe_block_norm_backward")(ctypes.byref(a), None) == cra.EP_OK
    a = block.MoeQuantizeInt8Args(**dict(QUANT, n_rows=0, rows=None))
    assert fn("moe_quantize_int8")(ctypes.byref(a), None) == cra.EP_OK
    for change in (dict(groups=0, a=None), dict(cap=0, out=None)):
        a = block.MoeGroupedGemmInt8Args(**dict(GEMM, **change))
        assert fn("moe_grouped_gemm_int8")(ctypes.byref(a), None) == cra.EP_OK
    a = block.MoeFewTokensArgs(**dict(FEW, tokens=0, x=None, workspace=None))
    assert fn("moe_few_tokens")(ctypes.byref(a), None) == cra.EP_OK
    assert cra.ep_last_error() == ""
    for name in block.BLOCK_EXPORTED:
        if name.endswith("_bytes"):
            continue
        assert fn(name)(None, None) == cra.EP_ERR_NULL


def test_norms_without_rows_take_any_pointers(fn):
    """Empty tensors have no address: which of them are given cannot be told."""
    a = block.MoeBlockNormArgs(**dict(NORM, rows=0, y=None, residual=None, residual_out=None,
                                      out=None, codes=None, scales=None))
    assert fn("moe_block_norm")(ctypes.byref(a), None) == cra.EP_OK
    a = block.MoeBlockNormArgs(**dict(NORM, rows=0, codes=None))
    assert fn("moe_block_norm")(ctypes.byref(a), None) == cra.EP_OK
    a = block.MoeBlockNormBackwardArgs(**dict(BACKWARD, rows=0, y=None, h=None, grad_h=None,
                                              grad_out=None, grad_y=None, grad_residual=None))
    assert fn("moe_block_norm_backward")(ctypes.byref(a), None) == cra.EP_OK
    # sizes are still checked
    a = block.MoeBlockNormArgs(**dict(NORM, rows=0, out=None, hidden=12))
    assert fn("moe_block_norm")(ctypes.byref(a), None) == cra.EP_ERR_ARG


def test_backward_workspace_bytes(fn):
    size = cra.moe_block_norm_backward_workspace_bytes
    assert size(64, 256, 4) == 64 * 256 * 12
    assert size(1, 8) == 8 * 12
    # never more parts than rows, whole parts for each group
    for rows, hidden, groups in ((16384, 7168, 8), (3000, 264, 3000), (5000, 32768, 1)):
        n = size(rows, hidden, groups)
        assert n % (12 * hidden) == 0 and n // (12 * hidden) <= rows
    for bad in ((0, 256, 1), (4, 12, 1), (4, 40000, 1), (4, 256, 3), (4, 256, 0)):
        with pytest.raises(cra.EpError):
            size(*bad)


@pytest.mark.parametrize("hidden", [256, 1032, 4096, 7168, 16392])
@pytest.mark.parametrize("rows", [1, 48, 768, 840, 1680, 15120])
def test_a_backward_workspace_is_enough_for_any_groups(fn, hidden, rows):
    """The size for some groups serves calls with others: those without counts
    have one group, whatever their tensors' leading size."""
    size = cra.moe_block_norm_backward_workspace_bytes
    groups = [g for g in (1, 2, 3, 4, 5, 6, 7, 8, 24, 48, 105, 280, 840, 1680, 15120)
              if rows % g == 0]
    for g in groups:
        a = block.MoeBlockNormBackwardArgs(**dict(
            BACKWARD, rows=rows, hidden=hidden, row_counts=FAKE if g > 1 else None,
            group_rows=rows // g, gate_rows=0, workspace_bytes=0))
        assert fn("moe_block_norm_backward")(ctypes.byref(a), None) == cra.EP_ERR_SIZE
        need = int(re.search(r"(\d+) are needed", cra.ep_last_error())[1])
        assert need > 0
        assert all(size(rows, hidden, other) >= need for other in groups)


def test_tensors_off_the_gpu_are_refused():
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        cra.moe_block_norm(x, x, w, 1e-6, out=x)
    with pytest.raises(TypeError, match="y must"):
        cra.moe_block_norm([1.0], x, w, 1e-6)
    with pytest.raises(ValueError, match="GPU"):
        cra.moe_block_norm_backward(x, x, 1e-6, x, grad_out=x, pre_weight=w)
    with pytest.raises(ValueError, match="GPU"):
        cra.moe_quantize_int8(x, x, w)
    for call in (cra.moe_grouped_gemm_int8, cra.moe_grouped_gemm_int8_swiglu):
        with pytest.raises(ValueError, match="GPU"):
            call(x, w, x, w, x)
        with pytest.raises(TypeError, match="a must"):
            call([1], w, x, w, x)
    with pytest.raises(ValueError, match="GPU"):
        cra.moe_few_tokens(x, x, None, x, w, x, w, x)


def test_the_other_headers_are_as_they_were():
    """moe.h's functions keep their own binding."""
    assert not set(block.BLOCK_EXPORTED) & set(moe.MOE_EXPORTED)
