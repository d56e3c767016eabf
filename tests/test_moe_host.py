"""Host-side checks of include/moe.h (no GPU needed, no kernel is launched):
every function is exported, and every bad argument is refused with its code
and a message that names it, before anything is enqueued. Pointers are fake
addresses that are never dereferenced."""
import ctypes
import math
import os
import re

import pytest

import combine_route_amd as cra
from combine_route_amd import moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F1000000000             # 16-byte aligned device-looking address


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(cra.LIB_PATH):
        import combine_route_amd.build as b
        b.build()
    return moe._lib()


def test_exports_every_declared_function(lib):
    with open(os.path.join(ROOT, "include", "moe.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z_]+)\s*\(", text))
    assert sorted(names) == sorted(moe.MOE_EXPORTED)
    for n in names:
        assert hasattr(lib, n), n


def norm_args(**kw):
    a = dict(x=FAKE, residual=FAKE, residual_out=FAKE, weight=FAKE, out=FAKE, codes=FAKE,
             scales=FAKE, row_counts=FAKE, rows=64, group_rows=16, hidden=256, dtype=cra.EP_BF16,
             weight_dtype=cra.EP_BF16, eps=1e-6)
    a.update(kw)
    return moe.MoeRmsNormArgs(**a)


BAD_NORM = [
    (dict(x=None), cra.EP_ERR_NULL, "x"),
    (dict(weight=None), cra.EP_ERR_NULL, "weight"),
    (dict(out=None, codes=None, scales=None), cra.EP_ERR_NULL, "out"),
    (dict(codes=None), cra.EP_ERR_ARG, "scales"),
    (dict(scales=None), cra.EP_ERR_ARG, "codes"),
    (dict(residual=None), cra.EP_ERR_ARG, "residual"),
    (dict(residual_out=None), cra.EP_ERR_ARG, "residual_out"),
    (dict(x=FAKE + 8), cra.EP_ERR_ALIGN, "x"),
    (dict(residual=FAKE + 2), cra.EP_ERR_ALIGN, "residual"),
    (dict(residual_out=FAKE + 2), cra.EP_ERR_ALIGN, "residual_out"),
    (dict(weight=FAKE + 4), cra.EP_ERR_ALIGN, "weight"),
    (dict(out=FAKE + 8), cra.EP_ERR_ALIGN, "out"),
    (dict(codes=FAKE + 8), cra.EP_ERR_ALIGN, "codes"),
    (dict(scales=FAKE + 2), cra.EP_ERR_ALIGN, "scales"),
    (dict(row_counts=FAKE + 2), cra.EP_ERR_ALIGN, "row_counts"),
    (dict(rows=-1), cra.EP_ERR_ARG, "rows"),
    (dict(group_rows=0), cra.EP_ERR_ARG, "group_rows"),
    (dict(group_rows=7), cra.EP_ERR_ARG, "group_rows"),
    (dict(hidden=0), cra.EP_ERR_ARG, "hidden"),
    (dict(hidden=-8), cra.EP_ERR_ARG, "hidden"),
    (dict(hidden=12), cra.EP_ERR_ARG, "hidden"),
    (dict(hidden=136), cra.EP_ERR_ARG, "multiple of 128"),
    (dict(hidden=65536 + 128), cra.EP_ERR_SIZE, "hidden"),
    (dict(dtype=cra.EP_FP8_E4M3), cra.EP_ERR_ARG, "dtype"),
    (dict(weight_dtype=cra.EP_FP16), cra.EP_ERR_ARG, "weight_dtype"),
    (dict(eps=-1.0), cra.EP_ERR_ARG, "eps"),
    (dict(eps=math.nan), cra.EP_ERR_ARG, "eps"),
    (dict(eps=math.inf), cra.EP_ERR_ARG, "eps"),
    (dict(rows=1 << 27, group_rows=1 << 20), cra.EP_ERR_SIZE, "rows"),
]


@pytest.mark.parametrize("change,code,word", BAD_NORM)
def test_rms_norm_refuses(lib, change, code, word):
    assert lib.moe_rms_norm(ctypes.byref(norm_args(**change)), None) == code
    assert word in cra.ep_last_error()


def test_rms_norm_without_rows_is_no_work(lib):
    assert lib.moe_rms_norm(None, None) == cra.EP_ERR_NULL
    assert lib.moe_rms_norm(ctypes.byref(norm_args(rows=0, x=None, out=None)), None) == cra.EP_OK
    assert cra.ep_last_error() == ""


def test_tensors_off_the_gpu_are_refused():
    import torch
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        cra.moe_rms_norm(x, torch.ones(128, dtype=torch.bfloat16), 1e-6, out=x)
    with pytest.raises(TypeError, match="x must"):
        cra.moe_rms_norm([1.0], x, 1e-6)
    with pytest.raises(TypeError, match="weight"):
        moe._refuse([1.0], "weight", (1,), (torch.float32,), 0)
    with pytest.raises(ValueError, match="GPU"):
        cra.moe_grouped_gemm(x, x, x, x, x)
    cfg = cra.make_config(2, 128, 4, 2, 2)
    with pytest.raises(ValueError, match="GPU"):
        cra.moe_dispatch_backward(0, cfg, 4, x, x)
    with pytest.raises(ValueError, match="GPU"):
        cra.moe_combine_backward(0, cfg, 4, x, x, None, None, x, None)


def test_backward_calls_refuse(lib):
    cb, db = moe.MoeCombineBackwardArgs(*[FAKE] * 6), moe.MoeDispatchBackwardArgs(FAKE, FAKE)
    assert lib.moe_combine_backward(None, ctypes.byref(cb), None) == cra.EP_ERR_NULL
    assert lib.moe_dispatch_backward(None, ctypes.byref(db), None) == cra.EP_ERR_NULL
    cfg = cra.make_config(2, 256, 16, 4, 2)
    plan, eplan = ctypes.c_void_p(), ctypes.c_void_p()
    assert lib.ep_plan_create(ctypes.byref(cfg), FAKE, 1 << 40, ctypes.byref(plan)) == 0
    assert lib.ep_expert_plan_create(plan, 8, FAKE, 1 << 40, ctypes.byref(eplan)) == 0

    def combine(code, word, **change):
        a = dict(zip([n for n, _ in moe.MoeCombineBackwardArgs._fields_], [FAKE] * 6))
        a.update(change)
        args = moe.MoeCombineBackwardArgs(**a)
        assert lib.moe_combine_backward(eplan, ctypes.byref(args), None) == code
        assert word in cra.ep_last_error()

    assert lib.moe_combine_backward(eplan, None, None) == cra.EP_ERR_NULL
    for name in ("grad_out", "indices", "grad_packed_y"):
        combine(cra.EP_ERR_NULL, name, **{name: None})
    for name in ("grad_out", "packed_y", "grad_packed_y"):
        combine(cra.EP_ERR_ALIGN, name, **{name: FAKE + 8})
    for name in ("indices", "weights", "grad_weights"):
        combine(cra.EP_ERR_ALIGN, name, **{name: FAKE + 2})
    combine(cra.EP_ERR_ARG, "packed_y", packed_y=None)
    combine(cra.EP_ERR_ARG, "packed_y", grad_weights=None)
    combine(cra.EP_ERR_ARG, "args.weights", weights=None)
    combine(cra.EP_ERR_STATE, "before any")
    assert lib.moe_dispatch_backward(eplan, None, None) == cra.EP_ERR_NULL
    for i, name in enumerate(("grad_packed_x", "grad_x")):
        for value, code in ((None, cra.EP_ERR_NULL), (FAKE + 8, cra.EP_ERR_ALIGN)):
            p = [FAKE, FAKE]
            p[i] = value
            args = moe.MoeDispatchBackwardArgs(*p)
            assert lib.moe_dispatch_backward(eplan, ctypes.byref(args), None) == code
            assert name in cra.ep_last_error()
    assert lib.moe_dispatch_backward(eplan, ctypes.byref(db), None) == cra.EP_ERR_STATE
    assert lib.ep_expert_plan_destroy(eplan) == 0
    assert lib.ep_plan_destroy(plan) == 0


def gemm_args(**kw):
    a = dict(a=FAKE, a_scales=FAKE, b=FAKE, b_scales=FAKE, counts=FAKE, out=FAKE, out_scales=None,
             groups=4, cap=64, n=256, k=256, out_dtype=cra.EP_BF16,
             epilogue=cra.MOE_EPILOGUE_ROWS)
    a.update(kw)
    return moe.MoeGroupedGemmArgs(**a)


SWIGLU = dict(epilogue=cra.MOE_EPILOGUE_SWIGLU, out_dtype=cra.EP_FP8_E4M3, out_scales=FAKE)
BAD_GEMM = [
    (dict(a=None), cra.EP_ERR_NULL, "args.a "),
    (dict(a_scales=None), cra.EP_ERR_NULL, "a_scales"),
    (dict(b=None), cra.EP_ERR_NULL, "args.b "),
    (dict(b_scales=None), cra.EP_ERR_NULL, "b_scales"),
    (dict(out=None), cra.EP_ERR_NULL, "out"),
    (dict(SWIGLU, out_scales=None), cra.EP_ERR_NULL, "out_scales"),
    (dict(out_scales=FAKE), cra.EP_ERR_ARG, "out_scales"),
    (dict(a=FAKE + 8), cra.EP_ERR_ALIGN, "args.a "),
    (dict(b=FAKE + 4), cra.EP_ERR_ALIGN, "args.b "),
    (dict(out=FAKE + 8), cra.EP_ERR_ALIGN, "out"),
    (dict(a_scales=FAKE + 2), cra.EP_ERR_ALIGN, "a_scales"),
    (dict(b_scales=FAKE + 2), cra.EP_ERR_ALIGN, "b_scales"),
    (dict(counts=FAKE + 2), cra.EP_ERR_ALIGN, "counts"),
    (dict(SWIGLU, out_scales=FAKE + 2), cra.EP_ERR_ALIGN, "out_scales"),
    (dict(groups=-1), cra.EP_ERR_ARG, "groups"),
    (dict(cap=-1), cra.EP_ERR_ARG, "cap"),
    (dict(k=0), cra.EP_ERR_ARG, "args.k"),
    (dict(k=192), cra.EP_ERR_ARG, "args.k"),
    (dict(n=0), cra.EP_ERR_ARG, "args.n"),
    (dict(n=12), cra.EP_ERR_ARG, "args.n"),
    (dict(SWIGLU, n=128), cra.EP_ERR_ARG, "256"),
    (dict(n=(1 << 20) + 8), cra.EP_ERR_SIZE, "args.n"),
    (dict(k=(1 << 20) + 128), cra.EP_ERR_SIZE, "args.k"),
    (dict(groups=1 << 16, cap=1 << 16), cra.EP_ERR_SIZE, "groups"),
    (dict(groups=(1 << 20) + 1, cap=1), cra.EP_ERR_SIZE, "groups"),
    (dict(out_dtype=cra.EP_FP8_E4M3), cra.EP_ERR_ARG, "out_dtype"),
    (dict(SWIGLU, out_dtype=cra.EP_BF16), cra.EP_ERR_ARG, "out_dtype"),
    (dict(epilogue=2), cra.EP_ERR_ARG, "epilogue"),
]


@pytest.mark.parametrize("change,code,word", BAD_GEMM)
def test_grouped_gemm_refuses(lib, change, code, word):
    assert lib.moe_grouped_gemm(ctypes.byref(gemm_args(**change)), None) == code
    assert word in cra.ep_last_error()


def test_grouped_gemm_without_rows_is_no_work(lib):
    assert lib.moe_grouped_gemm(None, None) == cra.EP_ERR_NULL
    for change in (dict(groups=0), dict(cap=0)):
        args = gemm_args(a=None, out=None, **change)
        assert lib.moe_grouped_gemm(ctypes.byref(args), None) == cra.EP_OK


def test_backward_of_another_devices_tensors_is_refused():
    import torch
    from types import SimpleNamespace as Fields
    op = Fields(_ex={"plan": 0}, workspace=Fields(device=torch.device("cuda:0")))
    state = cra.EpDispatchCombineOp._fused_state
    assert state(op, "call", Fields(device=torch.device("cuda:0")), "grad_out") is op._ex
    with pytest.raises(ValueError, match="grad_out is on cuda:1, the op on cuda:0"):
        state(op, "call", Fields(device=torch.device("cuda:1")), "grad_out")
    assert state(op, "call", [1.0], "grad_out") is op._ex
    op._ex = None
    with pytest.raises(cra.EpError, match="before any dispatch_standard_moe"):
        state(op, "call", Fields(device=torch.device("cuda:0")), "grad_out")
