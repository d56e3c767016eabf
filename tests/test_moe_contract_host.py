"""The contract of moe_grouped_gemm, as the header and the binding state it: which
form sums in FP32 throughout, and what the other's first step cuts."""
import os
import re

import combine_route_amd as cra

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def header_comment():
    with open(os.path.join(ROOT, "include", "moe.h")) as f:
        text = f.read()
    end = text.index("typedef struct moe_grouped_gemm_args")
    return re.sub(r"\s*\n \* *", " ", text[text.rindex("/* Grouped product", 0, end):end])


def test_the_header_states_each_forms_sums():
    text = header_comment()
    assert "with every sum in FP32" not in text
    assert "MOE_EPILOGUE_SWIGLU takes every sum in FP32" in text
    rows = text[text.index("MOE_EPILOGUE_ROWS rounds y once"):]
    assert "toward zero to a multiple of 2^(E - 13)" in rows
    assert "less than a_scales * b_scales * 7 * 2^(E - 13)" in rows


def test_the_binding_states_them_too():
    assert "2^(E - 13)" in cra.moe_grouped_gemm.__doc__
    assert "Every sum is in" in cra.moe_grouped_gemm_swiglu.__doc__
