"""The committed profile of the operators of a whole layer is of the committed
kernels: it records the sha256 prefix of their sources' code, comments aside."""
import glob
import hashlib
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROFILE = os.path.join(ROOT, "profiles", "kernel_stats_moe_block_operators.md")


def code_hash():
    h = hashlib.sha256()
    for path in sorted(glob.glob(os.path.join(ROOT, "combine_route_amd", "csrc", "block_*"))):
        with open(path) as f:
            h.update(" ".join(re.sub(r"//[^\n]*", "", f.read()).split()).encode())
    return h.hexdigest()[:16]


def test_the_profile_is_of_the_current_kernels():
    with open(PROFILE) as f:
        text = f.read()
    assert re.findall(r"block sources' code sha256\[:16\]: (\w+)", text) == [code_hash()]
    for kernel in ("block_norm_kernel", "block_norm_backward_kernel", "block_norm_reduce_kernel",
                   "block_quantize_kernel", "block_gemm_kernel", "block_few_up_kernel",
                   "block_few_down_kernel"):
        assert kernel in text
