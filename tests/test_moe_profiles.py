"""The committed profile of the layer operators is of the committed kernels: it
records the sha256 prefix of their sources' code, comments aside."""
import glob
import hashlib
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROFILE = os.path.join(ROOT, "profiles", "kernel_stats_moe_layer_operators.md")


def code_hash():
    h = hashlib.sha256()
    for path in sorted(glob.glob(os.path.join(ROOT, "combine_route_amd", "csrc", "moe_*"))):
        with open(path) as f:
            h.update(" ".join(re.sub(r"//[^\n]*", "", f.read()).split()).encode())
    return h.hexdigest()[:16]


def test_the_profile_is_of_the_current_kernels():
    with open(PROFILE) as f:
        text = f.read()
    assert re.findall(r"moe sources' code sha256\[:16\]: (\w+)", text) == [code_hash()]
    for kernel in ("moe_norm_kernel", "moe_gemm_kernel", "moe_combine_backward_kernel",
                   "moe_dispatch_backward_kernel"):
        assert kernel in text
