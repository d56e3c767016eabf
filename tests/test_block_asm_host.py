"""As test_moe_asm_host.py, of the inline assembly of the kernels of a whole MoE
block: every statement names the registers it changes."""
import glob
import os

import pytest

import test_moe_asm_host as moe_asm

FILES = sorted(glob.glob(os.path.join(moe_asm.CSRC, "block_*")))


def test_there_are_such_statements():
    found = [s for f in FILES for s in moe_asm.statements(f)]
    assert any("m0" in " ".join(lines) for lines, _ in found)


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_statements_name_what_they_change(path):
    moe_asm.test_statements_name_what_they_change(path)
