"""The inline assembly of the layer operators' kernels tells the compiler every
register it changes: a statement that writes M0 names it as overwritten, and one
that changes the lanes' mask puts back the mask it found."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "combine_route_amd", "csrc")


def statements(path):
    """(template text, everything after it) of each asm statement."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"asm\s+volatile\s*\(", text):
        depth, i = 1, m.end()
        while depth:
            c = text[i]
            if c == '"':
                i = text.index('"', i + 1)
            depth += (c == "(") - (c == ")")
            i += 1
        body = text[m.end():i - 1]
        template = re.match(r'\s*(?:"[^"]*"\s*)*', body).group(0)
        lines = "".join(re.findall(r'"([^"]*)"', template)).replace("\\t", "").split("\\n")
        yield [v.strip() for v in lines if v.strip()], body[len(template):]


FILES = sorted(glob.glob(os.path.join(CSRC, "moe_*")))


def test_the_product_has_such_statements():
    found = [s for f in FILES for s in statements(f)]
    assert sum("m0" in " ".join(lines) for lines, _ in found) == 3


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_statements_name_what_they_change(path):
    for lines, rest in statements(path):
        if any(re.search(r"^s_\w+\s+m0\b", v) for v in lines):
            assert '"m0"' in rest, lines
        changes = [v for v in lines if re.search(r"^s_\w+\s+exec", v)]
        if changes:
            saved = [re.match(r"s_mov_b64\s+(%\d+),\s*exec$", v) for v in lines]
            saved = [m.group(1) for m in saved if m]
            assert len(saved) == 1 and lines[-1] == f"s_mov_b64 exec, {saved[0]}", lines
            assert lines.index(f"s_mov_b64 {saved[0]}, exec") < lines.index(changes[0])
            # no lane that was off is switched on in between
            assert changes[:-1] == ["s_mov_b32 exec_hi, 0"], lines
