"""Wait states in the built gfx950 code of the layer operators' kernels. The
compiler inserts the ones that its own instructions need but does not look
into inline assembly, so the linked code is what is checked: over every path,
branches included, no instruction reads a register sooner after the one that
wrote it than the hardware allows without an interlock."""
import collections
import os
import re

import pytest

import combine_route_amd as cra
import combine_route_amd.build as build

# Wait states from a matrix instruction to a read of its result, by its passes
# of 4 cycles (4: 16x16x32 of 16 bits; 8: 16x16x128 of 8 bits and 32x32x32 of
# int8; any other is taken for one of 16 passes).
PASSES = {"v_mfma_f32_16x16x32_bf16": 4, "v_mfma_f32_16x16x32_f16": 4,
          "v_mfma_f32_16x16x128_f8f6f4": 8, "v_mfma_i32_32x32x32_i8": 8}
MATRIX_WAITS = {4: 8, 8: 12, 16: 20}
SCALAR_WAITS = 5    # a vector instruction's scalar result to a memory instruction
LANE_WAITS = 4      # the same to a lane number
DPP_WAITS = 2       # a vector result to an operand from other lanes
TRANS_WAITS = 1     # exp, rcp and their like to a vector instruction
M0_WAITS = 1        # M0 to a load to LDS
STORE_WAITS = 1     # a store of more than 8 bytes to a new value of what it stores

MEMORY = ("buffer_", "global_", "flat_", "scratch_")
TRANS = re.compile(r"v_(exp|log|rcp|rsq|sqrt|sin|cos)_(f16|f32|f64|iflag)")
DPP = re.compile(r"\b(quad_perm|row_\w+|wave_\w+|bank_mask)")

Inst = collections.namedtuple("Inst", "text op ops target")


def registers(token):
    token = token.strip().strip("-|").replace("neg(", "").replace("abs(", "").strip("()|-")
    m = re.match(r"([vas])\[(\d+):(\d+)\]$", token)
    if m:
        return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
    m = re.match(r"([vas])(\d+)$", token)
    if m:
        return {(m[1], int(m[2]))}
    return {("vcc", 0)} if token == "vcc" else {("m0", 0)} if token == "m0" else set()


def operands(text):
    """Register sets of an instruction's operands, in order; modifiers
    behind an operand are dropped."""
    return [registers(t.split()[0]) if t.split() else set() for t in text.split(",")]


def functions(asm, wanted):
    """(name, list of Inst) of the functions whose name has one of the wanted
    parts; a target is the index that a branch goes to."""
    for part in re.split(r"^[0-9a-f]{16} <", asm, flags=re.M)[1:]:
        name, body = part.split(">:", 1)
        if not any(w in name for w in wanted):
            continue
        rows, at = [], {}
        for m in re.finditer(r"^\t(\S+)([^\n]*?)\s*// ([0-9A-F]+):([^\n]*)$", body, re.M):
            at[int(m[3], 16)] = len(rows)
            rows.append((m[1], m[2].strip(), m[4]))
        base = min(at) if at else 0
        insts = []
        for op, rest, enc in rows:
            target = None
            if op.startswith(("s_cbranch", "s_branch")):
                m = re.search(r"\+0x([0-9a-f]+)>", enc)
                target = at[base + (int(m[1], 16) if m else 0)]
            insts.append(Inst(f"{op} {rest}", op, operands(rest), target))
        yield name, insts


def is_vector(op):
    return op.startswith("v_")


def is_lds_load(i):
    return i.op.startswith("buffer_load") and i.text.split()[-1] == "lds"


def split(i):
    """Registers an instruction writes, and reads."""
    if i.op.startswith(("ds_write", "ds_add", "ds_or")) or "_store_" in i.op or is_lds_load(i):
        n = 0
    elif i.op.startswith("s_cmp") or i.op.startswith("s_bitcmp"):
        n = 0
    elif re.match(r"v_(add|sub|subrev|addc|subb)_co_|v_div_scale|v_mad_[ui]64", i.op):
        n = 2
    else:
        n = 1
    writes = set().union(*i.ops[:n]) if i.ops[:n] else set()
    reads = set().union(*i.ops[n:]) if i.ops[n:] else set()
    if re.match(r"v_(fmac|mac|dot\w*c)_|v_writelane|v_swap", i.op):
        reads |= writes
    return writes, reads


def walk(insts, start, regs, limit, bad):
    """Instructions within `limit` states of `start` on any path for which
    bad(inst, live registers, states) holds."""
    found, seen = [], set()
    stack = [(start + 1, 0, frozenset(regs))]
    while stack:
        j, states, live = stack.pop()
        if states >= limit or j >= len(insts) or not live or (j, states, live) in seen:
            continue
        seen.add((j, states, live))
        i = insts[j]
        if bad(i, live, states):
            found.append((j, states))
            continue
        if i.op == "s_endpgm":
            continue
        if i.op == "s_nop":
            stack.append((j + 1, states + int(i.text.split()[1], 0) + 1, live))
            continue
        left = live - split(i)[0]
        if i.target is not None:
            stack.append((i.target, states + 1, left))
            if i.op == "s_branch":
                continue
        stack.append((j + 1, states + 1, left))
    return found


def hazards(insts):
    """(kind, writer, reader, states) of everything that comes too soon."""
    out = []

    def check(kind, n, regs, limit, bad):
        for j, states in walk(insts, n, regs, limit, bad):
            out.append((kind, insts[n].text, insts[j].text, states))

    def reads(i, live):
        return bool(split(i)[1] & live)

    for n, i in enumerate(insts):
        if re.match(r"(buffer|global|flat|scratch)_store_dwordx[34]", i.op):
            data = i.ops[0] if i.op.startswith("buffer_") else i.ops[1]
            if not (i.op.startswith("buffer_") and registers(i.text.split(",")[3].split()[0])):
                check("store", n, data, STORE_WAITS,
                      lambda k, live, s: is_vector(k.op) and bool(split(k)[0] & live))
            continue
        if not is_vector(i.op):
            if i.op.startswith("s_") and ("m0", 0) in split(i)[0]:
                check("m0", n, {("m0", 0)}, M0_WAITS, lambda k, live, s: is_lds_load(k))
            continue
        writes, _ = split(i)
        if i.op.startswith("v_mfma"):
            limit = MATRIX_WAITS[PASSES.get(i.op, 16)]
            check("matrix", n, writes, limit,
                  lambda k, live, s: not k.op.startswith("v_mfma") and
                  (reads(k, live) or (is_vector(k.op) and bool(split(k)[0] & live))))
            check("matrix operand", n, writes, limit,
                  lambda k, live, s: k.op.startswith("v_mfma") and
                  bool((k.ops[1] | k.ops[2]) & live))
            continue
        scalar = {r for r in writes if r[0] in ("s", "vcc")}
        if scalar:
            check("scalar", n, scalar, SCALAR_WAITS,
                  lambda k, live, s: k.op.startswith(MEMORY) and reads(k, live))
            check("lane", n, scalar, LANE_WAITS,
                  lambda k, live, s: re.match(r"v_(read|write)lane", k.op) is not None and
                  bool(k.ops[2] & live))
        vector = writes - scalar
        if vector:
            check("lanes", n, vector, DPP_WAITS,
                  lambda k, live, s: is_vector(k.op) and DPP.search(k.text) is not None and
                  bool(k.ops[1] & live))
        if TRANS.match(i.op):
            check("trans", n, vector, TRANS_WAITS,
                  lambda k, live, s: is_vector(k.op) and not TRANS.match(k.op) and reads(k, live))
    return out


@pytest.fixture(scope="module")
def code():
    if not os.path.exists(cra.LIB_PATH):
        build.build()
    return dict(functions(build.device_code(cra.LIB_PATH), ("3moe", "5block")))


def test_the_scan_sees_each_kind():
    """Each hazard in a few lines of its own, and the same with its waits."""
    def of(*lines):
        insts = []
        for t in lines:
            op, _, rest = t.partition(" ")
            target = int(rest) if op.startswith(("s_cbranch", "s_branch")) else None
            insts.append(Inst(t, op, operands(rest) if target is None else [], target))
        return [h[0] for h in hazards(insts)]

    load = "buffer_load_dwordx4 v1, s[4:7], s3 offen lds"
    for write in ("v_readfirstlane_b32 s5, v0", "v_readlane_b32 s3, v0, 4",
                  "v_cmp_gt_u32_e64 s[4:5], v0, v1"):
        assert of(write, "s_mov_b32 m0, s9", "s_nop 2", load) == ["scalar"]
        assert of(write, "s_mov_b32 m0, s9", "s_nop 3", load) == []
    # the register written again, by an instruction that is waited for
    assert of("v_readfirstlane_b32 s5, v0", "s_mov_b32 s5, 0", load) == []
    # behind a branch
    assert of("v_readfirstlane_b32 s5, v0", "s_cbranch_scc1 3", "s_nop 7", load) == ["scalar"]
    assert of("s_mov_b32 m0, s9", load) == ["m0"]
    assert of("s_mov_b32 m0, s9", "s_nop 0", load) == []
    mfma = "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]"
    assert of(mfma, "s_nop 6", "v_add_f32_e32 v9, v9, v3") == ["matrix"]
    assert of(mfma, "s_nop 7", "v_add_f32_e32 v9, v9, v3") == []
    assert of(mfma, "s_nop 6", "v_mov_b32_e32 v3, 0") == ["matrix"]
    assert of(mfma, "ds_write_b128 v20, v[0:3]") == ["matrix"]
    assert of(mfma, "s_cbranch_scc0 3", "s_nop 7", "v_add_f32_e32 v9, v9, v3") == ["matrix"]
    assert of(mfma, mfma.replace("v[8:11]", "v[0:3]")) == ["matrix operand"]
    assert of(mfma, mfma) == []
    assert of("v_mov_b32_e32 v2, 0", "v_mov_b32_dpp v3, v2 row_ror:4 row_mask:0xf bank_mask:0xf") \
        == ["lanes"]
    assert of("v_exp_f32_e32 v2, v2", "v_add_f32_e32 v3, v2, v2") == ["trans"]
    assert of("v_readfirstlane_b32 s5, v0", "v_readlane_b32 s6, v1, s5") == ["lane"]
    for store in ("buffer_store_dwordx4 v[0:3], v9, s[4:7], 0 offen",
                  "global_store_dwordx4 v9, v[0:3], s[4:5]"):
        assert of(store, "v_mov_b32_e32 v3, 0") == ["store"]
        assert of(store, "s_nop 0", "v_mov_b32_e32 v3, 0") == []


def test_no_register_is_read_too_soon(code):
    assert sum(i.op.startswith("v_mfma") for v in code.values() for i in v) > 1000
    assert sum(is_lds_load(i) for v in code.values() for i in v) > 1000
    found = {n: hazards(v) for n, v in code.items()}
    found = {n: h for n, h in found.items() if h}
    assert not found, "\n".join(
        f"{n[:80]}: {k}: {w} -> {r} ({s} states between)"
        for n, h in found.items() for k, w, r, s in h[:6])
