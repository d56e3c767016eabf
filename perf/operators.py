"""Cases and plain forms of the operators around the MoE dispatch and combine.

Five operators, each with the smallest calls a user makes, ordinary ones and
the largest:

  rms_norm   RMS norm of token rows with the residual's addition; out in the
             input's type and / or as FP8 E4M3 codes with one FP32 scale per
             128 elements, the rows an FP8 dispatch sends.
  gemm       product of the expert-major FP8 rows (a scale per row and 128
             elements) with each expert's FP8 weights (a scale per 128 x 128
             block), rows counted per expert on the GPU.
  swiglu     the same product with gate and up weights, silu(gate) * up taken
             in FP32 and written as FP8 rows with scales: the input of the
             experts' second product.
  combine_backward   gradient of the weighted expert-major combine.
  dispatch_backward  gradient of the expert-major dispatch.

``own = False`` computes them with elementary torch operations in 32 bits;
``own = True`` calls the framework. Everything else (cases, inputs, outputs'
layout) is common to both.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
TINY = 2.0 ** -100        # smallest block maximum that is scaled up to the codes' range
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of one rank: latency counts
        dict(name="norm_decode", op="rms_norm", groups=1, rows=128, hidden=7168, dtype="bf16",
             residual=True, out=True, quant=True, ragged=False),
        # ragged ranks, norm straight to the dispatch's FP8 rows, no residual
        dict(name="norm_ragged", op="rms_norm", groups=4, rows=1024, hidden=2048, dtype="fp16",
             residual=False, out=False, quant=True, ragged=True),
        # 8 ranks x 4096 tokens: the rows of a large dispatch
        dict(name="norm_prefill", op="rms_norm", groups=8, rows=4096, hidden=7168, dtype="bf16",
             residual=True, out=True, quant=True, ragged=False),
        # the smallest layer: 8 experts, 32 tokens, top-2
        dict(name="gemm_small", op="gemm", groups=8, cap=32, pairs=64, n=256, k=256, dtype="bf16",
             skew=False),
        # decode over all 256 experts, 8 x 128 tokens, top-8: every expert's weights are read
        dict(name="gemm_decode", op="gemm", groups=256, cap=256, pairs=8192, n=7168, k=2048,
             dtype="bf16", skew=False),
        # down projection of one rank's 32 experts in a prompt of 8 x 4096 tokens
        dict(name="gemm_prefill", op="gemm", groups=32, cap=2048, pairs=32768, n=7168, k=2048,
             dtype="bf16", skew=False),
        # gate and up projection of one rank's 32 experts, decode
        dict(name="swiglu_decode", op="swiglu", groups=32, cap=128, pairs=1024, inter=2048, k=7168,
             skew=False),
        # and in a prompt, with skewed routing (some experts overflow their capacity)
        dict(name="swiglu_prefill", op="swiglu", groups=32, cap=4096, pairs=32768, inter=2048,
             k=7168, skew=True),
        # gradient of a small layer's combine
        dict(name="combine_bwd_small", op="combine_backward", ranks=4, tokens=256, hidden=4096,
             experts=256, topk=8, cap=64, dtype="bf16", ragged=False, weighted=True,
             repeats=False),
        # and of a training step's: 8 ranks x 2048 tokens
        dict(name="combine_bwd_large", op="combine_backward", ranks=8, tokens=2048, hidden=7168,
             experts=256, topk=8, cap=768, dtype="bf16", ragged=False, weighted=True,
             repeats=False),
        # gradient of a ragged top-64 dispatch
        dict(name="dispatch_bwd_top64", op="dispatch_backward", ranks=4, tokens=1024, hidden=2048,
             experts=256, topk=64, cap=1024, dtype="fp16", ragged=True, repeats=False),
        # and of a training step's
        dict(name="dispatch_bwd_large", op="dispatch_backward", ranks=8, tokens=2048, hidden=7168,
             experts=256, topk=8, cap=768, dtype="bf16", ragged=False, repeats=False),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_norm(rng):
    quant = rng.random() < 0.7
    step = 128 if quant else 8
    hidden = step * _log(rng, 1, 16384 // step)
    rows = _log(rng, 1, max(1, min(32768, 200_000_000 // hidden)))
    groups = min(rows, rng.choice([1, 1, 2, 3, 4, 8]))
    return dict(op="rms_norm", groups=groups, rows=max(1, rows // groups), hidden=hidden,
                dtype=rng.choice(["bf16", "fp16"]), residual=rng.random() < 0.6,
                out=(not quant) or rng.random() < 0.5, quant=quant, ragged=rng.random() < 0.5)


def _draw_product(rng, op):
    k = 128 * _log(rng, 1, 56)
    n = 128 * _log(rng, 1, 16) if op == "swiglu" else 8 * _log(rng, 1, 896)
    wide = 2 * n if op == "swiglu" else n
    groups = _log(rng, 1, max(1, min(256, 3_000_000_000 // (wide * k))))
    most = min(65536, int(1.8e12 / (2.0 * wide * k)), 2_000_000_000 // (wide + k))
    pairs = _log(rng, 1, max(1, most))
    mean = max(1, pairs // groups)
    cap = max(1, min(int(mean * rng.uniform(0.7, 2.5)) + rng.randint(0, 16),
                     1_500_000_000 // (groups * (wide + k)) + 1))
    case = dict(op=op, groups=groups, cap=cap, pairs=pairs, k=k, skew=rng.random() < 0.4)
    if op == "swiglu":
        return dict(case, inter=n)
    return dict(case, n=n, dtype=rng.choice(["bf16", "fp16"]))


def _draw_backward(rng, op):
    ranks = rng.choice([1, 2, 3, 4, 8])
    hidden = 8 * _log(rng, 8, 896)
    topk = rng.choice([1, 2, 3, 4, 6, 8, 8, 16, 37, 64])
    experts = ranks * _log(rng, max(1, -(-topk // ranks)), max(64, 256 // ranks))
    most = max(1, min(4096, 700_000_000 // (ranks * topk * hidden)))
    tokens = _log(rng, 1, most)
    mean = ranks * tokens * topk / experts
    cap = max(1, min(ranks * tokens, int(mean * rng.uniform(0.6, 2.0)) + rng.randint(0, 8)))
    case = dict(op=op, ranks=ranks, tokens=tokens, hidden=hidden, experts=experts, topk=topk,
                cap=cap, dtype=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.5,
                repeats=rng.random() < 0.4)
    if op == "combine_backward":
        case["weighted"] = rng.random() < 0.7
    return case


def draw(rng):
    op = rng.choice(["rms_norm", "gemm", "swiglu", "combine_backward", "dispatch_backward"])
    if op == "rms_norm":
        return _draw_norm(rng)
    if op in ("gemm", "swiglu"):
        return _draw_product(rng, op)
    return _draw_backward(rng, op)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed, stream=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * seed + stream)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _ragged(groups, rows, g):
    return torch.randint(0, rows + 1, (groups,), generator=g, device="cuda", dtype=torch.int32)


def _popularity(groups, skew):
    """Share of the routed pairs each expert gets."""
    if not skew:
        return [1.0 / groups] * groups
    p = [(i + 1.0) ** -0.7 for i in range(groups)]
    return [v / sum(p) for v in p]


def _counts(case, g):
    """Rows routed to each expert: case["pairs"] of them in all, some maybe
    past the capacity, as a dispatch counts them."""
    groups = case["groups"]
    p = torch.tensor(_popularity(groups, case["skew"]), device="cuda")
    p = p[torch.randperm(groups, generator=g, device="cuda")]
    ids = torch.multinomial(p, case["pairs"], replacement=True, generator=g)
    return torch.zeros(groups, dtype=torch.int32, device="cuda").index_add_(
        0, ids, torch.ones_like(ids, dtype=torch.int32))


def _to_codes(v, dims):
    """FP8 codes of v and their scales, one per block reduced over dims."""
    amax = v.abs().amax(dims, keepdim=True).clamp_min(TINY)
    return (v * (E4M3_MAX / amax)).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), amax / E4M3_MAX


def _activation_rows(groups, cap, k, g):
    codes = torch.empty((groups, cap, k), dtype=E4M3, device="cuda")
    scales = torch.empty((groups, cap, k // 128), dtype=torch.float32, device="cuda")
    step = max(1, 100_000_000 // (cap * k))
    for i in range(0, groups, step):
        n = min(step, groups - i)
        c, s = _to_codes(_randn((n, cap, k // 128, 128), g), (3,))
        codes[i:i + n] = c.view(n, cap, k)
        scales[i:i + n] = s.view(n, cap, k // 128)
    return codes, scales


def _weight_blocks(groups, n, k, g):
    blocks = -(-n // 128)
    codes = torch.empty((groups, n, k), dtype=E4M3, device="cuda")
    scales = torch.empty((groups, blocks, k // 128), dtype=torch.float32, device="cuda")
    step = max(1, 100_000_000 // (blocks * 128 * k))
    for i in range(0, groups, step):
        m = min(step, groups - i)
        w = _randn((m, blocks, 128, k // 128, 128), g) * k ** -0.5
        c, s = _to_codes(w, (2, 4))
        codes[i:i + m] = c.view(m, blocks * 128, k)[:, :n]
        scales[i:i + m] = s.view(m, blocks, k // 128)
    return codes, scales


def _prepare_norm(case, seed):
    g = _gen(seed)
    dt = DTYPE[case["dtype"]]
    shape = (case["groups"], case["rows"], case["hidden"])
    s = dict(op="rms_norm", counts=None, residual=None, residual_out=None, out=None, codes=None,
             scales=None)
    s["x"] = _randn(shape, g).to(dt)
    s["weight"] = (1.0 + 0.1 * _randn(shape[2:], g)).to(dt)
    if case["residual"]:
        s["residual"] = (2.0 * _randn(shape, g)).to(dt)
        s["residual_out"] = torch.zeros(shape, dtype=dt, device="cuda")
    if case["out"]:
        s["out"] = torch.zeros(shape, dtype=dt, device="cuda")
    if case["quant"]:
        s["codes"] = torch.zeros(shape, dtype=torch.uint8, device="cuda").view(E4M3)
        s["scales"] = torch.zeros(shape[:2] + (shape[2] // 128,), dtype=torch.float32,
                                  device="cuda")
    if case["ragged"]:
        s["counts"] = _ragged(case["groups"], case["rows"], g)
    return s


def _prepare_product(case, seed):
    g = _gen(seed)
    groups, cap, k = case["groups"], case["cap"], case["k"]
    swiglu = case["op"] == "swiglu"
    wide = 2 * case["inter"] if swiglu else case["n"]
    s = dict(op=case["op"], counts=_counts(case, g))
    s["a"], s["a_scales"] = _activation_rows(groups, cap, k, g)
    s["b"], s["b_scales"] = _weight_blocks(groups, wide, k, g)
    if swiglu:
        inter = case["inter"]
        s["codes"] = torch.zeros((groups, cap, inter), dtype=torch.uint8, device="cuda").view(E4M3)
        s["scales"] = torch.zeros((groups, cap, inter // 128), dtype=torch.float32, device="cuda")
    else:
        s["out"] = torch.zeros((groups, cap, wide), dtype=DTYPE[case["dtype"]], device="cuda")
    return s


def _expert_ids(case, g):
    """[W, M, k] expert ids: distinct ones, or with repeats and ids that name
    no expert."""
    shape = (case["ranks"] * case["tokens"], case["topk"])
    E = case["experts"]
    if case["repeats"] or case["topk"] > E:
        ids = torch.randint(-1, E + 1, shape, generator=g, device="cuda")
    else:
        ids = torch.rand((shape[0], E), generator=g, device="cuda").argsort(1)[:, :shape[1]]
    return ids.to(torch.int32).view(case["ranks"], case["tokens"], case["topk"]).contiguous()


def _packed_rows(case, ids, ntok):
    """[N, k] packed row of each slot that is its expert's first in the token
    and within the capacity, else -1; and the [N, k] first slot of each slot's
    expert. An expert's rows are in token order."""
    E, cap, M = case["experts"], case["cap"], case["tokens"]
    flat = ids.view(-1, case["topk"]).long()
    n, k = flat.shape
    there = (torch.arange(M, device="cuda")[None] <
             torch.tensor(ntok, device="cuda")[:, None]).view(-1, 1)
    valid = (flat >= 0) & (flat < E) & there
    first = torch.zeros_like(flat)
    for j in range(k - 1, -1, -1):
        first = torch.where(flat == flat[:, j:j + 1], j, first)
    lead = valid & (first == torch.arange(k, device="cuda"))
    at = lead.nonzero()                       # token order
    e = flat[at[:, 0], at[:, 1]]
    order = torch.argsort(e, stable=True)
    count = torch.bincount(e, minlength=E)
    start = torch.cumsum(count, 0) - count
    pos = torch.empty_like(e)
    pos[order] = torch.arange(len(e), device="cuda") - start[e[order]]
    rows = torch.full_like(flat, -1)
    rows[at[:, 0], at[:, 1]] = torch.where(pos < cap, e * cap + pos, -1)
    return rows, first, valid


def _prepare_backward(case, seed):
    g = _gen(seed)
    dt = DTYPE[case["dtype"]]
    W, M, H, k = case["ranks"], case["tokens"], case["hidden"], case["topk"]
    E, cap = case["experts"], case["cap"]
    ntok = [M] * W
    if case["ragged"]:
        ntok = [int(v) for v in _ragged(W, M, g).cpu()]
    ids = _expert_ids(case, g)
    rows, first, valid = _packed_rows(case, ids, ntok)
    s = dict(op=case["op"], ids=ids, rows=rows, first=first, valid=valid, plan=None)
    if case["op"] == "combine_backward":
        s["grad_out"] = _randn((W, M, H), g).to(dt)
        s["packed_y"] = _randn((E * cap * H,), g).to(dt).view(W, E // W, cap, H)
        s["weights"] = None
        if case["weighted"]:
            s["weights"] = torch.softmax(_randn((W, M, k), g), -1)
        s["grad_packed_y"] = torch.zeros((W, E // W, cap, H), dtype=dt, device="cuda")
        s["grad_weights"] = torch.zeros((W, M, k), device="cuda") if case["weighted"] else None
    else:
        s["grad_packed_x"] = _randn((E * cap * H,), g).to(dt).view(W, E // W, cap, H)
        s["grad_x"] = torch.zeros((W, M, H), dtype=dt, device="cuda")
    if own:  # the forward's plan, which a training program holds
        import combine_route_amd as cra
        cfg = cra.make_config(W, H, M, E // W, k, case["dtype"])
        s["plan"] = cra.EpDispatchCombineOp(cfg, with_weights=False, expert_capacity=cap)
        s["plan"].dispatch_standard_moe(torch.zeros((W, M, H), dtype=dt, device="cuda"), None,
                                        None, ids, ntok)
    return s


def prepare(case, seed):
    if case["op"] == "rms_norm":
        return _prepare_norm(case, seed)
    if case["op"] in ("gemm", "swiglu"):
        return _prepare_product(case, seed)
    return _prepare_backward(case, seed)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _kept(counts, cap):
    """[G, cap, 1] truth values: rows that a group's count reaches."""
    return (torch.arange(cap, device="cuda")[None] < counts[:, None])[..., None]


def _quantized(y):
    """Codes and scales of y [..., H] in FP32, a scale per 128 elements."""
    b = y.unflatten(-1, (-1, 128))
    amax = b.abs().amax(-1, keepdim=True)
    up = amax.clamp_min(TINY)
    scale = torch.where(amax > 0, up / E4M3_MAX, 1.0)
    codes = (b * (E4M3_MAX / up)).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    return codes.flatten(-2), scale.squeeze(-1)


def _plain_norm(s):
    x, res = s["x"], s["residual"]
    keep = None if s["counts"] is None else _kept(s["counts"], x.shape[1])

    def masked(v):
        return v if keep is None else torch.where(keep, v, 0)

    h = x.float()
    r = {}
    if res is not None:
        stream = (h + res.float()).to(x.dtype)
        r["residual"] = masked(stream)
        h = stream.float()
    inv = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    y = h * inv * s["weight"].float()
    if s["out"] is not None:
        r["out"] = masked(y.to(x.dtype))
    if s["codes"] is not None:
        codes, scales = _quantized(y)
        r["codes"] = masked(codes.float()).to(E4M3)
        r["scales"] = masked(scales)
    return r


def _plain_product(s):
    a = (s["a"].float().unflatten(-1, (-1, 128)) * s["a_scales"][..., None]).flatten(-2)
    n = s["b"].shape[1]
    block = torch.arange(n, device="cuda") // 128
    b = (s["b"].float().unflatten(-1, (-1, 128)) * s["b_scales"][:, block, :, None]).flatten(-2)
    return torch.bmm(a, b.transpose(1, 2).contiguous())


def _plain_gemm(s):
    y = _plain_product(s)
    return torch.where(_kept(s["counts"], y.shape[1]), y, 0).to(s["out"].dtype)


def _plain_swiglu(s):
    y = _plain_product(s)
    inter = y.shape[2] // 2
    gate, up = y[..., :inter], y[..., inter:]
    codes, scales = _quantized(gate / (1.0 + torch.exp(-gate)) * up)
    keep = _kept(s["counts"], y.shape[1])
    return {"codes": torch.where(keep, codes.float(), 0).to(E4M3),
            "scales": torch.where(keep, scales, 0)}


def _plain_combine_backward(s):
    H = s["grad_out"].shape[-1]
    go = s["grad_out"].view(-1, H).float()
    rows = s["rows"]
    tok, slot = (rows >= 0).nonzero(as_tuple=True)
    at = rows[tok, slot]
    g = go[tok]
    gy = torch.zeros_like(s["packed_y"]).view(-1, H)
    if s["weights"] is None:
        gy[at] = g.to(gy.dtype)
        return {"grad_packed_y": gy.view_as(s["packed_y"])}
    w = s["weights"].view(rows.shape)
    # weight of an expert in a token: of all the slots that name it
    c = torch.zeros_like(w).scatter_add_(1, s["first"], w)
    gy[at] = (g * c[tok, slot][:, None]).to(gy.dtype)
    dots = torch.zeros_like(w)
    dots[tok, slot] = (g * s["packed_y"].view(-1, H)[at].float()).sum(-1)
    gw = torch.where(s["valid"], dots.gather(1, s["first"]), 0)
    return {"grad_packed_y": gy.view_as(s["packed_y"]), "grad_weights": gw.view_as(s["weights"])}


def _plain_dispatch_backward(s):
    H = s["grad_x"].shape[-1]
    gp = s["grad_packed_x"].view(-1, H)
    rows = s["rows"]
    picked = torch.where((rows >= 0)[..., None], gp[rows.clamp_min(0)].float(), 0)
    return picked.sum(1).to(s["grad_x"].dtype).view_as(s["grad_x"])


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own_norm(s):
    import combine_route_amd as cra
    cra.moe_rms_norm(s["x"], s["weight"], EPS, out=s["out"], residual=s["residual"],
                     residual_out=s["residual_out"], codes=s["codes"], scales=s["scales"],
                     counts=s["counts"])
    names = (("residual", "residual_out"), ("out", "out"), ("codes", "codes"),
             ("scales", "scales"))
    return {name: s[key] for name, key in names if s[key] is not None}


def _own_gemm(s):
    import combine_route_amd as cra
    cra.moe_grouped_gemm(s["a"], s["a_scales"], s["b"], s["b_scales"], s["out"],
                         counts=s["counts"])
    return s["out"]


def _own_swiglu(s):
    import combine_route_amd as cra
    cra.moe_grouped_gemm_swiglu(s["a"], s["a_scales"], s["b"], s["b_scales"], s["codes"],
                                s["scales"], counts=s["counts"])
    return {"codes": s["codes"], "scales": s["scales"]}


def _own_combine_backward(s):
    gy, gw = s["plan"].combine_standard_moe_backward(
        s["grad_out"], s["weights"], s["ids"], s["packed_y"] if s["weights"] is not None else None,
        grad_packed_y=s["grad_packed_y"], grad_weights=s["grad_weights"])
    return {"grad_packed_y": gy} if gw is None else {"grad_packed_y": gy, "grad_weights": gw}


def _own_dispatch_backward(s):
    return s["plan"].dispatch_standard_moe_backward(s["grad_packed_x"], grad_x=s["grad_x"])


def run(s):
    if own:
        return {"rms_norm": _own_norm, "gemm": _own_gemm, "swiglu": _own_swiglu,
                "combine_backward": _own_combine_backward,
                "dispatch_backward": _own_dispatch_backward}[s["op"]](s)
    return {"rms_norm": _plain_norm, "gemm": _plain_gemm, "swiglu": _plain_swiglu,
            "combine_backward": _plain_combine_backward,
            "dispatch_backward": _plain_dispatch_backward}[s["op"]](s)


# ---------------------------------------------------------------------------
# work and definition
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "rms_norm":
        H = case["hidden"]
        rows = case["groups"] * case["rows"] * (0.5 if case["ragged"] else 1.0)
        row = 2 * H * (1 + 2 * case["residual"] + case["out"]) + case["quant"] * (H + H // 32)
        return {"bytes": rows * row + 2 * H, "flops": rows * H * 8}
    if case["op"] in ("gemm", "swiglu"):
        swiglu = case["op"] == "swiglu"
        n, k = 2 * case["inter"] if swiglu else case["n"], case["k"]
        p = _popularity(case["groups"], case["skew"])
        hit = sum(1.0 - (1.0 - v) ** case["pairs"] for v in p)
        rows = sum(min(case["cap"], v * case["pairs"]) for v in p)
        out = n / 2 * (1 + 1 / 32) if swiglu else 2 * n
        return {"bytes": rows * (k * (1 + 1 / 32) + out) + hit * n * k * (1 + 4 / 16384),
                "flops": 2.0 * rows * n * k}
    H = case["hidden"]
    tokens = case["ranks"] * case["tokens"] * (0.5 if case["ragged"] else 1.0)
    pairs = min(tokens * case["topk"] * (0.8 if case["repeats"] else 1.0),
                case["experts"] * case["cap"])
    if case["op"] == "combine_backward":
        rows = tokens * H * 2 + pairs * H * 2 * (2 if case["weighted"] else 1)
        return {"bytes": rows + tokens * case["topk"] * (16 if case["weighted"] else 8),
                "flops": pairs * H * (3.0 if case["weighted"] else 1.0)}
    return {"bytes": pairs * H * 2 + tokens * H * 2 + tokens * case["topk"] * 4,
            "flops": pairs * H}


def _exact_blocks(y):
    """[..., H] in 64 bits -> values in units of the block scale, and scales."""
    top = y.abs().reshape(y.shape[:-1] + (-1, 128)).max(-1).values
    scale = torch.maximum(top, torch.full_like(top, TINY)) / E4M3_MAX
    scale = scale.masked_fill(top == 0, 1.0)
    return y / scale.repeat_interleave(128, -1), scale


def _exact_norm(case, seed):
    s = _prepare_norm(case, seed)
    G, M, H = s["x"].shape
    dt = s["x"].dtype
    r = {}
    for name, key in (("residual", "residual"), ("out", "out"), ("codes", "codes")):
        if s[key] is not None:
            r[name] = torch.zeros((G, M, H), dtype=torch.float64, device="cuda")
    if s["scales"] is not None:
        r["scales"] = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
    for g in range(G):
        n = M if s["counts"] is None else int(s["counts"][g])
        v = s["x"][g, :n].double()
        if s["residual"] is not None:
            v = v + s["residual"][g, :n].double()
            r["residual"][g, :n] = v
            v = v.to(dt).double()
        v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / H + EPS) * s["weight"].double()
        if "out" in r:
            r["out"][g, :n] = v
        if "codes" in r:
            r["codes"][g, :n], r["scales"][g, :n] = _exact_blocks(v)
    return r


def _exact_product(case, seed):
    s = _prepare_product(case, seed)
    G, cap, k = s["a"].shape
    n = s["b"].shape[1]
    swiglu = case["op"] == "swiglu"
    if swiglu:
        inter = n // 2
        codes = torch.zeros((G, cap, inter), dtype=torch.float64, device="cuda")
        scales = torch.zeros((G, cap, inter // 128), dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros((G, cap, n), dtype=torch.float64, device="cuda")
    for g in range(G):
        m = min(cap, int(s["counts"][g]))
        if m == 0:
            continue
        a = s["a"][g, :m].double() * s["a_scales"][g, :m].double().repeat_interleave(128, 1)
        sb = s["b_scales"][g].double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
        y = a @ (s["b"][g].double() * sb).t()
        if swiglu:
            gate, up = y[:, :inter], y[:, inter:]
            codes[g, :m], scales[g, :m] = _exact_blocks(gate * torch.sigmoid(gate) * up)
        else:
            out[g, :m] = y
    return {"codes": codes, "scales": scales} if swiglu else out


def _exact_combine_backward(case, seed):
    s = _prepare_backward(case, seed)
    H, k = case["hidden"], case["topk"]
    go, y = s["grad_out"].view(-1, H), s["packed_y"].view(-1, H)
    gy = torch.zeros(y.shape, dtype=torch.float64, device="cuda")
    ids = s["ids"].view(-1, k)
    w = None if s["weights"] is None else s["weights"].view(-1, k).double()
    gw = torch.zeros(ids.shape, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = (s["rows"][:, j] >= 0).nonzero().squeeze(1)
        row = s["rows"][t, j]
        if w is None:
            gy[row] = go[t].double()
            continue
        same = ids[t] == ids[t, j:j + 1]
        c = (w[t] * same).sum(1, keepdim=True)
        gy[row] = go[t].double() * c
        gw[t] += same * (go[t].double() * y[row].double()).sum(1, keepdim=True)
    r = {"grad_packed_y": gy.view(s["packed_y"].shape)}
    if w is not None:
        r["grad_weights"] = gw.view(s["weights"].shape)
    return r


def _exact_dispatch_backward(case, seed):
    s = _prepare_backward(case, seed)
    H = case["hidden"]
    gp = s["grad_packed_x"].view(-1, H)
    gx = torch.zeros((s["rows"].shape[0], H), dtype=torch.float64, device="cuda")
    for j in range(case["topk"]):
        t = (s["rows"][:, j] >= 0).nonzero().squeeze(1)
        gx[t] += gp[s["rows"][t, j]].double()
    return gx.view(s["grad_x"].shape)


def exact(case, seed):
    return {"rms_norm": _exact_norm, "gemm": _exact_product, "swiglu": _exact_product,
            "combine_backward": _exact_combine_backward,
            "dispatch_backward": _exact_dispatch_backward}[case["op"]](case, seed)
