"""Cases and plain forms of the operators of a whole MoE block: the norms
around it, its experts in 8-bit integers, and the layer of a few tokens.

  block_norm   RMS norm of a block's output, gate, scaled residual, and the
               next block's RMS norm; out as rows, as FP8 E4M3 codes with one
               FP32 scale per 128 elements, or as INT8 codes with one FP32
               scale per row.
  block_norm_backward   its gradients.
  gemm_int8    product of the expert-major INT8 rows (a scale per row) with
               each expert's INT8 weights (a scale per output channel), rows
               counted per expert on the GPU.
  mlp_int8     an expert's two products in INT8: gate and up with silu(gate) *
               up, those rows quantized, and the down product.
  few_tokens   a whole layer's experts for a few tokens, weights in FP8 (a
               scale per 128 x 128) or INT8 (a scale per channel), summed with
               the routing weights.

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
INT8_MAX = 127.0
TINY = 2.0 ** -100        # smallest maximum that is scaled up to the codes' range
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of one rank, norm to the rows of the FP8 dispatch: latency counts
        dict(name="norm_decode", op="block_norm", groups=1, rows=128, hidden=7168, dtype="bf16",
             post=True, gate="channel", scale=1.0, out=True, quant="fp8", ragged=False),
        # 8 ranks x 4096 tokens, norm to INT8 rows, a gate per rank's sequence
        dict(name="norm_prefill", op="block_norm", groups=8, rows=4096, hidden=7168, dtype="bf16",
             post=True, gate="group", scale=0.5, out=False, quant="int8", ragged=False),
        # gradients in a small ragged training step
        dict(name="norm_bwd_small", op="block_norm_backward", groups=4, rows=256, hidden=4096,
             dtype="fp16", post=True, gate="channel", scale=1.0, pre=True, ragged=True),
        # and in one of 8 ranks x 2048 tokens
        dict(name="norm_bwd_large", op="block_norm_backward", groups=8, rows=2048, hidden=7168,
             dtype="bf16", post=True, gate="group", scale=0.5, pre=True, ragged=False),
        # the smallest layer: 8 experts, 32 tokens, top-2
        dict(name="int8_small", op="gemm_int8", groups=8, cap=32, pairs=64, n=256, k=256,
             dtype="bf16", skew=False),
        # down projection over all 256 experts, 8 x 128 tokens, top-8
        dict(name="int8_decode", op="gemm_int8", groups=256, cap=256, pairs=8192, n=7168, k=2048,
             dtype="bf16", skew=False),
        # down projection of one rank's 32 experts in a prompt of 8 x 4096 tokens, skewed routing
        dict(name="int8_prefill", op="gemm_int8", groups=32, cap=4096, pairs=32768, n=7168, k=2048,
             dtype="fp16", skew=True),
        # both products of one rank's 32 experts, decode
        dict(name="mlp_decode", op="mlp_int8", groups=32, cap=128, pairs=1024, hidden=7168,
             inter=2048, dtype="bf16", skew=False),
        # and in a prompt
        dict(name="mlp_prefill", op="mlp_int8", groups=32, cap=2048, pairs=32768, hidden=7168,
             inter=2048, dtype="bf16", skew=False),
        # a single token through one of 8 ranks' 256 experts, top-8
        dict(name="one_token", op="few_tokens", experts=256, tokens=1, topk=8, hidden=7168,
             inter=2048, dtype="bf16", weights="fp8", weighted=True, repeats=False),
        # four tokens of a smaller layer, top-4, INT8 weights
        dict(name="four_tokens", op="few_tokens", experts=64, tokens=4, topk=4, hidden=4096,
             inter=1024, dtype="fp16", weights="int8", weighted=True, repeats=False),
        # the largest of the small batches
        dict(name="most_tokens", op="few_tokens", experts=256, tokens=64, topk=8, hidden=7168,
             inter=2048, dtype="bf16", weights="fp8", weighted=True, repeats=False),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_norm(rng, op):
    backward = op == "block_norm_backward"
    quant = rng.choice([None, "fp8", "int8"]) if not backward else None
    step = 128 if quant == "fp8" else 8
    hidden = step * _log(rng, 1, 16384 // step)
    most = 117_000_000 if backward else 230_000_000
    rows = _log(rng, 1, max(1, min(32768, most // hidden)))
    groups = min(rows, rng.choice([1, 1, 2, 3, 4, 8]))
    case = dict(op=op, groups=groups, rows=max(1, rows // groups), hidden=hidden,
                dtype=rng.choice(["bf16", "fp16"]), post=rng.random() < 0.8,
                gate=rng.choice([None, "channel", "group"]), scale=rng.choice([1.0, 0.5, 0.22]),
                ragged=rng.random() < 0.5)
    if backward:
        return dict(case, pre=rng.random() < 0.9)
    return dict(case, out=quant is None or rng.random() < 0.5, quant=quant)


def _draw_product(rng, op):
    if op == "mlp_int8":
        k, n = 16 * _log(rng, 4, 448), 16 * _log(rng, 2, 128)
        wide = 3 * n
    else:
        k, n = 16 * _log(rng, 1, 448), 8 * _log(rng, 1, 896)
        wide = n
    groups = _log(rng, 1, max(1, min(256, 2_000_000_000 // (wide * k))))
    most = min(65536, int(1.8e12 / (2.0 * wide * k)), 1_500_000_000 // (wide + k))
    pairs = _log(rng, 1, max(1, most))
    mean = max(1, pairs // groups)
    cap = max(1, min(int(mean * rng.uniform(0.7, 2.5)) + rng.randint(0, 16),
                     1_500_000_000 // (groups * (wide + k)) + 1))
    case = dict(op=op, groups=groups, cap=cap, pairs=pairs, dtype=rng.choice(["bf16", "fp16"]),
                skew=rng.random() < 0.4)
    return dict(case, hidden=k, inter=n) if op == "mlp_int8" else dict(case, n=n, k=k)


def _draw_few(rng):
    weights = rng.choice(["fp8", "int8"])
    if weights == "fp8":
        hidden, inter = 128 * _log(rng, 1, 56), 128 * _log(rng, 1, 16)
    else:
        hidden, inter = 16 * _log(rng, 4, 448), 16 * _log(rng, 2, 128)
    experts = _log(rng, 1, max(1, min(256, 2_000_000_000 // (3 * hidden * inter))))
    topk = min(rng.choice([1, 2, 3, 4, 6, 8, 8, 16, 37]), max(1, experts))
    return dict(op="few_tokens", experts=experts, tokens=min(64, _log(rng, 1, 64)), topk=topk,
                hidden=hidden, inter=inter, dtype=rng.choice(["bf16", "fp16"]), weights=weights,
                weighted=rng.random() < 0.8, repeats=rng.random() < 0.3)


def draw(rng):
    op = rng.choice(["block_norm", "block_norm_backward", "gemm_int8", "mlp_int8", "few_tokens",
                     "few_tokens"])
    if op.startswith("block_norm"):
        return _draw_norm(rng, op)
    if op in ("gemm_int8", "mlp_int8"):
        return _draw_product(rng, op)
    case = _draw_few(rng)
    if case["tokens"] * case["topk"] > 1024:
        case["tokens"] = 1024 // case["topk"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed, stream=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * seed + stream)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


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


def _row_codes(v):
    """INT8 codes of v's rows and their scales, one a row."""
    amax = v.abs().amax(-1, keepdim=True).clamp_min(TINY)
    return (v * (INT8_MAX / amax)).round().to(torch.int8), (amax / INT8_MAX).squeeze(-1)


def _int8_rows(groups, rows, k, g, size=1.0):
    codes = torch.empty((groups, rows, k), dtype=torch.int8, device="cuda")
    scales = torch.empty((groups, rows), dtype=torch.float32, device="cuda")
    step = max(1, 200_000_000 // (rows * k))
    for i in range(0, groups, step):
        n = min(step, groups - i)
        codes[i:i + n], scales[i:i + n] = _row_codes(_randn((n, rows, k), g) * size)
    return codes, scales


def _fp8_blocks(groups, n, k, g):
    codes = torch.empty((groups, n, k), dtype=E4M3, device="cuda")
    scales = torch.empty((groups, n // 128, k // 128), dtype=torch.float32, device="cuda")
    step = max(1, 200_000_000 // (n * k))
    for i in range(0, groups, step):
        m = min(step, groups - i)
        w = _randn((m, n // 128, 128, k // 128, 128), g) * k ** -0.5
        amax = w.abs().amax((2, 4), keepdim=True).clamp_min(TINY)
        c = (w * (E4M3_MAX / amax)).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
        codes[i:i + m] = c.view(m, n, k)
        scales[i:i + m] = (amax / E4M3_MAX).view(m, n // 128, k // 128)
    return codes, scales


def _prepare_norm(case, seed):
    g = _gen(seed)
    dt = DTYPE[case["dtype"]]
    G, M, H = case["groups"], case["rows"], case["hidden"]
    s = dict(op=case["op"], scale=case["scale"], counts=None, post=None, gate=None, pre=None)
    s["y"] = (0.3 * _randn((G, M, H), g)).to(dt)
    if case["post"]:
        s["post"] = (1.0 + 0.1 * _randn((H,), g)).to(dt)
    if case["gate"]:
        s["gate"] = (0.5 + 0.2 * _randn((G, H) if case["gate"] == "group" else (H,), g)).to(dt)
    if case["ragged"]:
        s["counts"] = torch.randint(0, M + 1, (G,), generator=g, device="cuda", dtype=torch.int32)
        s["counts"][0].clamp_(min=1)
    stream = (2.0 * _randn((G, M, H), g)).to(dt)  # the residual, or h in the backward
    if case["op"] == "block_norm":
        s["pre"] = (1.0 + 0.1 * _randn((H,), g)).to(dt)
        s["residual"] = stream
        s["residual_out"] = torch.zeros_like(stream)
        s["out"] = torch.zeros_like(stream) if case["out"] else None
        s["codes"] = s["scales"] = None
        if case["quant"]:
            s["codes"] = torch.zeros((G, M, H), dtype=torch.int8, device="cuda")
            s["scales"] = torch.zeros((G, M), device="cuda")
        if case["quant"] == "fp8":
            s["codes"] = s["codes"].view(E4M3)
            s["scales"] = torch.zeros((G, M, H // 128), device="cuda")
        return s
    s["h"] = stream
    s["grad_h"] = _randn((G, M, H), g).to(dt)
    s["grad_y"], s["grad_residual"] = torch.zeros_like(stream), torch.zeros_like(stream)
    s["grad_out"] = s["grad_pre"] = None
    if case["pre"]:
        s["pre"] = (1.0 + 0.1 * _randn((H,), g)).to(dt)
        s["grad_out"] = _randn((G, M, H), g).to(dt)
        s["grad_pre"] = torch.zeros((H,), device="cuda")
    s["grad_post"] = torch.zeros((H,), device="cuda") if case["post"] else None
    s["grad_gate"] = torch.zeros(s["gate"].shape, device="cuda") if case["gate"] else None
    s["workspace"] = None
    if own:  # which a training program keeps
        import combine_route_amd as cra
        groups = G if case["ragged"] or case["gate"] == "group" else 1
        s["workspace"] = torch.empty(cra.moe_block_norm_backward_workspace_bytes(G * M, H, groups),
                                     dtype=torch.uint8, device="cuda")
    return s


def _prepare_product(case, seed):
    g = _gen(seed)
    G, cap = case["groups"], case["cap"]
    dt = DTYPE[case["dtype"]]
    s = dict(op=case["op"], counts=_counts(case, g))
    if case["op"] == "gemm_int8":
        n, k = case["n"], case["k"]
        s["a"], s["a_scales"] = _int8_rows(G, cap, k, g)
        s["b"], s["b_scales"] = _int8_rows(G, n, k, g, k ** -0.5)
        s["out"] = torch.zeros((G, cap, n), dtype=dt, device="cuda")
        return s
    H, inter = case["hidden"], case["inter"]
    s["a"], s["a_scales"] = _int8_rows(G, cap, H, g)
    s["gate_up"], s["gate_up_scales"] = _int8_rows(G, 2 * inter, H, g, H ** -0.5)
    s["down"], s["down_scales"] = _int8_rows(G, H, inter, g, inter ** -0.5)
    s["hidden"] = torch.zeros((G, cap, inter), dtype=torch.bfloat16, device="cuda")
    s["codes"] = torch.zeros((G, cap, inter), dtype=torch.int8, device="cuda")
    s["scales"] = torch.zeros((G, cap), device="cuda")
    s["out"] = torch.zeros((G, cap, H), dtype=dt, device="cuda")
    return s


def _prepare_few(case, seed):
    g = _gen(seed)
    dt = DTYPE[case["dtype"]]
    E, T, k, H, inter = (case[n] for n in ("experts", "tokens", "topk", "hidden", "inter"))
    s = dict(op="few_tokens", workspace=None)
    s["x"] = _randn((T, H), g).to(dt)
    if case["repeats"]:  # ids that come twice in a token, or name no expert
        s["ids"] = torch.randint(-1, E + 1, (T, k), generator=g, device="cuda").to(torch.int32)
        s["ids"][0, 0].clamp_(0, E - 1)
    else:
        order = torch.rand((T, E), generator=g, device="cuda").argsort(1)
        s["ids"] = order[:, :k].to(torch.int32).contiguous()
    s["weights"] = torch.softmax(_randn((T, k), g), -1) if case["weighted"] else None
    if case["weights"] == "fp8":
        s["gate_up"], s["gate_up_scales"] = _fp8_blocks(E, 2 * inter, H, g)
        s["down"], s["down_scales"] = _fp8_blocks(E, H, inter, g)
    else:
        s["gate_up"], s["gate_up_scales"] = _int8_rows(E, 2 * inter, H, g, H ** -0.5)
        s["down"], s["down_scales"] = _int8_rows(E, H, inter, g, inter ** -0.5)
    s["out"] = torch.zeros((T, H), dtype=dt, device="cuda")
    if own:  # which a serving program keeps
        import combine_route_amd as cra
        s["workspace"] = torch.empty(cra.moe_few_tokens_workspace_bytes(T, k, H, inter),
                                     dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    if case["op"].startswith("block_norm"):
        return _prepare_norm(case, seed)
    if case["op"] == "few_tokens":
        return _prepare_few(case, seed)
    return _prepare_product(case, seed)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _kept(counts, cap):
    """[G, cap, 1] truth values: rows that a group's count reaches."""
    return (torch.arange(cap, device="cuda")[None] < counts[:, None])[..., None]


def _per_row(gate):
    """A gate [H] or [G, H] against rows [G, M, H]."""
    return gate.float() if gate.dim() == 1 else gate.float()[:, None]


def _inverse_rms(v):
    return torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    y, dt = s["y"].float(), s["y"].dtype
    if s["post"] is not None:
        y = y * _inverse_rms(y) * s["post"].float()
    if s["gate"] is not None:
        y = y * _per_row(s["gate"])
    h = s["scale"] * s["residual"].float() + y
    z = h * _inverse_rms(h) * s["pre"].float()
    keep = None if s["counts"] is None else _kept(s["counts"], y.shape[1])

    def masked(v):
        return v if keep is None else torch.where(keep, v, 0)

    r = {"residual": masked(h.to(dt))}
    if s["out"] is not None:
        r["out"] = masked(z.to(dt))
    if s["codes"] is None:
        return r
    b = z.unflatten(-1, (-1, 128)) if s["codes"].dtype == E4M3 else z[..., None, :]
    top = E4M3_MAX if s["codes"].dtype == E4M3 else INT8_MAX
    amax = b.abs().amax(-1, keepdim=True)
    up = amax.clamp_min(TINY)
    scale = torch.where(amax > 0, up / top, 1.0).squeeze(-1)
    codes = (b * (top / up)).flatten(-2)
    if s["codes"].dtype == E4M3:
        r["codes"] = masked(codes.clamp(-top, top).to(E4M3).float()).to(E4M3)
        r["scales"] = masked(scale)
    else:
        r["codes"] = masked(codes.round()).to(dt)
        r["scales"] = masked(scale).squeeze(-1)
    return r


def _plain_norm_backward(s):
    y, h, dh, dt = s["y"].float(), s["h"].float(), s["grad_h"].float(), s["y"].dtype
    keep = 1.0 if s["counts"] is None else _kept(s["counts"], y.shape[1]).float()
    r = {}
    if s["pre"] is not None:
        r2 = _inverse_rms(h)
        n2, go = h * r2, s["grad_out"].float() * keep
        d2 = go * s["pre"].float()
        dh = dh + r2 * (d2 - n2 * (d2 * n2).mean(-1, keepdim=True))
        r["grad_pre"] = (go * n2).sum((0, 1))
    dh = dh * keep
    r["grad_residual"] = (s["scale"] * dh).to(dt)
    n1 = y
    if s["post"] is not None:
        r1 = _inverse_rms(y)
        n1 = y * r1
    if s["gate"] is not None:
        u = n1 * s["post"].float() if s["post"] is not None else n1
        r["grad_gate"] = (dh * u).sum((0, 1) if s["gate"].dim() == 1 else 1)
        dh = dh * _per_row(s["gate"])
    if s["post"] is not None:
        r["grad_post"] = (dh * n1).sum((0, 1))
        d1 = dh * s["post"].float()
        dh = r1 * (d1 - n1 * (d1 * n1).mean(-1, keepdim=True))
    r["grad_y"] = dh.to(dt)
    return r


def _plain_product(a, a_scales, b, b_scales):
    y = torch.bmm(a.float(), b.float().transpose(1, 2).contiguous())
    return y * a_scales[..., None] * b_scales[:, None]


def _plain_gemm(s):
    y = _plain_product(s["a"], s["a_scales"], s["b"], s["b_scales"])
    return torch.where(_kept(s["counts"], y.shape[1]), y, 0).to(s["out"].dtype)


def _plain_mlp(s):
    y = _plain_product(s["a"], s["a_scales"], s["gate_up"], s["gate_up_scales"])
    gate, up = y.chunk(2, -1)
    z = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16).float()
    amax = z.abs().amax(-1, keepdim=True)
    top = amax.clamp_min(TINY)
    scales = torch.where(amax > 0, top / INT8_MAX, 1.0).squeeze(-1)
    y = _plain_product((z * (INT8_MAX / top)).round(), scales, s["down"], s["down_scales"])
    return torch.where(_kept(s["counts"], y.shape[1]), y, 0).to(s["out"].dtype)


def _widened(codes, scales):
    """Weights [G, N, K] in 32 bits."""
    if codes.dtype == torch.int8:
        return codes.float() * scales[..., None]
    G, n, k = codes.shape
    w = codes.float().view(G, n // 128, 128, k // 128, 128) * scales[:, :, None, :, None]
    return w.view(G, n, k)


def _plain_few(s):
    x, ids = s["x"].float(), s["ids"].long()
    T, k = ids.shape
    E, inter = s["gate_up"].shape[0], s["down"].shape[2]
    slot = torch.arange(k, device="cuda")
    same = ids[:, :, None] == ids[:, None, :]
    valid = (ids >= 0) & (ids < E)
    lead = valid & (torch.where(same, slot, k).amin(-1) == slot)  # an expert's first slot
    c = torch.ones_like(ids, dtype=torch.float32)
    if s["weights"] is not None:
        c = (same * s["weights"][:, None, :]).sum(-1)
    c = torch.where(lead, c, 0.0)
    at = torch.where(valid, ids, 0)

    def silu_up(y):
        return y[..., :inter] / (1.0 + torch.exp(-y[..., :inter])) * y[..., inter:]

    if T * k <= E:  # a pair's weights each
        def picked(w):
            return w.view(torch.uint8)[at.view(-1)].view(w.dtype)

        pick = at.view(-1)
        gate_up = _widened(picked(s["gate_up"]), s["gate_up_scales"][pick])
        rows = x.repeat_interleave(k, 0)[:, :, None]
        z = silu_up(torch.bmm(gate_up, rows).squeeze(-1))
        del gate_up
        y = torch.bmm(_widened(picked(s["down"]), s["down_scales"][pick]), z[:, :, None])
        out = (y.view(T, k, -1) * c[..., None]).sum(1)
    else:           # every token through every expert
        gate_up = _widened(s["gate_up"], s["gate_up_scales"])
        z = silu_up((gate_up.view(-1, x.shape[1]) @ x.t().contiguous())
                    .view(E, 2 * inter, T).transpose(1, 2))
        del gate_up
        coef = torch.zeros((T, E), device="cuda").scatter_add_(1, at, c)
        z = (z * coef.t()[..., None]).transpose(1, 2).contiguous()
        out = torch.bmm(_widened(s["down"], s["down_scales"]), z).sum(0).t()
    return out.to(s["out"].dtype)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own_norm(s):
    import combine_route_amd as cra
    cra.moe_block_norm(s["y"], s["residual"], s["pre"], EPS, out=s["out"],
                       residual_out=s["residual_out"], post_weight=s["post"], gate=s["gate"],
                       residual_scale=s["scale"], codes=s["codes"], scales=s["scales"],
                       counts=s["counts"])
    r = {"residual": s["residual_out"]}
    if s["out"] is not None:
        r["out"] = s["out"]
    if s["codes"] is not None:
        r["codes"] = s["codes"] if s["codes"].dtype == E4M3 else s["codes"].to(s["y"].dtype)
        r["scales"] = s["scales"]
    return r


def _own_norm_backward(s):
    import combine_route_amd as cra
    cra.moe_block_norm_backward(s["y"], s["h"], EPS, s["grad_y"], grad_out=s["grad_out"],
                                grad_h=s["grad_h"], grad_residual=s["grad_residual"],
                                pre_weight=s["pre"], post_weight=s["post"], gate=s["gate"],
                                residual_scale=s["scale"], grad_pre_weight=s["grad_pre"],
                                grad_post_weight=s["grad_post"], grad_gate=s["grad_gate"],
                                counts=s["counts"], workspace=s["workspace"])
    names = ("grad_y", "grad_residual", "grad_pre", "grad_post", "grad_gate")
    return {name: s[name] for name in names if s[name] is not None}


def _own_gemm(s):
    import combine_route_amd as cra
    cra.moe_grouped_gemm_int8(s["a"], s["a_scales"], s["b"], s["b_scales"], s["out"],
                              counts=s["counts"])
    return s["out"]


def _own_mlp(s):
    import combine_route_amd as cra
    cra.moe_grouped_gemm_int8_swiglu(s["a"], s["a_scales"], s["gate_up"], s["gate_up_scales"],
                                     s["hidden"], counts=s["counts"])
    cra.moe_quantize_int8(s["hidden"], s["codes"], s["scales"], counts=s["counts"])
    cra.moe_grouped_gemm_int8(s["codes"], s["scales"], s["down"], s["down_scales"], s["out"],
                              counts=s["counts"])
    return s["out"]


def _own_few(s):
    import combine_route_amd as cra
    cra.moe_few_tokens(s["x"], s["ids"], s["weights"], s["gate_up"], s["gate_up_scales"],
                       s["down"], s["down_scales"], s["out"], workspace=s["workspace"])
    return s["out"]


def run(s):
    if own:
        return {"block_norm": _own_norm, "block_norm_backward": _own_norm_backward,
                "gemm_int8": _own_gemm, "mlp_int8": _own_mlp, "few_tokens": _own_few}[s["op"]](s)
    return {"block_norm": _plain_norm, "block_norm_backward": _plain_norm_backward,
            "gemm_int8": _plain_gemm, "mlp_int8": _plain_mlp, "few_tokens": _plain_few}[s["op"]](s)


# ---------------------------------------------------------------------------
# work and definition
# ---------------------------------------------------------------------------

def work(case):
    if case["op"].startswith("block_norm"):
        H = case["hidden"]
        rows = case["groups"] * case["rows"] * (0.5 if case["ragged"] else 1.0)
        if case["op"] == "block_norm":
            row = H * (6 + 2 * case["out"] + bool(case["quant"]))
            row += {None: 0, "fp8": H // 32, "int8": 4}[case["quant"]]
            return {"bytes": rows * row + 6 * H, "flops": rows * H * 15}
        row = H * (10 + 2 * case["pre"])
        return {"bytes": rows * row + 18 * H, "flops": rows * H * 30}
    if case["op"] in ("gemm_int8", "mlp_int8"):
        p = _popularity(case["groups"], case["skew"])
        hit = sum(1.0 - (1.0 - v) ** case["pairs"] for v in p)
        rows = sum(min(case["cap"], v * case["pairs"]) for v in p)
        if case["op"] == "gemm_int8":
            n, k = case["n"], case["k"]
            return {"bytes": rows * (k + 4 + 2 * n) + hit * n * (k + 4), "flops": 2.0 * rows * n * k}
        H, inter = case["hidden"], case["inter"]
        return {"bytes": rows * (H + 4 + 2 * H) + hit * (3 * inter * H + 4 * (2 * inter + H)),
                "flops": 6.0 * rows * inter * H}
    E, T, k, H, inter = (case[n] for n in ("experts", "tokens", "topk", "hidden", "inter"))
    if case["repeats"]:
        hit = E * (1.0 - (1.0 - 1.0 / (E + 2)) ** (T * k))
        pairs = T * E * (1.0 - (1.0 - 1.0 / (E + 2)) ** k)
    else:
        hit = E * (1.0 - (1.0 - k / E) ** T)
        pairs = T * k
    return {"bytes": hit * 3.0 * inter * H + 4.0 * T * H + 8.0 * T * k,
            "flops": 6.0 * pairs * inter * H}


def _exact_norm(case, seed):
    s = _prepare_norm(case, seed)
    G, M, H = s["y"].shape
    kind = case["quant"]
    r = {"residual": torch.zeros((G, M, H), dtype=torch.float64, device="cuda")}
    for name in ("out", "codes"):
        if s[name] is not None:
            r[name] = torch.zeros_like(r["residual"])
    if kind:
        r["scales"] = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
    for g in range(G):
        m = M if s["counts"] is None else int(s["counts"][g])
        v = s["y"][g, :m].double()
        if s["post"] is not None:
            v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / H + EPS) * s["post"].double()
        if s["gate"] is not None:
            v = v * (s["gate"] if s["gate"].dim() == 1 else s["gate"][g]).double()
        v = v + s["residual"][g, :m].double() * s["scale"]
        r["residual"][g, :m] = v
        v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / H + EPS) * s["pre"].double()
        if "out" in r:
            r["out"][g, :m] = v
        if kind:
            n, top = (128, E4M3_MAX) if kind == "fp8" else (H, INT8_MAX)
            most = v.abs().reshape(m, H // n, n).max(-1).values
            unit = (torch.maximum(most, torch.full_like(most, TINY)) / top)
            unit = unit.masked_fill(most == 0, 1.0)
            v = v / unit.repeat_interleave(n, -1)
            r["codes"][g, :m] = v if kind == "fp8" else torch.round(v)
            r["scales"][g, :m] = unit if kind == "fp8" else unit[:, 0]
    return r


def _exact_norm_backward(case, seed):
    s = _prepare_norm(case, seed)
    G, M, H = s["y"].shape

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.float64, device="cuda")

    r = {"grad_y": zeros(G, M, H), "grad_residual": zeros(G, M, H)}
    for name, of in (("grad_pre", "pre"), ("grad_post", "post"), ("grad_gate", "gate")):
        if s[of] is not None:
            r[name] = zeros(*s[of].shape)
    for g in range(G):
        m = M if s["counts"] is None else int(s["counts"][g])
        y, h, d = (s[n][g, :m].double() for n in ("y", "h", "grad_h"))
        if s["pre"] is not None:
            go = s["grad_out"][g, :m].double()
            q = torch.sqrt((h * h).sum(-1, keepdim=True) / H + EPS)
            r["grad_pre"] += (go * h / q).sum(0)
            w = go * s["pre"].double()
            d = d + w / q - h * (w * h).sum(-1, keepdim=True) / (H * q ** 3)
        r["grad_residual"][g, :m] = d * s["scale"]
        gate = 1.0
        q = torch.sqrt((y * y).sum(-1, keepdim=True) / H + EPS) if s["post"] is not None else 1.0
        post = s["post"].double() if s["post"] is not None else 1.0
        if s["gate"] is not None:
            shared = s["gate"].dim() == 1
            gate = (s["gate"] if shared else s["gate"][g]).double()
            into = r["grad_gate"] if shared else r["grad_gate"][g]
            into += (d * y / q * post).sum(0)
        if s["post"] is not None:
            r["grad_post"] += (d * gate * y / q).sum(0)
        w = d * gate * post
        if s["post"] is not None:
            w = w / q - y * (w * y).sum(-1, keepdim=True) / (H * q ** 3)
        r["grad_y"][g, :m] = w
    return r


def _exact_gemm(case, seed):
    s = _prepare_product(case, seed)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for g in range(case["groups"]):
        m = min(case["cap"], int(s["counts"][g]))
        if m:
            y = s["a"][g, :m].double() @ s["b"][g].double().t()
            out[g, :m] = y * torch.outer(s["a_scales"][g, :m].double(), s["b_scales"][g].double())
    return out


def _exact_mlp(case, seed):
    s = _prepare_product(case, seed)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    inter = case["inter"]
    for g in range(case["groups"]):
        m = min(case["cap"], int(s["counts"][g]))
        if not m:
            continue
        x = s["a"][g, :m].double() * s["a_scales"][g, :m, None].double()
        w = s["gate_up"][g].double() * s["gate_up_scales"][g, :, None].double()
        gate, up = x @ w[:inter].t(), x @ w[inter:].t()
        z = (gate * torch.sigmoid(gate) * up).to(torch.bfloat16).double()
        most = z.abs().max(-1, keepdim=True).values
        unit = torch.maximum(most, torch.full_like(most, TINY)) / INT8_MAX
        z = torch.round(z / unit) * unit
        out[g, :m] = z @ (s["down"][g].double() * s["down_scales"][g, :, None].double()).t()
    return out


def _exact_weights(codes, scales):
    if codes.dtype == torch.int8:
        return codes.double() * scales[:, None].double()
    return codes.double() * scales.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def _exact_few(case, seed):
    s = _prepare_few(case, seed)
    inter = case["inter"]
    x, ids = s["x"].double(), s["ids"].tolist()
    w = [[1.0] * case["topk"]] * case["tokens"] if s["weights"] is None else s["weights"].tolist()
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    tokens = {}
    for t, row in enumerate(ids):
        for e in sorted(set(row)):
            if 0 <= e < case["experts"]:
                c = 1.0 if s["weights"] is None else sum(v for v, i in zip(w[t], row) if i == e)
                tokens.setdefault(e, []).append((t, c))
    for e, pairs in tokens.items():
        at = torch.tensor([t for t, _ in pairs], device="cuda")
        c = torch.tensor([v for _, v in pairs], dtype=torch.float64, device="cuda")
        y = x[at] @ _exact_weights(s["gate_up"][e], s["gate_up_scales"][e]).t()
        z = y[:, :inter] * torch.sigmoid(y[:, :inter]) * y[:, inter:]
        out[at] += c[:, None] * (z @ _exact_weights(s["down"][e], s["down_scales"][e]).t())
    return out


def exact(case, seed):
    return {"block_norm": _exact_norm, "block_norm_backward": _exact_norm_backward,
            "gemm_int8": _exact_gemm, "mlp_int8": _exact_mlp,
            "few_tokens": _exact_few}[case["op"]](case, seed)
