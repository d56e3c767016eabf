"""Plain 64-bit forms of the operators of include/moe_block.h and the bounds
their results are held to. Written from the definitions; no library code."""
import torch

from moe_reference import F32, TINY

INT8_MAX = 127.0


def rms_half_steps(H):
    """Bound of the relative error of r = 1 / sqrt(mean + eps) in half steps
    of binary32: H nonnegative squares added in chains of 8, a tree of 6
    levels and a chain of at most H / 512 + 4 chunk sums; the square root
    halves that sum's error, the roots and the division add 3, the product
    with the value and its weight 2."""
    return (16 + H / 512 + 4) / 2 + 5


def int8_close(codes, scales, want, rel32, abs32=0.0):
    """codes [..., H] (int8) and scales [...] stand for want: the scale is the
    row maximum over 127 (1 for zeros), each code within half of the value over
    the scale. abs32: FP32 error of the values on top of rel32 relative."""
    want = want.double()
    e = torch.as_tensor(abs32, dtype=torch.float64, device=want.device).expand(want.shape)
    amax = want.abs().amax(-1)
    u = amax.clamp_min(TINY)
    s = torch.where(amax > 0, u / INT8_MAX, 1.0)
    emax = e.amax(-1)
    tol = (rel32 + 4 * F32) * s + emax / INT8_MAX
    bad = ~((scales.double() - s).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((scales.double() - s).abs() / s)[bad].max()))
    v = want * (INT8_MAX / u)[..., None]
    slack = (2 * rel32 + 8 * F32) * v.abs() + e * (INT8_MAX / u)[..., None] + \
        v.abs() * (emax / u)[..., None]
    bad = ~((codes.double() - v).abs() <= 0.5 + slack)
    assert not bad.any(), (int(bad.sum()), float((codes.double() - v)[bad].abs().max()))


def per_row(gate, y):
    """gate [H] or [G, H] against rows [G, ..., H], in 64 bits."""
    g = gate.double()
    return g if g.dim() == 1 else g.view(g.shape[0], *[1] * (y.dim() - 2), g.shape[1])


def block_norm(y, residual, post, gate, scale, pre, eps):
    """h and out in 64 bits, and bounds of what FP32 work puts into them."""
    H = y.shape[-1]
    n = rms_half_steps(H) * F32
    u = y.double()
    if post is not None:
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * post.double()
    if gate is not None:
        u = u * per_row(gate, y)
    res = scale * residual.double()
    h = res + u
    # the factors' error, the gate's product, the scale's own rounding to
    # binary32, and the sum's one rounding
    h_err = (n + F32) * u.abs() + F32 * res.abs() + F32 * h.abs()
    if pre is None:
        return h, h_err, None, None
    ms = (h * h).mean(-1, keepdim=True)
    out = h / torch.sqrt(ms + eps) * pre.double()
    # what h's error does to the root of its mean square, relative to it
    shift = torch.sqrt((h_err * h_err).mean(-1, keepdim=True) / (ms + eps))
    out_err = (n + 2 * shift) * out.abs() + h_err / torch.sqrt(ms + eps) * pre.double().abs()
    return h, h_err, out, out_err


def block_norm_backward(y, h, gh, go, post, gate, scale, pre, eps, keep):
    """Gradients in 64 bits, each with a bound of its FP32 error: (grad_y,
    grad_residual, grad_post, grad_gate, grad_pre) -> (value, bound). keep:
    truth values [..., 1] of the rows that count. A mean over a row is of
    products of at most 5 factors, added in chains of 8 elements a chunk and
    at most 4 chunks, a tree of 6 levels and a chain of 16 waves: K half steps
    of the sum of magnitudes covers it and what is made of it."""
    H = y.shape[-1]
    K = (2 * rms_half_steps(H) + 32 + 6 + 16 + 16) * F32
    keep = keep.double()
    y, go_ = y.double(), torch.zeros_like(y, dtype=torch.float64) if go is None else go.double()
    y, go_ = y * keep, go_ * keep
    d = (torch.zeros_like(y) if gh is None else gh.double()) * keep
    d_abs = d.abs()
    n2 = torch.zeros_like(y)
    if go is not None:
        hh = h.double()
        r2 = 1 / torch.sqrt((hh * hh).mean(-1, keepdim=True) + eps)
        n2 = hh * r2 * keep
        d2 = go_ * pre.double()
        d = d + r2 * (d2 - n2 * (d2 * n2).mean(-1, keepdim=True))
        d_abs = d_abs + r2 * (d2.abs() + n2.abs() * (d2 * n2).abs().mean(-1, keepdim=True))
    rows = int(keep.sum())
    S = (rows + 64) * F32 + K

    def over_rows(v, a, gate_like=False):
        dims = tuple(range(v.dim() - 1))
        if gate_like and gate.dim() == 2:
            dims = dims[1:]
        return (v.sum(dims), S * a.sum(dims)) if dims else (v, S * a)

    res = {"grad_residual": (scale * d, 2 * K * abs(scale) * d_abs),
           "grad_pre": over_rows(go_ * n2, (go_ * n2).abs())}
    p = post.double() if post is not None else torch.ones(H, dtype=torch.float64, device=y.device)
    r1 = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) if post is not None else 1.0
    n1 = y * r1
    g = per_row(gate, y) if gate is not None else 1.0
    if gate is not None:
        res["grad_gate"] = over_rows(d * n1 * p, d_abs * (n1 * p).abs(), True)
    du, du_abs = d * g, d_abs * (g.abs() if gate is not None else 1.0)
    res["grad_post"] = over_rows(du * n1, du_abs * n1.abs())
    gy, gy_abs = du, du_abs
    if post is not None:
        d1, d1_abs = du * p, du_abs * p.abs()
        gy = r1 * (d1 - n1 * (d1 * n1).mean(-1, keepdim=True))
        gy_abs = r1 * (d1_abs + n1.abs() * (d1_abs * n1.abs()).mean(-1, keepdim=True))
    res["grad_y"] = (gy, 4 * K * gy_abs)
    return res


def weights_of(codes, scales):
    """Weights [E, N, K] in 64 bits: a scale per row (int8) or per 128 x 128."""
    if codes.dtype == torch.int8:
        return codes.double() * scales.double()[..., None]
    s = scales.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    return codes.view(torch.float8_e4m3fn).double() * s


def few_tokens(x, ids, w, gate_up, down):
    """The layer in 64 bits, weights [E, 2 I, H] and [E, H, I], and a bound of
    its FP32 error. A sum of n products in the matrix unit: n half steps of the
    sum of magnitudes, twice as much where it cuts instead of rounding. silu's
    derivative is at most 1.1; exponential, quotient and scales 16 half steps;
    the hidden value as two of bf16 2^-17."""
    T, H = x.shape
    E, inter = down.shape[0], down.shape[2]
    out = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)
    for t in range(T):
        row = ids[t].tolist()
        for e in dict.fromkeys(row):
            if not 0 <= e < E:
                continue
            c = 1.0 if w is None else sum(float(v) for v, i in zip(w[t].tolist(), row) if i == e)
            v = x[t].double()
            g, u = (gate_up[e] @ v).chunk(2)
            ge, ue = (2 * (H + 16) * F32 * (gate_up[e].abs() @ v.abs())).chunk(2)
            s = g * torch.sigmoid(g)
            z = s * u
            ze = 1.1 * ge * u.abs() + s.abs() * ue + ge * ue + (16 * F32 + 2.0 ** -17) * z.abs()
            y = down[e] @ z
            ye = down[e].abs() @ ze + 2 * (inter + 16) * F32 * (down[e].abs() @ (z.abs() + ze))
            out[t] += c * y
            n = ids.shape[1] + 8
            cabs = abs(c) if w is None else sum(abs(float(v)) for v, i in zip(w[t].tolist(), row)
                                                if i == e)
            err[t] += cabs * (ye + n * F32 * (y.abs() + ye))
    return out, err
