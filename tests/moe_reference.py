"""Plain 64-bit forms of the layer operators (include/moe.h) and the bounds
their results are held to. Written from the definitions; no library code."""
import torch

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
TINY = 2.0 ** -100
F32 = 2.0 ** -24          # half a step of binary32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close_to(got, want, dtype, rel32, abs32=0.0):
    """got (of dtype) is want (64 bits) rounded once to dtype, after FP32 work
    off by at most rel32 * |want| + abs32: half a step of dtype relative to
    the value that is rounded, or half the smallest step below the normal
    range."""
    got, want = got.double(), want.double()
    fi = torch.finfo(dtype)
    slack = rel32 * want.abs() + abs32
    tol = slack + torch.maximum(fi.eps / 2 * (want.abs() + slack),
                                torch.full_like(want, fi.tiny * fi.eps / 2))
    # overflow past the largest value rounds to infinity in both
    bad = ~(((got - want).abs() <= tol) | (got == want.to(dtype).double()) |
            (got.isnan() & want.isnan()))
    assert not bad.any(), (int(bad.sum()), float((got - want)[bad].abs().max()))


def quantized_close(codes, scales, want, rel32, abs32=0.0):
    """codes [..., H] (E4M3) and scales [..., H / 128] stand for want: the
    scale is the block maximum over 448 (1 for zeros), and each code is
    within half a step (2^-4 relative, 2^-10 below the normal range) of the
    value over the scale. abs32: FP32 error of the values, as [..., H] or a
    number, on top of rel32 relative."""
    b = want.double().unflatten(-1, (-1, 128))
    e = torch.as_tensor(abs32, dtype=torch.float64, device=want.device)
    e = (e.expand(want.shape) if e.dim() == 0 else e).unflatten(-1, (-1, 128))
    amax = b.abs().amax(-1)
    u = amax.clamp_min(TINY)
    s = torch.where(amax > 0, u / E4M3_MAX, 1.0)
    got_s = scales.double()
    tol_s = (rel32 + 4 * F32) * s + e.amax(-1) / E4M3_MAX
    bad = ~((got_s - s).abs() <= tol_s)
    assert not bad.any(), (int(bad.sum()), float(((got_s - s).abs() / s)[bad].max()))
    c = codes.view(E4M3).double().unflatten(-1, (-1, 128))
    v = b * (E4M3_MAX / u)[..., None]
    # error of the scaled value before its rounding: the value's own, and the
    # factor's (the maximum's error moves it by the same relative amount)
    slack = (2 * rel32 + 8 * F32) * v.abs() + e * (E4M3_MAX / u)[..., None] + \
        v.abs() * (e.amax(-1) / u)[..., None]
    tol = slack + torch.maximum(2.0 ** -4 * (v.abs() + slack),
                                torch.full_like(v, 2.0 ** -10))
    bad = ~((c - v).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((c - v)[bad].abs().max()))


def rms_norm(x, weight, eps, residual=None):
    """(h rounded to x's type, y) in 64 bits."""
    h = x.double()
    if residual is not None:
        # one FP32 addition of two bf16 / fp16 values, then one rounding: the
        # stored stream is part of the definition
        h = (x.float() + residual.float()).to(x.dtype).double()
    ms = (h * h).mean(-1, keepdim=True)
    return h, h / torch.sqrt(ms + eps) * weight.double()


def packed_rows(ids, ntok, E, cap):
    """ids [W, M, k] on the CPU -> ([W, M, k] packed row e * cap + p of each
    slot that is its expert's first in the token and within the capacity, else
    -1; [W, M, k] the first slot naming the slot's expert, -1 for none). An
    expert's rows are in source rank, then token order."""
    W, M, k = ids.shape
    rows = torch.full(ids.shape, -1, dtype=torch.int64)
    lead = torch.full(ids.shape, -1, dtype=torch.int64)
    count = [0] * E
    for r in range(W):
        for t in range(ntok[r]):
            seen = {}
            for j, e in enumerate(ids[r, t].tolist()):
                if not 0 <= e < E:
                    continue
                if e not in seen:
                    seen[e] = j
                    if count[e] < cap:
                        rows[r, t, j] = e * cap + count[e]
                    count[e] += 1
                lead[r, t, j] = seen[e]
    return rows, lead
