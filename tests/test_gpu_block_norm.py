"""moe_block_norm and moe_block_norm_backward on the GPU against the plain
64-bit forms; bounds in block_reference.py."""
import pytest
import torch

import block_reference as ref
import combine_route_amd as cra
from moe_reference import close_to, quantized_close

pytestmark = pytest.mark.gpu

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


def rand(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (shift + scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def inputs(G, M, H, dtype, wt, post, gate, seed):
    s = dict(y=rand((G, M, H), dtype, seed, 0.4), residual=rand((G, M, H), dtype, seed + 1, 2.0),
             pre=rand((H,), wt, seed + 2, 0.1, 1.0), post=None, gate=None)
    if post:
        s["post"] = rand((H,), wt, seed + 3, 0.1, 1.0)
    if gate:
        s["gate"] = rand((G, H) if gate == "group" else (H,), wt, seed + 4, 0.3, 0.6)
    return s


def keep_of(counts, G, M):
    c = torch.tensor([M] * G if counts is None else counts)
    return (torch.arange(M)[None] < c[:, None])[..., None].cuda()


def forward(s, quant, scale=0.7, eps=1e-6, counts=None, out=True, stream=None):
    y = s["y"]
    G, M, H = y.shape
    o = dict(residual=torch.full_like(y, 77), out=torch.full_like(y, 77) if out else None,
             codes=None, scales=None)
    if quant == "fp8":
        o["codes"] = torch.full(y.shape, 77, dtype=torch.uint8, device="cuda").view(E4M3)
        o["scales"] = torch.full((G, M, H // 128), 77.0, device="cuda")
    elif quant == "int8":
        o["codes"] = torch.full(y.shape, 77, dtype=torch.int8, device="cuda")
        o["scales"] = torch.full((G, M), 77.0, device="cuda")
    cra.moe_block_norm(y, s["residual"], s["pre"], eps, out=o["out"], residual_out=o["residual"],
                       post_weight=s["post"], gate=s["gate"], residual_scale=scale,
                       codes=o["codes"], scales=o["scales"],
                       counts=None if counts is None else torch.tensor(
                           counts, dtype=torch.int32).cuda(), stream=stream)
    return o


def check_forward(s, o, scale=0.7, eps=1e-6, counts=None):
    y = s["y"]
    G, M, H = y.shape
    n = ref.rms_half_steps(H) * 2.0 ** -24
    h, h_err, want, err = ref.block_norm(y, s["residual"], s["post"], s["gate"], scale, s["pre"],
                                         eps)
    for g in range(G):
        c = M if counts is None else max(0, min(M, counts[g]))
        close_to(o["residual"][g, :c], h[g, :c], y.dtype, 0.0, h_err[g, :c])
        if o["out"] is not None:
            close_to(o["out"][g, :c], want[g, :c], y.dtype, 0.0, err[g, :c])
        if o["codes"] is not None and c:
            check = ref.int8_close if o["codes"].dtype == torch.int8 else quantized_close
            check(o["codes"][g, :c], o["scales"][g, :c], want[g, :c], n, err[g, :c])
        for t in o.values():  # rows past the count, as they were
            if t is not None:
                rest = t[g, c:]
                rest = rest.view(torch.uint8) if rest.dtype == E4M3 else rest
                assert bool((rest == 77).all())


@pytest.mark.parametrize("G,M,H,quant", [
    (1, 1, 8, "int8"), (1, 3, 16, None), (2, 5, 136, "int8"), (3, 7, 128, "fp8"),
    (1, 9, 520, "int8"), (2, 33, 1024, "fp8"), (1, 130, 2056, "int8"), (2, 64, 4096, "fp8"),
    (1, 20, 7168, "int8"), (1, 4, 8200, None), (1, 3, 16384, "fp8"), (1, 2, 32768, "int8"),
    (1, 9000, 256, "fp8"), (1, 9000, 264, "int8"), (4, 2300, 1032, "int8")])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_rows(G, M, H, quant, dtype):
    s = inputs(G, M, H, dtype, dtype if H % 16 else F32, True, "group" if G > 1 else "channel", H)
    check_forward(s, forward(s, quant))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "group"])
@pytest.mark.parametrize("wt", [BF16, F32])
def test_parts(post, gate, wt):
    s = inputs(3, 5, 640, BF16, wt, post, gate, 5)
    for scale in (1.0, 0.0, -1.5):
        check_forward(s, forward(s, "fp8", scale, out=False), scale)
        check_forward(s, forward(s, "int8", scale), scale)


@pytest.mark.parametrize("H", [256, 7168])
@pytest.mark.parametrize("counts", [[0, 3, 9, -2], [9, 1, 0, 40], [0, 0, 0, 0]])
def test_counts(H, counts):
    s = inputs(4, 9, H, BF16, BF16, True, "group", H)
    for quant in ("fp8", "int8"):
        check_forward(s, forward(s, quant, counts=counts), counts=counts)


def test_without_a_second_norm_and_in_place():
    s = inputs(2, 6, 768, FP16, FP16, True, "channel", 9)
    want = forward(s, None)
    res, y = s["residual"].clone(), s["y"].clone()
    cra.moe_block_norm(y, res, None, 1e-6, post_weight=s["post"], gate=s["gate"],
                       residual_scale=0.7)
    assert torch.equal(res, want["residual"])
    res = s["residual"].clone()
    cra.moe_block_norm(y, res, s["pre"], 1e-6, out=y, post_weight=s["post"], gate=s["gate"],
                       residual_scale=0.7)
    assert torch.equal(res, want["residual"]) and torch.equal(y, want["out"])


def test_rows_do_not_depend_on_the_call():
    """The same row alone, among few and among many rows: one wave or many."""
    s = inputs(1, 9000, 2048, BF16, BF16, True, "channel", 11)
    many = forward(s, "int8")
    for lo, hi in ((0, 1), (17, 100), (8000, 9000)):
        part = dict(s, y=s["y"][:, lo:hi].contiguous(),
                    residual=s["residual"][:, lo:hi].contiguous())
        few = forward(part, "int8")
        for k in few:
            assert torch.equal(few[k], many[k][:, lo:hi]), k


def test_rows_without_numbers():
    """Zeros, infinities and NaN: what the formula gives, marked in the scale
    of INT8 rows, and the rows beside them untouched by it."""
    s = inputs(1, 6, 512, BF16, F32, True, None, 13)
    clean = forward(s, "int8")
    s["y"][0, 0] = 0
    s["residual"][0, 0] = 0
    s["residual"][0, 1, 7] = float("nan")
    s["residual"][0, 2, 9] = float("inf")
    s["y"][0, 3, 5] = float("nan")
    o = forward(s, "int8")
    assert bool((o["out"][0, 0] == 0).all() and (o["codes"][0, 0] == 0).all())
    assert float(o["scales"][0, 0]) == 1.0
    for r in (1, 3):
        assert bool(o["out"][0, r].isnan().all()) and bool(o["scales"][0, r].isnan())
    assert bool(o["scales"][0, 2].isnan()) and float(o["residual"][0, 2, 9]) == float("inf")
    assert bool((o["codes"][0, :4] == 0).all())
    for r in (4, 5):
        for k in o:
            assert torch.equal(o[k][0, r], clean[k][0, r])
    check_forward({k: v[:, 4:] if k in ("y", "residual") else v for k, v in s.items()},
                  {k: v[:, 4:] for k, v in o.items()})
    # subnormal rows: quantized as if their largest were 2^-100
    s = inputs(1, 2, 64, BF16, F32, False, None, 1)
    s["y"].zero_()
    s["residual"].copy_(torch.tensor(2.0 ** -120))
    s["pre"].fill_(1.0)
    o = forward(s, "int8", scale=1.0, eps=1.0)
    assert bool((o["codes"] == 0).all())
    assert torch.equal(o["scales"], torch.full_like(o["scales"], 2.0 ** -100 / 127))


@pytest.mark.parametrize("shape", [(0, 128), (3, 0, 128), (0, 5, 128)])
@pytest.mark.parametrize("quant", [None, "fp8", "int8"])
def test_no_rows(shape, quant):
    y = torch.empty(shape, dtype=BF16, device="cuda")
    w = torch.ones(128, dtype=BF16, device="cuda")
    codes = scales = None
    if quant:
        codes = torch.empty(shape, dtype=torch.int8 if quant == "int8" else E4M3, device="cuda")
        scales = torch.empty(shape[:-1] + ((1,) if quant == "fp8" else ()), device="cuda")
    for gate in (None, w, w.repeat(3, 1)) if shape[0] == 3 else (None, w):
        cra.moe_block_norm(y, y, w, 1e-6, out=y, post_weight=w, gate=gate, codes=codes,
                           scales=scales)
        cra.moe_block_norm(y, y, None, 1e-6, post_weight=w, gate=gate)
        cra.moe_block_norm_backward(y, y, 1e-6, y, grad_out=y, grad_h=y, grad_residual=y,
                                    pre_weight=w, post_weight=w, gate=gate)
    if quant == "int8":
        cra.moe_quantize_int8(y, codes, scales)
    torch.cuda.synchronize()


def backward_inputs(G, M, H, dtype, wt, post, gate, pre, gh, seed):
    s = inputs(G, M, H, dtype, wt, post, gate, seed)
    s["h"] = s.pop("residual")
    s["gh"] = rand((G, M, H), dtype, seed + 5) if gh else None
    s["go"] = rand((G, M, H), dtype, seed + 6) if pre else None
    if not pre:
        s["pre"] = None
    return s


def backward(s, scale=0.7, eps=1e-6, counts=None, workspace=None, stream=None, fill=77.0):
    y = s["y"]
    H = y.shape[-1]

    def f32(there, shape):
        return torch.full(shape, fill, device="cuda") if there is not None else None

    o = dict(grad_y=torch.full_like(y, fill), grad_residual=torch.full_like(y, fill),
             grad_pre=f32(s["pre"], (H,)), grad_post=f32(s["post"], (H,)),
             grad_gate=f32(s["gate"], s["gate"].shape if s["gate"] is not None else None))
    cra.moe_block_norm_backward(
        y, s["h"], eps, o["grad_y"], grad_out=s["go"], grad_h=s["gh"],
        grad_residual=o["grad_residual"], pre_weight=s["pre"], post_weight=s["post"],
        gate=s["gate"], residual_scale=scale, grad_pre_weight=o["grad_pre"],
        grad_post_weight=o["grad_post"], grad_gate=o["grad_gate"], workspace=workspace,
        counts=None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda(),
        stream=stream)
    return {k: v for k, v in o.items() if v is not None}


def check_backward(s, o, scale=0.7, eps=1e-6, counts=None):
    y = s["y"]
    G, M, H = y.shape
    keep = keep_of(counts, G, M)
    want = ref.block_norm_backward(y, s["h"], s["gh"], s["go"], s["post"], s["gate"], scale,
                                   s["pre"], eps, keep)
    for k, got in o.items():
        v, err = want[k]
        if k in ("grad_y", "grad_residual"):
            there = keep.expand(y.shape)
            close_to(got[there], v[there], y.dtype, 0.0, err[there])
            assert bool((got[~there] == 77).all()), k
        else:
            bad = ~((got.double() - v).abs() <= err + 2.0 ** -24 * v.abs())
            assert not bad.any(), (k, int(bad.sum()), float((got.double() - v).abs().max()))


@pytest.mark.parametrize("G,M,H", [
    (1, 1, 8), (1, 3, 16), (2, 5, 136), (1, 40, 512), (3, 7, 1032), (1, 300, 2048), (2, 64, 4096),
    (1, 700, 4104), (2, 300, 7168), (1, 5, 8192), (1, 9, 8200), (1, 5, 16384), (1, 3, 16392),
    (1, 2, 32768), (700, 2, 128), (3000, 1, 264)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_gradients(G, M, H, dtype):
    s = backward_inputs(G, M, H, dtype, dtype if H % 16 else F32, True,
                        "group" if G > 1 else "channel", True, True, H)
    check_backward(s, backward(s))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "group"])
@pytest.mark.parametrize("pre,gh", [(True, True), (True, False), (False, True)])
def test_gradients_of_parts(post, gate, pre, gh):
    s = backward_inputs(3, 5, 640, BF16, F32 if gh else BF16, post, gate, pre, gh, 5)
    check_backward(s, backward(s, -1.5), -1.5)
    if not pre:
        check_backward(s, backward(dict(s, h=None), -1.5), -1.5)


@pytest.mark.parametrize("G,M,H", [(4, 9, 256), (4, 600, 1024), (1500, 3, 72)])
@pytest.mark.parametrize("gate", ["channel", "group"])
@pytest.mark.parametrize("which", ["ragged", "none"])
def test_gradients_with_counts(G, M, H, gate, which):
    counts = [0] * G if which == "none" else [
        (0, M + 3, 1, M // 2, -1)[g % 5] for g in range(G)]
    s = backward_inputs(G, M, H, BF16, BF16, True, gate, True, True, H)
    o = backward(s, counts=counts)
    check_backward(s, o, counts=counts)
    if which == "none":
        assert all(bool((o[k] == 0).all()) for k in ("grad_pre", "grad_post", "grad_gate"))


def test_gradients_are_the_forward_differences():
    """Central differences of the 64-bit forward along random directions."""
    s = backward_inputs(2, 3, 64, FP16, F32, True, "group", True, True, 3)
    res = rand((2, 3, 64), FP16, 99)
    base = {k: s[k].double() for k in ("y", "post", "gate", "pre")}
    base["residual"] = res.double()

    def loss(v):
        h, _, out, _ = ref.block_norm(v["y"], v["residual"], v["post"], v["gate"], 0.7, v["pre"],
                                      1e-6)
        return (h * s["gh"].double()).sum() + (out * s["go"].double()).sum(), h

    _, h = loss(base)
    s["h"] = h.to(FP16)
    o = backward(s)
    names = dict(y="grad_y", residual="grad_residual", post="grad_post", gate="grad_gate",
                 pre="grad_pre")
    for name, grad in names.items():
        d = rand(base[name].shape, torch.float64, 7)
        step = 1e-5
        up, _ = loss(dict(base, **{name: base[name] + step * d}))
        down, _ = loss(dict(base, **{name: base[name] - step * d}))
        got, terms = (o[grad].double() * d).sum(), (o[grad].double() * d).abs().sum()
        # fp16's rounding of h and of the results: 2^-11 a term each, h's taken
        # through the norm's derivative at most 3 times
        assert abs(float((up - down) / (2 * step) - got)) <= 4 * 2.0 ** -11 * float(terms) + 1e-6, name


def test_gradients_in_place_and_of_few():
    s = backward_inputs(1, 50, 1024, BF16, BF16, True, "channel", True, True, 21)
    want = backward(s)
    y, h = s["y"].clone(), s["h"].clone()
    cra.moe_block_norm_backward(y, h, 1e-6, y, grad_out=s["go"], grad_h=s["gh"], grad_residual=h,
                                pre_weight=s["pre"], post_weight=s["post"], gate=s["gate"],
                                residual_scale=0.7)
    assert torch.equal(y, want["grad_y"]) and torch.equal(h, want["grad_residual"])
    gh, go = s["gh"].clone(), s["go"].clone()
    only = torch.full((1024,), 5.0, device="cuda")
    cra.moe_block_norm_backward(s["y"], s["h"], 1e-6, gh, grad_out=go, grad_h=gh,
                                grad_residual=go, pre_weight=s["pre"], post_weight=s["post"],
                                gate=s["gate"], residual_scale=0.7, grad_gate=only)
    assert torch.equal(gh, want["grad_y"]) and torch.equal(go, want["grad_residual"])
    assert torch.equal(only, want["grad_gate"])


@pytest.mark.parametrize("H", [1024, 8192, 8200, 16392, 32768])
@pytest.mark.parametrize("rows", [3, 600])
def test_gradients_in_place_of_rows_of_any_size(H, rows):
    """Long rows are read twice, the second time between the stores to the same
    buffers; 600 are several a block."""
    s = backward_inputs(1, rows, H, BF16, BF16, True, "channel", True, True, H)
    want = backward(s)
    for y_of, res_of in (("y", "h"), ("gh", "go"), ("y", "go"), ("gh", "h")):
        b = {k: s[k].clone() for k in ("y", "h", "gh", "go")}
        o = {k: torch.full((H,), 5.0, device="cuda") for k in ("pre", "post", "gate")}
        cra.moe_block_norm_backward(
            b["y"], b["h"], 1e-6, b[y_of], grad_out=b["go"], grad_h=b["gh"],
            grad_residual=b[res_of], pre_weight=s["pre"], post_weight=s["post"], gate=s["gate"],
            residual_scale=0.7, grad_pre_weight=o["pre"], grad_post_weight=o["post"],
            grad_gate=o["gate"])
        assert torch.equal(b[y_of], want["grad_y"]) and torch.equal(b[res_of],
                                                                    want["grad_residual"])
        for k in o:
            assert torch.equal(o[k], want["grad_" + k]), k


@pytest.mark.parametrize("shape", [(0, 64), (3, 0, 64), (0, 5, 64)])
def test_gradients_of_no_rows_are_zeros(shape):
    """As those of rows that are all past their counts."""
    y = torch.empty(shape, dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    side = torch.cuda.Stream()
    for gate in (w, w.repeat(3, 1)) if shape[0] == 3 else (w,):
        for stream in (None, side, side.cuda_stream, 0):
            grads = [torch.full(g.shape, 77.0, device="cuda") for g in (w, w, gate)]
            torch.cuda.synchronize()
            cra.moe_block_norm_backward(y, y, 1e-6, y, grad_out=y, grad_h=y, grad_residual=y,
                                        pre_weight=w, post_weight=w, gate=gate,
                                        grad_pre_weight=grads[0], grad_post_weight=grads[1],
                                        grad_gate=grads[2], stream=stream)
            torch.cuda.synchronize()
            assert all(bool((g == 0).all()) for g in grads)


def test_streams_and_graphs():
    """A side stream, and a graph of both calls replayed over new inputs with
    eager calls on another workspace in between."""
    s = backward_inputs(2, 40, 1024, BF16, BF16, True, "group", True, True, 31)
    s["residual"] = rand((2, 40, 1024), BF16, 77)
    ws = torch.empty(cra.moe_block_norm_backward_workspace_bytes(80, 1024, 2), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        # the call's tensors are made on the stream it runs on
        with torch.cuda.stream(side if stream else torch.cuda.default_stream()):
            o = backward(s, stream=stream)
        torch.cuda.synchronize()
        check_backward(s, o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = forward(s, "int8")
        b = backward(s, workspace=ws)
    for seed in range(3):
        new = backward_inputs(2, 40, 1024, BF16, BF16, True, "group", True, True, 50 + seed)
        for k in ("y", "h", "gh", "go"):
            s[k].copy_(new[k])
        eager = backward(dict(s, **{k: new[k] for k in ("y", "h", "gh", "go")}))
        graph.replay()
        want = forward(s, "int8")
        torch.cuda.synchronize()
        for k in f:
            assert torch.equal(f[k], want[k])
        for k in b:
            assert torch.equal(b[k], eager[k])
