"""The layer operators together, as a serving layer uses them: residual
addition and RMS norm to FP8 rows, the fused FP8 dispatch, the experts' two
products, and the weighted combine; against the same in 64 bits."""
import pytest
import torch

import combine_route_amd as cra
import moe_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


def blocks(w):
    """E4M3 codes and FP32 scales of w [E, n, k] per 128 x 128 block."""
    E, n, k = w.shape
    v = w.view(E, n // 128, 128, k // 128, 128)
    s = v.abs().amax((2, 4), keepdim=True) / 448
    return (v / s).to(ref.E4M3).view(E, n, k), s.view(E, n // 128, k // 128)


def unblocked(codes, scales):
    return codes.double() * scales.double().repeat_interleave(128, 1).repeat_interleave(128, 2)


def setup(W=2, M=20, H=256, inter=128, E=8, k=3, cap=16, seed=0):
    g = torch.Generator().manual_seed(seed)
    d = dict(W=W, M=M, H=H, E=E, k=k, cap=cap)
    d["x"] = torch.randn((W, M, H), generator=g).to(torch.bfloat16)
    d["residual"] = torch.randn((W, M, H), generator=g).to(torch.bfloat16)
    d["norm_w"] = (1 + 0.1 * torch.randn((H,), generator=g)).to(torch.bfloat16)
    d["ids"] = torch.rand((W, M, E), generator=g).argsort(-1)[..., :k].to(torch.int32).contiguous()
    d["w"] = torch.softmax(torch.randn((W, M, k), generator=g), -1)
    d["gu"], d["gus"] = blocks(torch.randn((E, 2 * inter, H), generator=g) / H ** 0.5)
    d["dn"], d["dns"] = blocks(torch.randn((E, H, inter), generator=g) / inter ** 0.5)
    d["ntok"] = [M, M - 7][:W]
    d["op"] = cra.EpDispatchCombineOp(
        cra.make_config(W, H, M, E // W, k, "fp8", "bf16", scale_dim=H // 128), with_weights=False,
        expert_capacity=cap)
    d["dev"] = {n: v.cuda() for n, v in d.items() if isinstance(v, torch.Tensor)}
    d["counts"] = torch.tensor(d["ntok"], dtype=torch.int32, device="cuda")
    d["codes"] = torch.zeros((W, M, H), dtype=torch.uint8, device="cuda")
    d["scales"] = torch.zeros((W, M, H // 128), device="cuda")
    return d


def layer(d):
    t, op = d["dev"], d["op"]
    cra.moe_rms_norm(t["x"], t["norm_w"], 1e-6, residual=t["residual"],
                     residual_out=d.setdefault("stream", torch.zeros_like(t["x"])),
                     codes=d["codes"], scales=d["scales"], counts=d["counts"])
    px, count, _, _ = op.dispatch_standard_moe(d["codes"], None, d["scales"], t["ids"], d["ntok"])
    y = op.expert_mlp(px, count, t["gu"], t["gus"], t["dn"], t["dns"])
    return op.combine_standard_moe(y, t["w"], t["ids"])


def test_serving_layer():
    d = setup()
    out = layer(d).cpu()
    h, y = ref.rms_norm(d["x"], d["norm_w"], 1e-6, d["residual"])
    rows, _ = ref.packed_rows(d["ids"], d["ntok"], d["E"], d["cap"])
    gu, dn = unblocked(d["gu"], d["gus"]), unblocked(d["dn"], d["dns"])
    inter = gu.shape[1] // 2
    dropped = 0
    for r in range(d["W"]):
        n = d["ntok"][r]
        assert torch.equal(d["stream"][r, :n].cpu().double(), h[r, :n])
        for t in range(n):
            want = torch.zeros(d["H"], dtype=torch.float64)
            for j in range(d["k"]):
                if rows[r, t, j] < 0:
                    dropped += 1
                    continue
                e = int(d["ids"][r, t, j])
                z = gu[e] @ y[r, t]
                z = z[:inter] * torch.sigmoid(z[:inter]) * z[inter:]
                want += float(d["w"][r, t, j]) * (dn[e] @ z)
            # two roundings to E4M3 (half a step 2^-4 each, of random signs: in
            # the 2-norm below it) dominate
            off = (out[r, t].double() - want).norm()
            assert float(off) <= 2 * 2.0 ** -4 * float(want.norm()) + 1e-6
    assert dropped > 0


def test_convert_path_gives_the_same():
    """The two-step dispatch and convert feed the experts the same rows."""
    d = setup(seed=1)
    fused = layer(d).clone()
    t, op = d["dev"], d["op"]
    op2 = cra.EpDispatchCombineOp(op.cfg, expert_capacity=d["cap"])
    out_x, out_w, out_s, out_i, _ = op2.dispatch(d["ntok"], d["codes"], t["ids"], t["w"],
                                                 d["scales"])
    px, count, _, _ = op2.convert_dispatch_output(out_x, out_i, out_s, out_w)
    y = op2.expert_mlp(px, count, t["gu"], t["gus"], t["dn"], t["dns"])
    out, _ = op2.combine(op2.convert_combine_input(y, apply_weights=True))
    for r in range(d["W"]):
        n = d["ntok"][r]
        assert torch.equal(out[r, :n], fused[r, :n])


def test_layer_in_a_graph():
    d = setup(seed=2)
    want = layer(d).clone()
    out = d["op"].combine_out
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(d)
    for _ in range(3):
        out.zero_()
        d["codes"].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for r in range(d["W"]):
            assert torch.equal(out[r, :d["ntok"][r]], want[r, :d["ntok"][r]])


def test_expert_mlp_refuses():
    d = setup()
    t = d["dev"]
    px, count, _, _ = d["op"].dispatch_standard_moe(d["codes"], None, d["scales"], t["ids"])
    with pytest.raises(ValueError, match="gate_up"):
        d["op"].expert_mlp(px, count, t["gu"][:, :128].contiguous(), t["gus"], t["dn"], t["dns"])
    with pytest.raises(ValueError, match="down"):
        d["op"].expert_mlp(px, count, t["gu"], t["gus"], t["dn"][:, :128].contiguous(), t["dns"])
    plain = cra.EpDispatchCombineOp(cra.make_config(2, 256, 20, 4, 3), expert_capacity=16)
    with pytest.raises(ValueError, match="fp8"):
        plain.expert_mlp(px, count, t["gu"], t["gus"], t["dn"], t["dns"])


def test_expert_mlp_on_a_stream_takes_no_memory_still_in_use():
    """New buffers of a call on another stream do not lie over memory whose
    last use is pending on torch's current one."""
    d = setup(seed=4)
    want = layer(d).clone()
    t, op = d["dev"], d["op"]
    px, count, _, _ = op.dispatch_standard_moe(d["codes"], None, d["scales"], t["ids"], d["ntok"])
    hidden, hidden_scales, y = op._expert_state().pop("mlp")[128]
    wants = y.clone()
    sizes = [(v.shape, v.dtype) for v in (hidden, hidden_scales, y)]
    del hidden, hidden_scales, y
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    used = [torch.empty(shape, dtype=dt, device="cuda") for shape, dt in sizes]
    torch.cuda._sleep(20_000_000)
    for v in used:
        v.fill_(1)
    del used, v
    y = op.expert_mlp(px, count, t["gu"], t["gus"], t["dn"], t["dns"], stream=s)
    torch.cuda.synchronize()
    n = count.flatten().tolist()
    for g, c in enumerate(n):
        assert torch.equal(y.view(len(n), -1, d["H"])[g, :c], wants.view(len(n), -1, d["H"])[g, :c])
    out = op.combine_standard_moe(y, t["w"], t["ids"])
    for r in range(d["W"]):
        assert torch.equal(out[r, :d["ntok"][r]], want[r, :d["ntok"][r]])
