"""The block's operators together, as a layer runs them: norm to INT8 rows,
dispatch, INT8 experts, combine, and the norm after the block; and a training
step of the same shape with its gradients."""
import pytest
import torch

import block_reference as ref
import combine_route_amd as cra
from moe_reference import close_to

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
HALF = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


def rand(shape, seed, scale=1.0, shift=0.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (shift + scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def int8_weights(shape, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(-127, 128, shape, generator=g).to(torch.int8).cuda()
    s = (0.5 + torch.rand(shape[:2], generator=g)).cuda() * shape[2] ** -0.5 / 73
    return w, s


W, M, H, ER, K, INTER = 2, 24, 256, 4, 2, 96


def layer_op(cap=48):
    cfg = cra.make_config(W, H, M, ER, K, "fp8", "bf16", scale_dim=1)
    return cra.EpDispatchCombineOp(cfg, with_weights=False, expert_capacity=cap)


def routing(seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand((W, M, W * ER), generator=g).argsort(-1)[..., :K].to(torch.int32).cuda()
    return ids, torch.rand((W, M, K), generator=g).cuda()


def test_int8_layer():
    op = layer_op()
    y, res = rand((W, M, H), 1, 0.5), rand((W, M, H), 2, 2.0)
    post, pre, gate = (rand((H,), 3 + i, 0.1, 1.0) for i in range(3))
    up, ups = int8_weights((W * ER, 2 * INTER, H), 7)
    down, downs = int8_weights((W * ER, H, INTER), 8)
    ids, w = routing(9)
    codes = torch.empty((W, M, H), dtype=torch.int8, device="cuda")
    scales = torch.empty((W, M), device="cuda")
    cra.moe_block_norm(y, res, pre, 1e-6, post_weight=post, gate=gate, residual_scale=0.5,
                       codes=codes, scales=scales)
    px, count, _, _ = op.dispatch_standard_moe(codes.view(torch.uint8), None,
                                               scales.view(W, M, 1), ids)
    out_y = op.expert_mlp_int8(px, count, up, ups, down, downs)
    out = op.combine_standard_moe(out_y, w, ids)
    again = torch.full((W, M, H), 77.0, dtype=BF16, device="cuda")
    stream = res.clone()
    cra.moe_block_norm(out, res, pre, 1e-6, out=again, post_weight=post, gate=gate)
    torch.cuda.synchronize()

    # each stage against the definition, from what the stage before left
    x = codes.double() * scales.double()[..., None]
    h = (x.view(-1, H) @ (up.double() * ups.double()[..., None]).view(-1, H).t()).view(
        W * M, W * ER, 2 * INTER)
    z = (h[..., :INTER] * torch.sigmoid(h[..., :INTER]) * h[..., INTER:])
    # hidden rows off by bf16's half step and half a code's of their largest
    q = z.abs().amax(-1, keepdim=True) / 254 + 2.0 ** -8 * z.abs()
    wd = down.double() * downs.double()[..., None]
    ey = torch.einsum("tei,ehi->teh", z, wd)
    ey_err = torch.einsum("tei,ehi->teh", q * 1.02, wd.abs()) + 2.0 ** -8 * ey.abs()
    c = torch.zeros((W * M, W * ER), dtype=torch.float64, device="cuda").scatter_(
        1, ids.view(-1, K).long(), w.view(-1, K).double())
    want = (c[..., None] * ey).sum(1)
    err = (c[..., None] * ey_err).sum(1) + 3 * 2.0 ** -8 * (c[..., None] * ey).abs().sum(1)
    bad = ~((out.view(-1, H).double() - want).abs() <= err)
    assert not bad.any(), int(bad.sum())
    hh, h_err, n, n_err = ref.block_norm(out, stream, post, gate, 1.0, pre, 1e-6)
    close_to(res, hh, BF16, 0.0, h_err)
    close_to(again, n, BF16, 0.0, n_err)
    op.close()


def test_expert_mlp_int8_is_its_calls_and_refuses():
    op = layer_op(40)
    ids, _ = routing(1)
    x, s = torch.empty((W, M, H), dtype=torch.int8, device="cuda"), torch.empty((W, M),
                                                                                device="cuda")
    cra.moe_quantize_int8(rand((W, M, H), 4), x, s)
    px, count, _, _ = op.dispatch_standard_moe(x.view(torch.uint8), None, s.view(W, M, 1), ids)
    assert px[0].dtype == torch.float8_e4m3fn or px[0].dtype == torch.uint8
    G, cap = W * ER, 40
    rows, rs = px[0].view(torch.int8).view(G, cap, H), px[1].view(torch.float32).view(G, cap)
    for inter in (96, 32):
        up, ups = int8_weights((G, 2 * inter, H), 7)
        down, downs = int8_weights((G, H, inter), 8)
        got = op.expert_mlp_int8(px, count, up, ups, down, downs)
        z = torch.zeros((G, cap, inter), dtype=BF16, device="cuda")
        cra.moe_grouped_gemm_int8_swiglu(rows, rs, up, ups, z, counts=count.view(G))
        q, qs = torch.zeros(z.shape, dtype=torch.int8, device="cuda"), torch.zeros((G, cap),
                                                                                   device="cuda")
        cra.moe_quantize_int8(z, q, qs, counts=count.view(G))
        y = torch.zeros((G, cap, H), dtype=BF16, device="cuda")
        cra.moe_grouped_gemm_int8(q, qs, down, downs, y, counts=count.view(G))
        for g, c in enumerate(count.flatten().tolist()):
            assert torch.equal(got.view(G, cap, H)[g, :c], y[g, :c])
    with pytest.raises(ValueError, match="gate_up"):
        op.expert_mlp_int8(px, count, up[:, :40], ups, down, downs)
    with pytest.raises(ValueError, match="gate_up and down"):
        op.expert_mlp_int8(px, count, up, ups, down[:1], downs)
    with pytest.raises(ValueError, match="must be"):
        op.expert_mlp_int8(px, count, up.view(torch.uint8), ups, down, downs)
    op.close()
    other = cra.EpDispatchCombineOp(cra.make_config(W, H, M, ER, K, "fp8", "bf16", scale_dim=2),
                                    with_weights=False)
    with pytest.raises(ValueError, match="scale_dim 1"):
        other.expert_mlp_int8(px, count, up, ups, down, downs)
    other.close()


def test_int8_layer_in_a_graph():
    """Norm, dispatch, experts and combine captured together: each replay over
    new inputs is the eager layer's, with eager calls in between."""
    op, eager = layer_op(), layer_op()
    y, res = rand((W, M, H), 1, 0.5), rand((W, M, H), 2, 2.0)
    pre = rand((H,), 3, 0.1, 1.0)
    up, ups = int8_weights((W * ER, 2 * INTER, H), 7)
    down, downs = int8_weights((W * ER, H, INTER), 8)
    ids, w = routing(9)

    def layer(op, y, res, ids):
        codes = torch.empty((W, M, H), dtype=torch.int8, device="cuda")
        scales, h = torch.empty((W, M), device="cuda"), torch.empty_like(res)
        cra.moe_block_norm(y, res, pre, 1e-6, residual_out=h, codes=codes, scales=scales)
        px, count, _, _ = op.dispatch_standard_moe(codes.view(torch.uint8), None,
                                                   scales.view(W, M, 1), ids)
        return op.combine_standard_moe(op.expert_mlp_int8(px, count, up, ups, down, downs), w, ids)

    layer(op, y, res, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(op, y, res, ids)
    for seed in range(3):
        y.copy_(rand((W, M, H), 20 + seed, 0.5))
        ids.copy_(routing(30 + seed)[0])
        want = layer(eager, y, res, ids)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    op.close()
    eager.close()


def test_training_step():
    """Gradients of norm, dispatch, a linear expert and combine, against
    automatic differentiation of the plain layer in 64 bits."""
    cfg = cra.make_config(W, H, M, ER, K, "bf16")
    op = cra.EpDispatchCombineOp(cfg, with_weights=False, expert_capacity=W * M)
    y, res = rand((W, M, H), 1, 0.5), rand((W, M, H), 2)
    post, pre = rand((H,), 3, 0.1, 1.0), rand((H,), 4, 0.1, 1.0)
    gate = rand((W, H), 5, 0.2, 0.6)
    ids, w = routing(9)
    e_scale = rand((W * ER, 1, H), 6, 0.3, 1.0, torch.float32)  # the experts: y = scale * x
    n, h = torch.empty_like(y), torch.empty_like(y)
    cra.moe_block_norm(y, res, pre, 1e-6, out=n, residual_out=h, post_weight=post, gate=gate,
                       residual_scale=0.7)
    px, count, _, _ = op.dispatch_standard_moe(n, None, None, ids)
    cap = W * M
    py = (px.view(W * ER, cap, H).float() * e_scale).to(BF16).view(px.shape)
    out = op.combine_standard_moe(py, w, ids)
    go, gh = rand((W, M, H), 11), rand((W, M, H), 12)
    gpy, gw = op.combine_standard_moe_backward(go, w, ids, py)
    gpx = (gpy.view(W * ER, cap, H).float() * e_scale).to(BF16).view(px.shape)
    gn = op.dispatch_standard_moe_backward(gpx)
    g = dict(y=torch.empty_like(y), res=torch.empty_like(y), pre=torch.empty(H, device="cuda"),
             post=torch.empty(H, device="cuda"), gate=torch.empty((W, H), device="cuda"))
    cra.moe_block_norm_backward(y, h, 1e-6, g["y"], grad_out=gn, grad_h=gh,
                                grad_residual=g["res"], pre_weight=pre, post_weight=post, gate=gate,
                                residual_scale=0.7, grad_pre_weight=g["pre"],
                                grad_post_weight=g["post"], grad_gate=g["gate"])
    torch.cuda.synchronize()

    v = {k: t.double().cpu().requires_grad_() for k, t in
         dict(y=y, res=res, pre=pre, post=post, gate=gate, w=w).items()}

    def norm(x):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)

    hh = 0.7 * v["res"] + v["gate"][:, None] * norm(v["y"]) * v["post"]
    nn = norm(hh) * v["pre"]
    s = e_scale.double().cpu()[:, 0][ids.cpu().long()]            # [W, M, K, H]
    oo = (v["w"][..., None] * s * nn[:, :, None]).sum(2)
    ((oo * go.double().cpu()).sum() + (hh * gh.double().cpu()).sum()).backward()
    # bf16 rounds out, the rows between the operators (5 of them, each at most
    # 2^-8 of its norm, twice through a norm's derivative) and the results
    for name, got in dict(g, w=gw).items():
        want = v[name].grad
        off = float((got.double().cpu() - want).norm() / want.norm())
        assert off <= 16 * 2.0 ** -8, (name, off)
    off = float((out.double().cpu() - oo.detach()).norm() / oo.detach().norm())
    assert off <= 8 * 2.0 ** -8
    op.close()
