"""The streams of the op's layer methods on the GPU: the default stream by its
handle, what close() waits for, and two hidden sizes over one output buffer."""
import pytest
import torch

import combine_route_amd as cra

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


def test_stream_handle_0_is_the_default_stream():
    """Where a call on handle 0 makes its tensors: on the default stream, by
    torch's own account; and the gradients of such a call are those of a call
    on torch's current stream."""
    op = cra.EpDispatchCombineOp(cra.make_config(2, 64, 8, 4, 2), with_weights=False,
                                 expert_capacity=16)
    seen = []

    def make(shape, dtype, device):
        seen.append(torch.cuda.current_stream(device).cuda_stream)
        return torch.empty(shape, dtype=dtype, device=device)

    default = torch.cuda.default_stream().cuda_stream
    assert default == 0
    op._new((4,), torch.int32, default, make)
    side = torch.cuda.Stream()
    op._new((4,), torch.int32, side.cuda_stream, make)
    op._new((4,), torch.int32, side, make)
    assert seen == [default, side.cuda_stream, side.cuda_stream]
    g = torch.Generator().manual_seed(0)
    ids = torch.rand((2, 8, 8), generator=g).argsort(-1)[..., :2].to(torch.int32).cuda()
    x = torch.randn((2, 8, 64), generator=g).to(torch.bfloat16).cuda()
    px, _, _, _ = op.dispatch_standard_moe(x, None, None, ids)
    y = torch.randn(px.shape, generator=g).to(torch.bfloat16).cuda()
    w = torch.rand((2, 8, 2), generator=g).cuda()
    want = op.combine_standard_moe_backward(x, w, ids, y)
    got = op.combine_standard_moe_backward(x, w, ids, y, stream=default)
    gx = op.dispatch_standard_moe_backward(want[0]), op.dispatch_standard_moe_backward(
        want[0], stream=default)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(*gx)


def test_close_waits_for_expert_mlp_on_another_stream():
    op = cra.EpDispatchCombineOp(cra.make_config(2, 256, 8, 2, 2, "fp8", "bf16", scale_dim=2),
                                 with_weights=False, expert_capacity=16)
    codes = torch.zeros((2, 8, 256), dtype=torch.uint8, device="cuda")
    scales = torch.ones((2, 8, 2), device="cuda")
    ids = torch.tensor([0, 3], dtype=torch.int32, device="cuda").expand(2, 8, 2).contiguous()
    px, count, _, _ = op.dispatch_standard_moe(codes, None, scales, ids)
    up, ups = torch.zeros((4, 256, 256), dtype=torch.uint8, device="cuda"), torch.ones(
        (4, 2, 2), device="cuda")
    down, downs = torch.zeros((4, 256, 128), dtype=torch.uint8, device="cuda"), torch.ones(
        (4, 2, 1), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    y = op.expert_mlp(px, count, up, ups, down, downs, stream=side)
    op.close()
    assert side.query()
    n = count.flatten().tolist()
    for g, c in enumerate(n):
        assert bool((y.view(4, 16, 256)[g, :c] == 0).all())


def test_expert_mlp_of_two_hidden_sizes_in_turn():
    """Two expert sizes share the outputs' buffer: each call's outputs are its
    own, eager and as replays of one graph that holds both."""
    op = cra.EpDispatchCombineOp(cra.make_config(2, 256, 8, 2, 2, "fp8", "bf16", scale_dim=2),
                                 with_weights=False, expert_capacity=16)
    g = torch.Generator().manual_seed(3)

    def codes(*shape):
        return torch.randint(0, 0x40, shape, generator=g, dtype=torch.uint8).cuda()

    ids = torch.tensor([1, 2], dtype=torch.int32, device="cuda").expand(2, 8, 2).contiguous()
    px, count, _, _ = op.dispatch_standard_moe(codes(2, 8, 256), None,
                                               torch.ones((2, 8, 2), device="cuda"), ids)
    experts = []
    for inter in (128, 384):
        experts.append((codes(4, 2 * inter, 256), torch.full((4, inter // 64, 2), 2.0 ** -8,
                                                             device="cuda"),
                        codes(4, 256, inter), torch.ones((4, 2, inter // 128), device="cuda")))

    def outputs(y):
        return torch.cat([y.view(4, 16, 256)[e, :c] for e, c in enumerate(rows)])

    rows = count.flatten().tolist()
    want = []
    for e in experts:
        y = op.expert_mlp(px, count, *e)
        want.append(outputs(y).clone())
    assert sum(rows) == 32 and not torch.equal(*want)
    assert op.expert_mlp(px, count, *experts[0]).data_ptr() == y.data_ptr()
    for e, w in zip(experts, want):
        assert torch.equal(outputs(op.expert_mlp(px, count, *e)), w)
    kept = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for e, k in zip(experts, kept):
            k.copy_(outputs(op.expert_mlp(px, count, *e)))
    for _ in range(3):
        for k in kept:
            k.zero_()
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, w in zip(kept, want):
            assert torch.equal(k, w)
