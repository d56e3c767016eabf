"""Gradients of the fused dispatch and combine on the GPU: against the
formula in 64 bits, against differences of the forward call, and as a pair
(the dispatch's gradient of the combine's).

Bounds: a row of grad_packed_y is one FP32 product of grad_out and the sum of
at most k weights, rounded once. A dot of grad_weights adds at most H / 64
products a lane in a chain, then 6 levels of a tree over the lanes and at most
16 shares of the row: (H / 64 + 24) half steps of binary32 times the sum of
the products' magnitudes. grad_x adds at most k rows in FP32."""
import pytest
import torch

import combine_route_amd as cra
import moe_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


class Case:
    """A fused dispatch that has run, with its map from the definition."""

    def __init__(self, W, M, H, k, E, cap, dtype, ntok=None, ids="distinct", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.W, self.M, self.H, self.k, self.E, self.cap = W, M, H, k, E, cap
        self.dt = TYPES[dtype]
        self.ntok = [M] * W if ntok is None else ntok
        if ids == "distinct":
            self.ids = torch.rand((W, M, E), generator=g).argsort(-1)[..., :k].to(torch.int32)
        elif ids == "any":  # repeats, and ids that name no expert
            self.ids = torch.randint(-2, E + 2, (W, M, k), generator=g).to(torch.int32)
        else:               # one expert for all
            self.ids = torch.full((W, M, k), int(ids), dtype=torch.int32)
        self.ids = self.ids.contiguous()
        self.rows, self.lead = ref.packed_rows(self.ids, self.ntok, E, cap)
        self.w = torch.rand((W, M, k), generator=g) + 0.1
        self.go = torch.randn((W, M, H), generator=g).to(self.dt)
        self.y = torch.randn((W, E // W, cap, H), generator=g).to(self.dt)
        self.op = cra.EpDispatchCombineOp(cra.make_config(W, H, M, E // W, k, dtype),
                                          with_weights=False, expert_capacity=cap)
        self.x = torch.randn((W, M, H), generator=g).to(self.dt).cuda()
        self.dev_ids = self.ids.cuda()
        self.op.dispatch_standard_moe(self.x, None, None, self.dev_ids, self.ntok)

    def pairs(self):
        """(source rank, token, slot, packed row) of every kept pair."""
        r, t, j = (self.rows >= 0).nonzero(as_tuple=True)
        return r, t, j, self.rows[r, t, j]

    def pair_weights(self):
        same = self.ids[..., :, None] == self.ids[..., None, :]
        return (same * self.w.double()[..., None, :]).sum(-1)

    def combine_backward(self, weighted=True, dots=True, **kw):
        gy = torch.full(self.y.shape, 7.0, dtype=self.dt, device="cuda")
        gw = torch.full(self.w.shape, 7.0, device="cuda") if dots else None
        return self.op.combine_standard_moe_backward(
            self.go.cuda(), self.w.cuda() if weighted else None, self.dev_ids,
            self.y.cuda() if dots else None, grad_packed_y=gy, grad_weights=gw, **kw)

    def check_combine(self, gy, gw, weighted=True):
        r, t, j, p = self.pairs()
        c = self.pair_weights()[r, t, j] if weighted else torch.ones(len(p), dtype=torch.float64)
        gy = gy.cpu().view(-1, self.H)
        ref.close_to(gy[p], c[:, None] * self.go[r, t].double(), self.dt, (self.k + 1) * ref.F32)
        rest = torch.ones(gy.shape[0], dtype=torch.bool)
        rest[p] = False
        assert bool((gy[rest] == 7).all())
        if gw is None:
            return
        prod = self.go[r, t].double() * self.y.view(-1, self.H)[p].double()
        want = torch.zeros(self.w.shape, dtype=torch.float64)
        tol = torch.zeros(self.w.shape, dtype=torch.float64)
        want[r, t, j] = prod.sum(-1)
        tol[r, t, j] = prod.abs().sum(-1) * (self.H / 64 + 24) * ref.F32
        lead = self.lead.clamp_min(0)
        want = torch.where(self.lead >= 0, want.gather(2, lead), 0.0)
        tol = torch.where(self.lead >= 0, tol.gather(2, lead), 0.0)
        for s in range(self.W):
            n = self.ntok[s]
            d = (gw.cpu()[s, :n].double() - want[s, :n]).abs()
            assert bool((d <= tol[s, :n]).all()), float((d - tol[s, :n]).max())
            assert bool((gw[s, n:] == 7).all())

    def check_dispatch(self, gp, gx):
        r, t, j, p = self.pairs()
        want = torch.zeros((self.W, self.M, self.H), dtype=torch.float64)
        size = torch.zeros((self.W, self.M, self.H), dtype=torch.float64)
        v = gp.cpu().view(-1, self.H)[p].double()
        want.index_put_((r, t), v, accumulate=True)
        size.index_put_((r, t), v.abs(), accumulate=True)
        for s in range(self.W):
            n = self.ntok[s]
            ref.close_to(gx.cpu()[s, :n], want[s, :n], self.dt, 0.0,
                         self.k * ref.F32 * size[s, :n])
            assert bool((gx[s, n:] == 7).all())

    def dispatch_backward(self, gp):
        gx = torch.full((self.W, self.M, self.H), 7.0, dtype=self.dt, device="cuda")
        return self.op.dispatch_standard_moe_backward(gp, grad_x=gx)


CASES = [
    dict(W=1, M=1, H=8, k=1, E=1, cap=1),
    dict(W=2, M=5, H=64, k=2, E=8, cap=10),
    dict(W=2, M=70, H=520, k=3, E=6, cap=9),                       # overflows
    dict(W=4, M=33, H=1000, k=8, E=64, cap=40, ntok=[33, 0, 7, 20]),
    dict(W=2, M=40, H=2048, k=64, E=128, cap=30, ids="any"),
    dict(W=3, M=17, H=4096, k=6, E=12, cap=51, ids="any", ntok=[17, 1, 0]),
    dict(W=2, M=64, H=7168, k=8, E=32, cap=128),
    dict(W=2, M=9, H=16384, k=4, E=8, cap=18),
    dict(W=1, M=3, H=36864, k=2, E=4, cap=3),                      # more than one pass of a wave
    dict(W=2, M=20, H=256, k=4, E=4, cap=7, ids=2),                # one expert, most dropped
    dict(W=2, M=20, H=256, k=4, E=4, cap=7, ids=99),               # no expert at all
    dict(W=2, M=20, H=256, k=4, E=4, cap=7, ntok=[0, 0]),          # no token
    dict(W=8, M=2100, H=64, k=2, E=16, cap=5000),                  # a large call's geometry
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_against_the_formula(case, dtype):
    c = Case(dtype=dtype, **case)
    c.check_combine(*c.combine_backward())
    c.check_combine(*c.combine_backward(dots=False))
    c.check_combine(*c.combine_backward(weighted=False, dots=False), weighted=False)
    gp = torch.randn(c.y.shape, generator=torch.Generator().manual_seed(3)).to(c.dt)
    # rows no pair was given are not read
    mask = torch.zeros(c.E * c.cap, dtype=torch.bool)
    mask[c.pairs()[3]] = True
    gp.view(-1, c.H)[~mask] = float("nan")
    c.check_dispatch(gp, c.dispatch_backward(gp.cuda()))


@pytest.mark.parametrize("ids", ["distinct", "any"])
def test_against_differences_of_the_forward(ids):
    """Small whole numbers: every product and sum of the forward is exact, so
    the loss <grad_out, combine(y, w)> moves by exactly the gradient."""
    c = Case(2, 6, 64, 4, 6, 5, "fp16", ids=ids, seed=5)
    g = torch.Generator().manual_seed(6)
    c.go = torch.randint(-2, 3, c.go.shape, generator=g).to(c.dt)
    c.y = torch.randint(-3, 4, c.y.shape, generator=g).to(c.dt)
    c.w = 2.0 ** torch.randint(-1, 2, c.w.shape, generator=g).float()

    def loss(y, w):
        out = c.op.combine_standard_moe(y.cuda(), w.cuda(), c.dev_ids)
        return float((out.double().cpu() * c.go.double()).sum())

    gy, gw = c.combine_backward()
    base = loss(c.y, c.w)
    pairs = c.pairs()[3].tolist()
    for i in range(0, len(pairs), 3):
        y = c.y.clone()
        y.view(-1, c.H)[pairs[i], i % c.H] += 1
        assert loss(y, c.w) - base == float(gy.view(-1, c.H)[pairs[i], i % c.H])
    for i in range(0, c.w.numel(), 5):
        w = c.w.clone()
        w.view(-1)[i] += 0.5
        assert 2 * (loss(c.y, w) - base) == float(gw.view(-1)[i])
    # the dispatch copies a token to its rows: moving one element of the
    # token moves every copy
    gp = torch.randint(-3, 4, c.y.shape, generator=g).to(c.dt).cuda()
    kept = torch.zeros((c.E * c.cap, 1), device="cuda")
    kept[c.pairs()[3].cuda()] = 1

    def packed_loss(x):
        px = c.op.dispatch_standard_moe(x, None, None, c.dev_ids, c.ntok)[0]
        return float((torch.where(kept > 0, px.view(-1, c.H), 0).double() *
                      gp.view(-1, c.H).double()).sum())

    x = torch.randint(-3, 4, c.x.shape, generator=g).to(c.dt).cuda()
    gx = c.dispatch_backward(gp)
    base = packed_loss(x)
    for i in range(0, x.numel(), 61):
        moved = x.clone()
        moved.view(-1)[i] += 1
        assert packed_loss(moved) - base == float(gx.view(-1)[i])


def test_layer_backward_matches_torch():
    """One layer step: dispatch, an expert per row (a matrix each), weighted
    combine, and back, against torch's own gradient of the same in 64 bits."""
    c = Case(2, 24, 128, 3, 8, 30, "bf16", seed=8)
    g = torch.Generator().manual_seed(9)
    mats = (torch.randn((c.E, c.H, c.H), generator=g) / c.H ** 0.5).double()
    px, count, _, _ = c.op.dispatch_standard_moe(c.x, None, None, c.dev_ids, c.ntok)
    rows = torch.arange(c.cap)[None] < count.cpu().view(-1)[:, None]
    xe = torch.where(rows[..., None], px.cpu().view(c.E, c.cap, c.H).double(), 0)
    y = torch.matmul(xe, mats).to(c.dt)
    gy, gw = c.op.combine_standard_moe_backward(c.go.cuda(), c.w.cuda(), c.dev_ids,
                                                y.view(c.y.shape).cuda())
    gp = torch.matmul(gy.cpu().view(c.E, c.cap, c.H).double(), mats.transpose(1, 2)).to(c.dt)
    gx = c.op.dispatch_standard_moe_backward(gp.view(c.y.shape).cuda())

    x64 = c.x.cpu().double().requires_grad_()
    w64 = c.w.double().requires_grad_()
    out = torch.zeros((c.W, c.M, c.H), dtype=torch.float64)
    for j in range(c.k):
        out = out + w64[..., j, None] * torch.matmul(x64[..., None, :],
                                                     mats[c.ids[..., j].long()])[..., 0, :]
    out.backward(c.go.double())
    # three roundings to bf16 on the way (y, grad rows, grad of x), each half a
    # step of values of about the result's size
    for got, want in ((gx, x64.grad), (gw, w64.grad)):
        d = got.cpu().double() - want
        assert float(d.norm() / want.norm()) < 3 * ref.half_step(torch.bfloat16)


def test_refusals():
    c = Case(2, 5, 64, 2, 8, 10, "bf16")
    go, w, y = c.go.cuda(), c.w.cuda(), c.y.cuda()
    fresh = cra.EpDispatchCombineOp(c.op.cfg, expert_capacity=10)
    with pytest.raises(cra.EpError, match="before any"):
        fresh.combine_standard_moe_backward(go, w, c.dev_ids, y)
    fresh._expert_state()
    with pytest.raises(cra.EpError, match="before any"):
        fresh.dispatch_standard_moe_backward(y)
    with pytest.raises(cra.EpError, match="grad_weights needs"):
        c.op.combine_standard_moe_backward(go, None, c.dev_ids, y)
    with pytest.raises(ValueError, match="grad_out"):
        c.op.combine_standard_moe_backward(go.half(), w, c.dev_ids, y)
    with pytest.raises(ValueError, match="indices"):
        c.op.combine_standard_moe_backward(go, w, c.dev_ids.long(), y)
    with pytest.raises(ValueError, match="packed_y"):
        c.op.combine_standard_moe_backward(go, w, c.dev_ids, y[..., :32].contiguous())
    with pytest.raises(ValueError, match="grad_x"):
        c.op.dispatch_standard_moe_backward(y, grad_x=go.float())
    wire = cra.EpDispatchCombineOp(cra.make_config(2, 128, 5, 4, 2, combine_wire="fp8_block128"),
                                   expert_capacity=10)
    x = torch.zeros((2, 5, 128), dtype=torch.bfloat16, device="cuda")
    wire.dispatch_standard_moe(x, None, None, c.dev_ids)
    with pytest.raises(cra.EpError, match="combine_wire"):
        wire.dispatch_standard_moe_backward(torch.zeros((2, 4, 10, 128), dtype=torch.bfloat16,
                                                        device="cuda"))


def test_a_conversion_ends_the_map():
    c = Case(2, 5, 64, 2, 8, 10, "bf16")
    c.op.dispatch(c.ntok, c.x, c.dev_ids)
    c.op.convert_dispatch_output(c.op.out_x, c.op.out_indices)
    with pytest.raises(cra.EpError, match="convert_dispatch_output came since"):
        c.dispatch_backward(c.y.cuda())


def test_graph_and_stream():
    c = Case(2, 50, 1024, 4, 16, 30, "bf16")
    want = c.combine_backward()
    gp = c.y.cuda()
    want_x = c.dispatch_backward(gp)
    go, w, y = c.go.cuda(), c.w.cuda(), c.y.cuda()
    got = [torch.full_like(v, 7.0) for v in want]
    got_x = torch.full_like(want_x, 7.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.op.combine_standard_moe_backward(go, w, c.dev_ids, y, *got)
        c.op.dispatch_standard_moe_backward(gp, grad_x=got_x)
    for _ in range(3):
        for v in got + [got_x]:
            v.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got + [got_x], list(want) + [want_x]):
            assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gy, gw = c.op.combine_standard_moe_backward(go, w, c.dev_ids, y, stream=s)
    gx = c.op.dispatch_standard_moe_backward(gp, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(gx, want_x)  # every token is there
    assert torch.equal(gw, want[1])
    written = torch.zeros((c.E * c.cap, 1), dtype=torch.bool, device="cuda")
    written[c.pairs()[3].cuda()] = True
    assert torch.equal(gy.view(-1, c.H), torch.where(written, want[0].view(-1, c.H), 0))


@pytest.mark.parametrize("ids", ["distinct", "any"])
def test_few_tokens_give_the_bits_of_many(ids):
    """A call of few tokens takes their slots in groups, one of many takes them
    together: the first tokens' results (their rows are the experts' first)
    are the same bits."""
    many = Case(1, 2100, 1000, 64, 80, 2100, "bf16", ids=ids, seed=7)
    gy, gw = many.combine_backward()
    for n in (1, 3, 40):
        few = Case(1, 2100, 1000, 64, 80, 2100, "bf16", ntok=[n], ids=ids, seed=7)
        assert torch.equal(few.ids, many.ids) and torch.equal(few.y, many.y)
        fy, fw = few.combine_backward()
        assert torch.equal(fw[:, :n], gw[:, :n]) and bool((fw[:, n:] == 7).all())
        p = few.pairs()[3]
        assert torch.equal(few.rows[:, :n], many.rows[:, :n])
        assert torch.equal(fy.view(-1, few.H)[p], gy.view(-1, few.H)[p])
