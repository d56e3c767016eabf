"""The largest sizes that include/moe_block.h allows in each dimension, calls from
several threads on streams of their own at once, and the INT8 experts on a stream
of their own."""
import threading

import pytest
import torch

import block_reference as ref
import combine_route_amd as cra
from moe_reference import close_to

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(shape, seed, dtype=BF16, scale=1.0):
    return (scale * torch.randn(shape, generator=gen(seed), device="cuda")).to(dtype)


def codes(shape, seed):
    return torch.randint(-127, 128, shape, generator=gen(seed), device="cuda").to(torch.int8)


def layer(E, T, k, H, I, kind, seed, dtype=BF16):
    ids = torch.rand((T, E), generator=gen(seed), device="cuda").argsort(-1)[:, :k]
    s = dict(x=rand((T, H), seed + 1, dtype), ids=ids.to(torch.int32).contiguous(),
             w=torch.rand((T, k), generator=gen(seed + 2), device="cuda"))
    for name, n, cols in (("up", 2 * I, H), ("down", H, I)):
        if kind == "int8":
            s[name] = codes((E, n, cols), seed + 3)
            shape, size = (E, n), 73
        else:
            s[name] = (rand((E, n, cols), seed + 3, torch.float32) * 60).clamp_(-448, 448).to(E4M3)
            shape, size = (E, n // 128, cols // 128), 60
        s[name + "s"] = (0.5 + torch.rand(shape, generator=gen(seed + 4), device="cuda")) * \
            cols ** -0.5 / size
    return s


def few(s, stream=None):
    out = torch.full_like(s["x"], 77.0)
    cra.moe_few_tokens(s["x"], s["ids"], s["w"], s["up"], s["ups"], s["down"], s["downs"], out,
                       stream=stream)
    return out


@pytest.mark.parametrize("E,T,k,H,I", [
    (1, 64, 1, 65536, 128), (1, 1, 1, 65536, 128), (8, 3, 8, 65536, 128), (1, 64, 1, 128, 65536),
    (1, 1, 1, 128, 65536), (4, 5, 4, 128, 65536), (8, 2, 8, 128, 65536), (64, 16, 64, 256, 256)])
@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_few_tokens(E, T, k, H, I, kind):
    s = layer(E, T, k, H, I, kind, T + k)
    out = few(s)
    rows = sorted({0, T // 2, T - 1})
    want, err = ref.few_tokens(s["x"][rows], s["ids"][rows], s["w"][rows],
                               ref.weights_of(s["up"], s["ups"]),
                               ref.weights_of(s["down"], s["downs"]))
    close_to(out[rows], want, BF16, 0.0, err)
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("n", [1 << 20, (1 << 20) - 16])
def test_product_of_the_most_columns(n):
    a, sa = codes((1, 3, 16), 1), rand((1, 3), 2, torch.float32).abs()
    b, sb = codes((1, n, 16), 3), rand((1, n), 4, torch.float32).abs() * 0.01
    out = torch.full((1, 3, n), 77.0, dtype=BF16, device="cuda")
    cra.moe_grouped_gemm_int8(a, sa, b, sb, out)
    sums = (a[0].double() @ b[0].double().t()).float()
    assert torch.equal(out[0], (sa[0][:, None] * (sb[0][None] * sums)).to(BF16))


@pytest.mark.parametrize("G,counted", [(1 << 20, False), (1 << 16, True)])
def test_product_of_the_most_groups(G, counted):
    a, sa = codes((G, 2, 16), 1), rand((G, 2), 2, torch.float32).abs()
    b, sb = codes((G, 8, 16), 3), rand((G, 8), 4, torch.float32).abs() * 0.01
    out = torch.full((G, 2, 8), 77.0, dtype=BF16, device="cuda")
    counts = torch.randint(-1, 4, (G,), generator=gen(5), device="cuda", dtype=torch.int32)
    cra.moe_grouped_gemm_int8(a, sa, b, sb, out, counts=counts if counted else None)
    sums = (a[:, :, None].float() * b[:, None].float()).sum(-1)  # whole numbers below 2^18
    want = (sa[..., None] * (sb[:, None] * sums)).to(BF16)
    if counted:
        there = torch.arange(2, device="cuda")[None, :] < counts[:, None]
        want = torch.where(there[..., None], want, torch.tensor(77.0, dtype=BF16, device="cuda"))
    assert torch.equal(out, want)


def test_two_threads_at_once():
    """Each call from two threads on two streams: the results of one alone."""
    y, res, h, go = (rand((4, 60, 1032), i) for i in range(4))
    w = rand((1032,), 5)
    s = layer(8, 6, 3, 384, 256, "fp8", 7)
    t = layer(40, 30, 4, 144, 80, "int8", 8)
    a, sa = codes((5, 70, 208), 9), rand((5, 70), 10, torch.float32).abs()
    b, sb = codes((5, 272, 208), 11), rand((5, 272), 12, torch.float32).abs() * 0.01

    def norm(stream):
        o = [torch.empty_like(y), torch.empty_like(y),
             torch.empty(y.shape, dtype=torch.int8, device="cuda"),
             torch.empty(y.shape[:2], device="cuda")]
        cra.moe_block_norm(y, res, w, 1e-6, out=o[0], residual_out=o[1], post_weight=w,
                           codes=o[2], scales=o[3], stream=stream)
        return o

    def gradient(stream):
        o = [torch.empty_like(y), torch.empty_like(y)] + [torch.empty(1032, device="cuda")
                                                          for _ in range(3)]
        cra.moe_block_norm_backward(y, h, 1e-6, o[0], grad_out=go, grad_h=go, grad_residual=o[1],
                                    pre_weight=w, post_weight=w, gate=w, grad_pre_weight=o[2],
                                    grad_post_weight=o[3], grad_gate=o[4], stream=stream)
        return o

    def quantize(stream):
        o = [torch.empty(y.shape, dtype=torch.int8, device="cuda"),
             torch.empty(y.shape[:2], device="cuda")]
        cra.moe_quantize_int8(y, o[0], o[1], stream=stream)
        return o

    def rows(stream):
        o = torch.empty((5, 70, 272), dtype=FP16, device="cuda")
        cra.moe_grouped_gemm_int8(a, sa, b, sb, o, stream=stream)
        return [o]

    def swiglu(stream):
        o = torch.empty((5, 70, 136), dtype=BF16, device="cuda")
        cra.moe_grouped_gemm_int8_swiglu(a, sa, b, sb, o, stream=stream)
        return [o]

    calls = [norm, gradient, quantize, rows, swiglu, lambda v: [few(s, v)], lambda v: [few(t, v)]]
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    failed, streams = [], [torch.cuda.Stream() for _ in range(2)]

    def work(n):
        try:
            with torch.cuda.stream(streams[n]):
                for i in range(12):
                    for k in range(len(calls)):
                        k = (k + n * 3 + i) % len(calls)
                        got = calls[k](streams[n])
                        streams[n].synchronize()
                        if not all(torch.equal(p, q) for p, q in zip(got, want[k])):
                            failed.append((n, i, k))
        except Exception as e:  # (a thread's own would be lost)
            failed.append((n, repr(e)))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for v in threads:
        v.start()
    for v in threads:
        v.join()
    assert not failed, failed[:5]


@pytest.mark.parametrize("cap", [7, 48])
def test_int8_experts_on_a_stream(cap):
    """All of dispatch, experts and combine on a side stream, with fewer places
    than rows for some experts, is what it is on the current one."""
    W, M, H, Er, K, inter = 2, 24, 256, 4, 2, 96
    cfg = cra.make_config(W, H, M, Er, K, "fp8", "bf16", scale_dim=1)
    x, s = codes((W, M, H), 1), rand((W, M, 1), 2, torch.float32).abs()
    ids = torch.rand((W, M, W * Er), generator=gen(3), device="cuda").argsort(-1)[..., :K]
    ids = ids.to(torch.int32).contiguous()
    w = torch.rand((W, M, K), generator=gen(4), device="cuda")
    up, down = codes((W * Er, 2 * inter, H), 5), codes((W * Er, H, inter), 6)
    ups = rand((W * Er, 2 * inter), 7, torch.float32).abs() * 1e-3
    downs = rand((W * Er, H), 8, torch.float32).abs() * 1e-3
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for stream in (None, side, side.cuda_stream):
        op = cra.EpDispatchCombineOp(cfg, with_weights=False, expert_capacity=cap)
        torch.cuda.synchronize()
        px, count, _, _ = op.dispatch_standard_moe(x.view(torch.uint8), None, s, ids, stream=stream)
        y = op.expert_mlp_int8(px, count, up, ups, down, downs, stream=stream)
        out = op.combine_standard_moe(y, w, ids, stream=stream)
        torch.cuda.synchronize()
        got.append(out.clone())
        assert cap > 7 or bool((count > cap).any())
        op.close()
    assert bool(got[0].isfinite().all()) and bool((got[0] != 0).any())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
