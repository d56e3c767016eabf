"""The streams of the op's layer methods, without a GPU: torch's stream objects
and the library's calls are stand-ins that record what they are asked for."""
from types import SimpleNamespace as Fields

import pytest
import torch

import combine_route_amd as cra

CPU = torch.device("cpu")


@pytest.fixture
def log(monkeypatch):
    """Streams made and entered, calls and waits, in order."""
    log = []

    class Entered:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            log.append(("enter", self.stream.handle))

        def __exit__(self, *exc):
            log.append(("leave", self.stream.handle))

    def stream(handle):
        return Fields(handle=handle, synchronize=lambda: log.append(("wait", handle)))

    monkeypatch.setattr(torch.cuda, "stream", Entered)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev=None: stream("default"))
    # as torch's: a handle of 0 is taken for none and gives a stream of the pool
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle, device=None: stream(handle or "pool"))
    return log


def test_stream_handle_0_is_the_default_stream(log):
    """New tensors of a call on handle 0 are made on the default stream, where
    the call itself runs, not on one that is unordered with it."""
    op = object.__new__(cra.EpDispatchCombineOp)
    op._ex = op.plan = None
    op.workspace = Fields(device=CPU)
    made = op._zeros((3,), torch.float32, 0)
    assert log == [("enter", "default"), ("leave", "default")] and made.tolist() == [0, 0, 0]
    log.clear()
    op._new((3,), torch.float32, 0x1230)
    assert log == [("enter", 0x1230), ("leave", 0x1230)]
    log.clear()
    op._new((3,), torch.float32, None)
    assert log == []


def mlp_op(monkeypatch, log):
    """An op whose products are stand-ins, over CPU memory."""
    for name in ("moe_grouped_gemm_swiglu", "moe_grouped_gemm"):
        monkeypatch.setattr(cra, name, lambda *a, name=name: log.append((name, a[-1])))
    monkeypatch.setattr(cra, "ep_expert_plan_destroy", lambda plan: log.append(("destroy", plan)))
    op = object.__new__(cra.EpDispatchCombineOp)
    op.cfg = cra.make_config(2, 256, 4, 2, 2, "fp8", "bf16", scale_dim=2)
    op.expert_capacity, op.plan, op._dev_index = 8, None, 0
    op.workspace = Fields(device=CPU)
    op._ex = {"plan": 7}
    return op


def mlp(op, inter=128, stream=0x10):
    G, cap, H = 4, op.expert_capacity, 256
    rows = torch.zeros((2, 2, cap, H), dtype=torch.uint8)
    scales = torch.zeros((2, 2, cap, H // 128 * 4), dtype=torch.uint8)
    up, down = torch.zeros((G, 2 * inter, H), dtype=torch.uint8), torch.zeros((G, H, inter),
                                                                              dtype=torch.uint8)
    return op.expert_mlp((rows, scales), torch.zeros((2, 2), dtype=torch.int32), up, None, down,
                         None, stream=stream)


@pytest.mark.parametrize("streams,last", [([0x10], 0x10), ([0x10, 0x20], 0x20), ([0x10, 0], "default")])
def test_close_waits_for_the_last_expert_mlp(monkeypatch, log, streams, last):
    """Destroying the plan waits for the plan's own last stream; the products
    may be on another one, and their buffers go with the op."""
    op = mlp_op(monkeypatch, log)
    for s in streams:
        mlp(op, stream=s)
    log.clear()
    op.close()
    assert log == [("wait", last), ("destroy", 7)]


def test_close_without_expert_mlp_waits_for_no_stream(monkeypatch, log):
    op = mlp_op(monkeypatch, log)
    op.close()
    assert log == [("destroy", 7)]


def test_close_frees_the_plan_when_the_wait_fails(monkeypatch, log):
    op = mlp_op(monkeypatch, log)
    mlp(op, stream=0x10)
    log.clear()

    def refused(handle, device=None):
        raise RuntimeError("no such stream")

    monkeypatch.setattr(torch.cuda, "ExternalStream", refused)
    with pytest.raises(RuntimeError, match="no such stream"):
        op.close()
    assert log == [("destroy", 7)] and op._ex is None


def test_expert_mlp_has_one_output_buffer(monkeypatch, log):
    """The experts' outputs do not depend on the hidden size: one buffer, for
    every size that is used."""
    op = mlp_op(monkeypatch, log)
    y = mlp(op)
    assert y.shape == (2, 2, 8, 256) and y.dtype == torch.bfloat16
    for inter in (256, 384, 128):
        assert mlp(op, inter).data_ptr() == y.data_ptr()
    hidden = {b[0].shape[2]: b[0].data_ptr() for b in op._ex["mlp"].values()}
    assert sorted(hidden) == [128, 256, 384] and len(set(hidden.values())) == 3
    op.close()
