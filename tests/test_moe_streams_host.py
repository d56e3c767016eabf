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
