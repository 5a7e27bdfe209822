"""The Python side of the training-step operators without a GPU: streams, devices and threads of their handles,
against a stand-in for torch's streams and for the C entry points."""
import types

import pytest

import counted_notify_sync_gb300 as cns
from counted_notify_sync_gb300 import _native


class Stream:
    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def wait_stream(self, other):
        self.log.append(("wait", self.cuda_stream, other.cuda_stream))


class Nothing:
    def __enter__(self):
        return self

    def __exit__(self, *_):
        return False


@pytest.fixture
def enqueued(monkeypatch):
    """What new_step_workspace enqueues, in order, with stream `log.current` as torch's current stream."""
    import torch

    class Log(list):
        current, capturing = 0, False

    log = Log()
    cuda = types.SimpleNamespace(
        device=lambda d: Nothing(), current_stream=lambda *_: Stream(log.current, log),
        default_stream=lambda *_: Stream(0, log), ExternalStream=lambda h, *_: Stream(h, log),
        is_current_stream_capturing=lambda: log.capturing)
    fake = types.SimpleNamespace(cuda=cuda, int32=torch.int32, device=torch.device,
                                 empty=lambda n, dtype, device: torch.empty(n, dtype=dtype))
    monkeypatch.setattr(cns, "_torch", lambda: fake)
    monkeypatch.setattr(_native, "cns_step_workspace_init",
                        lambda ws, n, stream=None: log.append(("zero", _native.stream_handle(stream) or 0)) or 0)
    return log


@pytest.mark.parametrize("current", [0, 0x70])
@pytest.mark.parametrize("given", [None, 0x70, 0x90])
def test_a_workspace_is_zeroed_before_the_streams_that_use_it(enqueued, current, given):
    """Zeroed on the stream that its memory comes from; the default stream and the given one come after that."""
    enqueued.current = current
    cns.new_step_workspace(1 << 20, stream=given)
    assert enqueued[0] == ("zero", current)
    for user in {0, given or 0} - {current}:
        assert ("wait", user, current) in enqueued[1:]


def test_a_captured_workspace_leaves_the_default_stream_alone(enqueued):
    enqueued.current, enqueued.capturing = 0x70, True
    cns.new_step_workspace(1 << 20, stream=0x70)
    assert enqueued == [("zero", 0x70)]
