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


def route_handle(monkeypatch, tokens=8, experts=16, top_k=2):
    """What new_route returns, on CPU tensors (whose device index is -1), with device -1 the current one of several."""
    import torch
    monkeypatch.setitem(cns._CODES, torch.float32, _native.CNS_DT_F32)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    r = _native.Route()
    r.ids = torch.zeros((tokens, top_k), dtype=torch.int32)
    r.capacity, r.index, r.others, r.types = tokens, -1, True, (torch.int32, torch.float32)
    r.experts, r.top_k = experts, top_k
    r.backward = _native.RouteGrad(experts=experts, top_k=top_k, score=1, renorm=1, scale=1.0)
    return r


def test_threads_share_a_route_for_their_gradients(monkeypatch):
    """Each call's arguments are its own: while one is in the library, another one fills in its."""
    import torch
    r = route_handle(monkeypatch)
    calls = [dict(logits=torch.zeros(8, 16), dweights=torch.zeros(8, 2), ids=torch.zeros((8, 2), dtype=torch.int32),
                  dlogits=torch.zeros(8, 16)) for _ in range(2)]
    seen = []

    def entry(g):
        if not seen:
            seen.append(None)
            cns.run_route_backward(r, calls[1]["logits"][:4], calls[1]["dweights"], ids=calls[1]["ids"],
                                   dlogits=calls[1]["dlogits"][:4], stream=0x50)   # from another thread, say
        seen.append((g.logits_dev, g.dweights_dev, g.ids_dev, g.dlogits_dev, g.tokens, g.stream))
        return 0

    monkeypatch.setattr(_native, "cns_route_backward", entry)
    cns.run_route_backward(r, calls[0]["logits"], calls[0]["dweights"], ids=calls[0]["ids"], dlogits=calls[0]["dlogits"])
    want = [tuple(c[k].data_ptr() for k in ("logits", "dweights", "ids", "dlogits")) for c in calls]
    assert seen[1:] == [want[1] + (4, 0x50), want[0] + (8, None)]


def test_a_handle_of_another_device_is_refused_before_the_launch(monkeypatch):
    """The library launches on the current device: a handle whose tensors are elsewhere must not get there."""
    import torch
    r = route_handle(monkeypatch)
    g = _native.GradClip()
    g.index, g.others, g.norm = -1, True, torch.zeros(())
    reached = []
    for entry in ("cns_route", "cns_route_backward", "cns_grad_norm", "cns_grad_clip"):
        monkeypatch.setattr(_native, entry, lambda *_, entry=entry: reached.append(entry) or 0)
    x = torch.zeros(8, 16)
    calls = (lambda: cns.run_route(r, x), lambda: cns.run_route_backward(r, x, torch.zeros(8, 2), dlogits=torch.zeros(8, 16)),
             lambda: cns.run_grad_norm(g), lambda: cns.run_grad_clip(g))
    for call in calls:
        call()
    assert len(reached) == 4
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for call in calls:
        with pytest.raises(ValueError, match="current"):
            call()
    assert len(reached) == 4
