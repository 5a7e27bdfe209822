"""Handles of the training-step operators on the GPU: the streams that they are made and used on."""
import threading

import numpy as np
import pytest

from oracle import steps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cns():
    import torch
    import counted_notify_sync_gb300 as c
    c.build()
    torch.cuda.set_device(0)
    return c


def busy(torch, n=12):
    """Some milliseconds of work on the current stream."""
    a = torch.randn(4096, 4096, device="cuda")
    for _ in range(n):
        a @ a


def test_handles_made_and_used_on_a_side_stream(cns):
    """From memory that held ones, with the default stream busy: the zeroing comes before the first call."""
    import torch
    side = torch.cuda.Stream()
    x, g = torch.randn(3000, 64, device="cuda"), torch.randn(2_000_000, device="cuda")
    need = max(cns.cns_route_workspace_bytes(3000, 64, 4)[1], cns.cns_grad_workspace_bytes(1)[1])
    for given in (None, side):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            ones = [torch.full((need // 4 + 4,), -1, dtype=torch.int32, device="cuda") for _ in range(4)]
            del ones
        side.synchronize()
        busy(torch)
        with torch.cuda.stream(side):
            r = cns.new_route(3000, 64, 4, stream=given)
            cns.run_route(r, x, stream=side)
            clip = cns.new_grad_clip([g], 1.0, outs=[torch.empty_like(g)], stream=given)
            cns.run_grad_clip(clip, stream=side)
        side.synchronize()
        assert cns.syncall_read_workspace(r.workspace, side)[3] == 0
        want = np.argsort(-x.cpu().numpy(), -1, kind="stable")[:, :4]
        assert np.array_equal(r.ids.cpu().numpy(), want)
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip((r.offsets, r.order, r.places), steps.plan(want, 64)))
        assert abs(clip.norm.item() / float(torch.linalg.vector_norm(g.double())) - 1) < 4.1e-6
        # and on the default stream, which comes after
        cns.run_route(r, x, sync=True)
        assert np.array_equal(r.ids.cpu().numpy(), want)
        torch.cuda.synchronize()


def test_a_handle_made_within_a_capture(cns):
    """Its zeroing is part of the graph, on the capturing stream."""
    import torch
    s = torch.cuda.Stream()
    x = torch.randn(500, 32, device="cuda")
    cns.run_route(cns.new_route(500, 32, 4), x, sync=True)         # the kernels are loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        r = cns.new_route(500, 32, 4)
        cns.run_route(r, x, stream=s)
    graph.replay()
    torch.cuda.synchronize()
    want = np.argsort(-x.cpu().numpy(), -1, kind="stable")[:, :4]
    assert np.array_equal(r.ids.cpu().numpy(), want)


def test_threads_with_routings_of_other_sizes(cns):
    """The same kernel with other amounts of shared memory, from four threads: no call is refused."""
    import torch
    fails = []

    def work(experts):
        s = torch.cuda.Stream()
        x = torch.randn(5000, experts, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        r = cns.new_route(5000, experts, 4, stream=s)
        try:
            for _ in range(3000):
                cns.run_route(r, x, stream=s)
        except cns.CnsError as e:
            fails.append((experts, str(e)))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(e,)) for e in (500, 400, 512, 420)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not fails


def test_a_new_gradient_tensor_is_of_the_calls_stream(cns):
    """Not of memory that the current stream has still to write."""
    import torch
    x, dw = torch.randn(3000, 64, device="cuda"), torch.randn(3000, 4, device="cuda")
    r = cns.new_route(3000, 64, 4)
    cns.run_route(r, x, sync=True)
    want = cns.run_route_backward(r, x, dw)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    for current, given in ((torch.cuda.default_stream(), side), (side, None), (side, other), (side, side)):
        torch.cuda.synchronize()
        with torch.cuda.stream(current):
            late = torch.empty_like(x)
            busy(torch)
            late.fill_(7.0)
            del late
            got = cns.run_route_backward(r, x, dw, stream=given)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_gradients_and_norms_in_a_graph(cns):
    """cns_route_backward and cns_grad_norm captured, with the routing and the clipping around them; replays compute
    on what the tensors then hold."""
    import torch
    s = torch.cuda.Stream()
    r = cns.new_route(3000, 96, 6, score=steps.SIGMOID, scale=2.5)
    x, dw = torch.randn(3000, 96, device="cuda"), torch.randn(3000, 6, device="cuda")
    dx, out = torch.empty_like(x), torch.empty_like(x)
    small = torch.randn(40, device="cuda")
    norm, clip = cns.new_grad_clip([dx, small]), cns.new_grad_clip([dx], 0.5, outs=[out])
    cns.run_route_backward(cns.run_route(r, x), x, dw)              # the kernels are loaded
    cns.run_grad_norm(norm)
    cns.run_grad_clip(clip)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cns.run_route(r, x, stream=s)
        cns.run_route_backward(r, x, dw, dlogits=dx, stream=s)
        cns.run_grad_norm(norm, stream=s)
        cns.run_grad_clip(clip, stream=s)
    results = lambda: [t.clone() for t in (r.ids, r.weights, r.order, dx, norm.norm, clip.norm, out)]  # noqa: E731
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        dw.copy_(torch.randn_like(dw))
        small.copy_(torch.randn_like(small))
        for t in (dx, out, norm.norm, clip.norm):
            t.fill_(-7.0)
        graph.replay()
        replayed = results()
        torch.cuda.synchronize()
        for t in (dx, out, norm.norm, clip.norm):
            t.fill_(-7.0)
        cns.run_route(r, x)
        cns.run_route_backward(r, x, dw, dlogits=dx)
        cns.run_grad_norm(norm)
        cns.run_grad_clip(clip)
        assert all(torch.equal(a, b) for a, b in zip(replayed, results()))
        both = torch.cat([dx.reshape(-1), small]).double()
        assert abs(norm.norm.item() / float(torch.linalg.vector_norm(both)) - 1) < 4.1e-6
        assert clip.norm.item() < norm.norm.item()
