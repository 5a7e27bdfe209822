"""The operators around a layer of experts as they are used together: the norm with its 8-bit output, the routing, rows to
the experts and back into the residual, and all gradients, against the layer in 64 bits; the same in a CUDA graph; and the
example's block inside torch's autograd."""
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
    torch.backends.cuda.matmul.allow_tf32 = False
    return c


def layer64(x, residual, gain, router, up, ids, eps):
    """The layer with the choice that was made, differentiable, in 64 bits: (y of the norm, output)."""
    import torch
    h = x + residual
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * gain
    there = ids >= 0
    chosen = (y @ router).gather(1, ids.clamp(min=0))
    w = torch.softmax(torch.where(there, chosen, torch.full_like(chosen, -1e300)), -1)      # a number: no row of NaN
    out = h
    for j in range(ids.shape[1]):
        e = torch.einsum("td,tdh->th", y, up[ids[:, j].clamp(min=0)])
        out = out + torch.where(there[:, j:j + 1], w[:, j:j + 1] * e, torch.zeros_like(e))
    return y, out


def test_a_layer_and_its_gradient(cns):
    import torch
    torch.manual_seed(11)
    t, width, e, k, eps = 403, 96, 16, 3, 1e-6
    x, residual = torch.randn(t, width, device="cuda"), torch.randn(t, width, device="cuda")
    gain, router = torch.rand(width, device="cuda") + 0.5, torch.randn(width, e, device="cuda") * width ** -0.5
    up = torch.randn(e, width, width, device="cuda") * width ** -0.5
    norm, route = cns.new_rms_norm(width, eps=eps), cns.new_route(500, e, k)
    h, y, _, _ = cns.run_rms_norm(norm, x, gain, residual=residual)
    logits = y @ router
    logits[7, :] = -float("inf")                      # a padded token
    logits[9, 1:] = -float("inf")                     # one with a single expert left
    cns.run_route(route, logits)
    ids = route.ids[:t].long()
    starts = route.offsets.tolist()
    assert starts[-1] == t * k - 3 - 2
    rows = cns.run_dispatch(route, y)
    out_rows = torch.cat([rows[a:b] @ up[i] for i, (a, b) in enumerate(zip(starts, starts[1:]))])
    out = cns.run_combine(route, out_rows, base=h)
    # the gradient of a weighted sum of the output
    dout = torch.randn_like(out)
    drows_out, dweights = cns.run_combine_backward(route, out_rows, dout)
    drows = torch.cat([drows_out[a:b] @ up[i].t() for i, (a, b) in enumerate(zip(starts, starts[1:]))])
    dup = torch.stack([rows[a:b].t() @ drows_out[a:b] for a, b in zip(starts, starts[1:])])
    dlogits = cns.run_route_backward(route, logits, dweights)
    dy = cns.run_dispatch_backward(route, drows) + dlogits @ router.t()
    dx, dgain = cns.run_rms_norm_backward(norm, h, gain, dy, dh=dout)

    leaves = [v.double().requires_grad_() for v in (x, residual, gain, router, up)]
    y64, out64 = layer64(*leaves, ids, eps)
    (out64 * dout.double()).sum().backward()
    # Each value is a sum of at most 96 * 96 * 3 products of values near 1 along a path of some 500 roundings in 32 bits:
    # 500 * 2^-24 against the largest value of each
    for name, got, want in (("y", y, y64), ("out", out, out64), ("dx", dx, leaves[0].grad), ("dresidual", dx, leaves[1].grad),
                            ("dgain", dgain, leaves[2].grad), ("drouter", y.t() @ dlogits, leaves[3].grad),
                            ("dup", dup, leaves[4].grad)):
        assert (got.double() - want).abs().max() <= 500 * 2.0 ** -24 * want.abs().max(), name
    assert torch.equal(out[7], h[7])


def test_eight_bit_rows_reach_their_experts(cns):
    """The norm's 8-bit output with its scales, sorted by expert: each row stands for the token's normalised row."""
    import torch
    torch.manual_seed(5)
    t, width, e, k = 1000, 520, 32, 4
    x, residual = (torch.randn(t, width, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    gain = torch.rand(width, device="cuda", dtype=torch.bfloat16) + 0.5
    for block, kind in ((128, cns.CNS_SCALE_F32), (32, cns.CNS_SCALE_E8M0), (0, cns.CNS_SCALE_F32)):
        norm, route = cns.new_rms_norm(width, scale_block=block, scale_type=kind), cns.new_route(t, e, k)
        h, y, q, s = cns.run_rms_norm(norm, x, gain, residual=residual)
        cns.run_route(route, torch.randn(t, e, device="cuda"))
        rows, scales = cns.run_dispatch(route, q, scales=s)
        token = torch.div(route.order.long(), k, rounding_mode="floor")
        assert torch.equal(rows.view(torch.uint8), q.view(torch.uint8)[token])
        assert torch.equal(scales.view(torch.uint8), s.view(torch.uint8)[token])
        values = rows.float() * scales.float().repeat_interleave(block or width, 1)[:, :width]
        want = steps.rms_norm(h.double().cpu().numpy(), gain.double().cpu().numpy())[token.cpu().numpy()]
        step = np.abs(want) * 2.0 ** -4 + scales.double().cpu().numpy().max(1, keepdims=True) * 2.0 ** -10
        assert (np.abs(values.double().cpu().numpy() - want) <= step * (1 + 1e-5)).all()


def test_the_layer_in_a_graph(cns):
    """Forward and backward operators captured together; two graphs of the same handles; replays compute on what the
    tensors then hold."""
    import torch
    torch.manual_seed(6)
    t, width, e, k = 700, 256, 16, 2
    s = torch.cuda.Stream()
    x, residual, dout = (torch.randn(t, width, device="cuda") for _ in range(3))
    gain, router = torch.rand(width, device="cuda"), torch.randn(width, e, device="cuda")
    norm, route = cns.new_rms_norm(width, scale_block=32), cns.new_route(t, e, k)
    work = torch.empty(cns.cns_rms_norm_workspace_bytes(t, width)[1], dtype=torch.uint8, device="cuda")

    def forward(stream):
        h, y, q, scales = cns.run_rms_norm(norm, x, gain, residual=residual, stream=stream)
        cns.run_route(route, y @ router, stream=stream)
        rows = cns.run_dispatch(route, y, stream=stream)
        eight, eight_scales = cns.run_dispatch(route, q, scales=scales, stream=stream)
        return h, y, rows, eight, eight_scales, cns.run_combine(route, rows, base=h, stream=stream)

    def backward(h, rows, stream):
        drows, dweights = cns.run_combine_backward(route, rows, dout, stream=stream)
        dy = cns.run_dispatch_backward(route, drows, stream=stream)
        dx, dgain = cns.run_rms_norm_backward(norm, h, gain, dy, dh=dout, workspace=work, stream=stream)
        return drows, dweights, dy, dx, dgain

    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        f = forward(s)                                 # the kernels are loaded
        backward(f[0], f[2], s)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first, stream=s):
        f = forward(s)
    with torch.cuda.graph(second, stream=s):
        b = backward(f[0], f[2], s)
    for _ in range(3):
        for v in (x, residual, dout):
            v.copy_(torch.randn_like(v))
        work.fill_(255)
        first.replay()
        second.replay()
        replayed = [v.clone() for v in f + b]
        torch.cuda.synchronize()
        again = forward(None)
        again += backward(again[0], again[2], None)
        torch.cuda.synchronize()
        for a, c in zip(replayed, again):
            assert torch.equal(a.contiguous().view(torch.uint8), c.contiguous().view(torch.uint8))


def test_the_examples_block(cns):
    """Gradients of the block with its residual against torch's own of the same layer in 64 bits; it runs and clips."""
    import torch
    from examples.expert_training_step import Block, train
    torch.manual_seed(4)
    t, width, hidden, e, k = 200, 32, 48, 16, 2
    block = Block(t, width, hidden, e, k)
    with torch.no_grad():
        block.gain.uniform_(0.5, 1.5)
    x, residual = (torch.randn(t, width, device="cuda", requires_grad=True) for _ in range(2))
    dout = torch.randn(t, width, device="cuda")
    (block(x, residual) * dout).sum().backward()
    ids = block.experts.route.ids[:t].long()
    params = [x, residual, *block.parameters()]
    w = [p.detach().double().requires_grad_() for p in params]
    x64, r64, gain, router, up, down = w
    h = x64 + r64
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * gain
    score = torch.sigmoid(y @ router).gather(1, ids)
    score = score / score.sum(-1, keepdim=True)
    out = h + sum((torch.relu(torch.einsum("td,tdh->th", y, up[ids[:, j]])).unsqueeze(1) @ down[ids[:, j]]).squeeze(1)
                  * score[:, j:j + 1] for j in range(k))
    (out * dout.double()).sum().backward()
    for p, q in zip(params, w):
        # as for the layer: some 500 roundings, against the largest
        assert (p.grad.double() - q.grad).abs().max() <= 500 * 2.0 ** -24 * q.grad.abs().max()
    first = torch.autograd.grad(block(x, residual).square().mean(), x, create_graph=True)[0]
    with pytest.raises(RuntimeError, match="once"):
        first.square().sum().backward()
    losses, norms = train(steps=5, kind=Block)
    assert np.isfinite(losses).all()
    for before, after in norms:
        assert after <= min(before, 0.05) * (1 + 1e-5)


def test_threads_share_handles(cns):
    """Calls of several threads, each on a stream and tensors of its own, by one route and one norm."""
    import threading

    import torch
    torch.manual_seed(8)
    t, width, e, k = 900, 520, 16, 4
    norm, route = cns.new_rms_norm(width, scale_block=128), cns.new_route(t, e, k)
    cns.run_route(route, torch.randn(t, e, device="cuda"), sync=True)
    places, weights = route.places.clone(), route.weights.clone()
    gain = torch.randn(width, device="cuda")

    def step(x, dy, stream):
        h, y, q, scales = cns.run_rms_norm(norm, x, gain, residual=dy, stream=stream)
        rows = cns.run_dispatch(route, y, places=places, stream=stream)
        out = cns.run_combine(route, rows, weights=weights, places=places, base=h, stream=stream)
        drows, dweights = cns.run_combine_backward(route, rows, dy, weights=weights, places=places, stream=stream)
        dx, dgain = cns.run_rms_norm_backward(norm, h, gain, cns.run_dispatch_backward(route, drows, places=places, stream=stream),
                                              dh=dy, stream=stream)
        return h, y, q, scales, rows, out, drows, dweights, dx, dgain

    inputs = [(torch.randn(t, width, device="cuda"), torch.randn(t, width, device="cuda")) for _ in range(4)]
    want = [step(x, dy, None) for x, dy in inputs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                got = step(*inputs[i], s)
                s.synchronize()
                if not all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong
