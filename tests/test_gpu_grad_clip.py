"""cns_grad_norm and cns_grad_clip on the GPU against the definition in 64 bits.

Tolerance of the norm.  All terms of the sum are positive, so its relative
error is at most the number of roundings on the longest path from a square to
the sum times 2^-24: 16 within a lane's tile, 3 joining its accumulators, 64
tiles of a block and (here) at most 16 blocks, 10 in the CTA's two trees, 5 +
5 across the CTAs with 2 for the quotients: below 128.  The root halves that,
and three roots round once more: (64 + 3) * 2^-24 < 4.1e-6.

The clipped values have no tolerance: the factor is min(1, max_norm / (norm +
eps)) in 32 bits of the norm that came back, and each value one product in 32
bits rounded once to its type, so they are equal bit for bit."""
import numpy as np
import pytest

from oracle import steps

pytestmark = pytest.mark.gpu

NORM_RTOL = 4.1e-6


@pytest.fixture(scope="module")
def cns():
    import torch
    import counted_notify_sync_gb300 as c
    c.build()
    torch.cuda.set_device(0)
    return c


def types():
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make(sizes, dtypes, offset=0, seed=0, scale=1.0):
    """Tensors carved out of one allocation per type, back to back from `offset` elements on."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    out, used = [], {}
    total = {d: sum(n for n, e in zip(sizes, dtypes) if e == d) for d in set(dtypes)}
    flat = {d: (torch.randn(n + offset + 8, generator=gen, device="cuda") * scale).to(types()[d]) for d, n in total.items()}
    for n, d in zip(sizes, dtypes):
        at = offset + used.get(d, 0)
        out.append(flat[d][at:at + n])
        used[d] = used.get(d, 0) + n
    return out, flat


def expected(tensors, norm, max_norm, eps, out_types):
    """The clipped values that follow from the returned norm, on the CPU."""
    import torch
    f = np.float32(max_norm) / (np.float32(norm) + np.float32(eps))
    f = f if f < 1 or np.isnan(f) else np.float32(1)
    return [(t.cpu().float() * torch.tensor(f)).to(d) for t, d in zip(tensors, out_types)]


def same_bits(a, b):
    import torch
    view = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.cpu().contiguous().view(view), b.cpu().contiguous().view(view))


SIZES = {
    "one": [1], "tile": [128, 1024, 4096], "empty-among": [0, 5, 0, 77, 0], "odd": [3, 1, 17, 1023, 4097, 33],
    "two-rounds": [1_300_001, 7, 999_983, 12], "many-small": [1 + i % 9 for i in range(700)],
    "beyond-arguments": [1 + (i * 7) % 50 for i in range(1100)], "mixed": [1000 + 37 * i for i in range(70)],
    "many-rounds": [17_000_001, 3, 13_000_000],
}


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16", "mix"])
@pytest.mark.parametrize("offset", [0, 3])
def test_norm_and_clip(cns, name, dtype, offset):
    import torch
    sizes = SIZES[name]
    dts = [["f32", "bf16", "f16"][i % 3] if dtype == "mix" else dtype for i in range(len(sizes))]
    grads, _ = make(sizes, dts, offset, seed=len(sizes))
    before = [g.clone() for g in grads]
    want = steps.grad_norm([g.cpu().double().numpy() for g in grads])
    max_norm = float(want) / 3
    for out in ("f32", "same", "place"):
        odt = [types()["f32"] if out == "f32" else types()[d] for d in dts]
        names = ["f32"] * len(dts) if out == "f32" else dts
        outs, flat = (None, {}) if out == "place" else make(sizes, names, offset, seed=99)
        guard = {d: f.clone() for d, f in flat.items()}
        plan = cns.new_grad_clip(grads, max_norm, outs=outs)
        norm = cns.run_grad_norm(plan, sync=True).item()
        assert abs(norm - want) <= NORM_RTOL * want
        assert all(same_bits(a, b) for a, b in zip(grads, before))
        again = cns.run_grad_clip(plan, sync=True).item()
        assert again == norm                                       # the same sum every time
        got = grads if outs is None else outs
        for a, b in zip(got, expected(before, norm, max_norm, 1e-6, odt)):
            assert same_bits(a, b)
        for d, f in flat.items():                                  # nothing written beside the tensors
            n = sum(k for k, e in zip(sizes, names) if e == d)
            assert same_bits(f[:offset], guard[d][:offset]) and same_bits(f[offset + n:], guard[d][offset + n:])
        if outs is None:
            for g, b in zip(grads, before):
                g.copy_(b)


@pytest.mark.parametrize("shift", [1, 2, 3, 5, 7])
def test_outputs_at_other_alignments_than_their_gradients(cns, shift):
    import torch
    for src, dst in (("bf16", "f32"), ("f32", "bf16"), ("f16", "f16"), ("f32", "f32")):
        grads, _ = make([5001, 64, 40_000], [src] * 3, 0, seed=4)
        outs, _ = make([5001, 64, 40_000], [dst] * 3, shift, seed=5)
        plan = cns.new_grad_clip(grads, 0.5, outs=outs)
        norm = cns.run_grad_clip(plan, sync=True).item()
        for a, b in zip(outs, expected(grads, norm, 0.5, 1e-6, [types()[dst]] * 3)):
            assert same_bits(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_inf_norm_is_exact(cns, dtype):
    for name in ("one", "odd", "two-rounds"):
        grads, _ = make(SIZES[name], [dtype] * len(SIZES[name]), 1, seed=7)
        plan = cns.new_grad_clip(grads, 0.1, norm_type=cns.CNS_NORM_INF)
        before = [g.clone() for g in grads]
        want = steps.grad_norm([g.cpu().double().numpy() for g in grads], inf=True)
        norm = cns.run_grad_clip(plan, sync=True).item()
        assert norm == want
        assert all(same_bits(a, b) for a, b in zip(grads, expected(before, norm, 0.1, 1e-6, [types()[dtype]] * len(grads))))


@pytest.mark.parametrize("norm_type", [0, 1])
@pytest.mark.parametrize("poison", [float("inf"), float("nan"), -float("inf")])
@pytest.mark.parametrize("n", [100, 3_000_000])
def test_infinite_and_nan_gradients(cns, norm_type, poison, n):
    import torch
    for at in (0, n // 2, n - 1):
        g = torch.ones(n, device="cuda")
        g[at] = poison
        plan = cns.new_grad_clip([g], 1.0, norm_type=norm_type)
        norm = cns.run_grad_clip(plan, sync=True)
        if np.isnan(poison):
            assert torch.isnan(norm) and torch.isnan(g).all()
        else:
            # the factor is 0: zeros, and 0 * inf where the infinity was
            assert torch.isposinf(norm) and torch.isnan(g[at]) and int((g == 0).sum()) == n - 1


def test_factor_limits(cns):
    import torch
    g, _ = make([1000, 3], ["f32", "f32"], 1, seed=1)
    before = [t.clone() for t in g]
    for max_norm in (float("inf"), 1e9):                           # nothing to clip
        cns.run_grad_clip(cns.new_grad_clip(g, max_norm), sync=True)
        assert all(same_bits(a, b) for a, b in zip(g, before))
    out = [torch.empty_like(t) for t in g]
    cns.run_grad_clip(cns.new_grad_clip(g, 1e9, outs=out), sync=True)
    assert all(same_bits(a, b) for a, b in zip(out, before))
    cns.run_grad_clip(cns.new_grad_clip(g, 0.0), sync=True)
    assert all((t == 0).all() for t in g)
    zero = torch.zeros(50, device="cuda")
    plan = cns.new_grad_clip([zero], 1.0, eps=0.0)                 # 1 / 0 = inf, at most 1
    assert cns.run_grad_clip(plan, sync=True).item() == 0.0 and (zero == 0).all()
    empty = cns.new_grad_clip([], 1.0)
    assert cns.run_grad_clip(empty, sync=True).item() == 0.0
    assert cns.run_grad_norm(cns.new_grad_clip([torch.empty(0, device="cuda")]), sync=True).item() == 0.0


def test_large_magnitudes_across_ctas(cns):
    """CTAs' sums near the top of the range: their join must not overflow."""
    import torch
    g = torch.full((152 * 1024 * 4,), 5e16, device="cuda")
    norm = cns.run_grad_norm(cns.new_grad_clip([g]), sync=True).item()
    want = float(np.float32(5e16)) * np.sqrt(g.numel())
    assert abs(norm - want) <= NORM_RTOL * want


def test_more_elements_than_31_bits_count(cns):
    import torch
    n = 2 ** 31 + 5
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    g[-1] = 256.0
    plan = cns.new_grad_clip([g], 2.0 ** 10)
    norm = cns.run_grad_clip(plan, sync=True).item()
    want = np.sqrt(n - 1 + 65536.0)
    assert abs(norm - want) <= NORM_RTOL * want
    ends = torch.cat([g[:3], g[2 ** 31 - 2:]])
    src = torch.ones(ends.numel(), dtype=torch.bfloat16)
    src[-1] = 256.0
    assert same_bits(ends, expected([src], norm, 2.0 ** 10, 1e-6, [torch.bfloat16])[0])
    assert int((g[:-1] != g[0]).sum()) == 0


def test_streams_graphs_and_shared_workspaces(cns):
    import torch
    ws = cns.new_step_workspace(cns.cns_grad_workspace_bytes(1200)[1])
    plans = []
    for k, name in enumerate(("one", "two-rounds", "beyond-arguments", "odd", "many-small")):
        grads, _ = make(SIZES[name], ["bf16"] * len(SIZES[name]), 0, seed=k)
        outs, _ = make(SIZES[name], ["f32"] * len(SIZES[name]), 0, seed=50 + k)
        plans.append((cns.new_grad_clip(grads, 0.7, outs=outs, workspace=ws), grads, outs))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):                                             # one workspace, grids of every size in turn
        for plan, _, _ in plans:
            cns.run_grad_clip(plan, stream=s)
    s.synchronize()
    for plan, grads, outs in plans:
        assert all(same_bits(a, b) for a, b in zip(outs, expected(grads, plan.norm.item(), 0.7, 1e-6, [torch.float32] * len(outs))))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for plan, _, _ in plans:
            cns.run_grad_clip(plan, stream=s)
    for plan, grads, outs in plans:                                # new values in the same tensors
        for t in grads:
            t.mul_(1.5)
        for t in outs:
            t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for plan, grads, outs in plans:
        want = steps.grad_norm([t.cpu().double().numpy() for t in grads])
        assert abs(plan.norm.item() - want) <= NORM_RTOL * want
        assert all(same_bits(a, b) for a, b in zip(outs, expected(grads, plan.norm.item(), 0.7, 1e-6, [torch.float32] * len(outs))))


def test_a_failed_workspace_is_refused_until_it_is_initialised(cns):
    import torch
    g = torch.ones(3_000_000, device="cuda")
    plan = cns.new_grad_clip([g], 1.0)
    plan.norm.fill_(-1.0)
    plan.workspace[32] = cns.CNS_ERR_TIMEOUT                       # what a wait that ran out leaves
    plan.workspace[33] = 1
    with pytest.raises(cns.CnsError) as e:
        cns.run_grad_clip(plan, sync=True)
    assert e.value.code == cns.CNS_ERR_TIMEOUT
    assert plan.norm.item() == -1.0 and (g == 1).all()
    cns.check(cns.cns_step_workspace_init(plan.workspace, plan.workspace.numel() * 4))
    assert abs(cns.run_grad_clip(plan, sync=True).item() - np.sqrt(3e6)) < 0.01


def test_a_failed_workspace_refuses_the_norm_too(cns):
    import torch
    plan = cns.new_grad_clip([torch.ones(3_000_000, device="cuda")], 1.0)
    plan.norm.fill_(-1.0)
    plan.workspace[32] = cns.CNS_ERR_TIMEOUT
    plan.workspace[33] = 1
    with pytest.raises(cns.CnsError):
        cns.run_grad_norm(plan, sync=True)
    assert plan.norm.item() == -1.0
    cns.check(cns.cns_step_workspace_init(plan.workspace, plan.workspace.numel() * 4))
    assert abs(cns.run_grad_norm(plan, sync=True).item() - np.sqrt(3e6)) < 0.01


def test_norms_and_clippings_of_all_sizes_share_a_workspace(cns):
    """One after the other without a wait between them: the same bits as each alone."""
    import torch
    sizes = [7, 40_000, 3_000_000, 900_000, 1]
    grads = [torch.randn(n, device="cuda") for n in sizes]
    ws = cns.new_step_workspace(cns.cns_grad_workspace_bytes(1)[1])
    plans = [cns.new_grad_clip([g], 1.0, outs=[torch.empty_like(g)], workspace=ws) for g in grads]
    alone = [cns.run_grad_norm(cns.new_grad_clip([g]), sync=True).item() for g in grads]
    got = []
    for i in range(40):
        plan = plans[i % 5]
        got.append((cns.run_grad_clip if i % 3 == 0 else cns.run_grad_norm)(plan).clone())
    torch.cuda.synchronize()
    assert [g.item() for g in got] == [alone[i % 5] for i in range(40)]
    assert cns.syncall_read_workspace(ws)[3] == 0


def test_python_refusals(cns):
    import torch
    a = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        cns.new_grad_clip([a, a[10:20]], 1.0)
    with pytest.raises(ValueError, match="overlap"):
        cns.new_grad_clip([a[:32]], 1.0, outs=[a[16:48]])
    cns.new_grad_clip([a, a[10:20]], 1.0, outs=[torch.zeros_like(a), torch.zeros(10, device="cuda")])   # read twice only
    with pytest.raises(ValueError, match="dense"):
        cns.new_grad_clip([a[::2]], 1.0)
    with pytest.raises(TypeError):
        cns.new_grad_clip([a.double()], 1.0)
    with pytest.raises(ValueError, match="expected"):
        cns.new_grad_clip([torch.zeros(4)], 1.0)
    with pytest.raises(ValueError, match="shape"):
        cns.new_grad_clip([a], 1.0, outs=[torch.zeros(63, device="cuda")])
    m = torch.randn(8, 16, device="cuda").t()                      # dense, columns first
    want = steps.grad_norm([m.cpu().numpy()])
    assert abs(cns.run_grad_norm(cns.new_grad_clip([m]), sync=True).item() - want) <= NORM_RTOL * want
