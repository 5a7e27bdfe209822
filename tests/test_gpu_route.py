"""cns_route and cns_route_backward on the GPU against the definitions in 64 bits.

Choices are compared exactly.  Choices by logit are exact whatever the logits.
Choices by score and bias compare sums in 32 bits that the GPU and the oracle
round apart by a few units of 2^-24, so their inputs are drawn from grids whose
sums are either equal (logit and bias equal: the lower index first) or further
apart than 4e-6; a test checks that of its inputs before it uses them.

Tolerances.  expf is within 2 units in the last place, the sum and the quotient
round once each: a sigmoid score is within 4 * 2^-24; with renorm the sum of at
most 32 of them adds 6 roundings and the quotient and the scale one each: below
16 * 2^-24 = 9.6e-7.  A softmax exponent l - top, at most 40 here, is rounded
at 2^-24 relative, which e^x makes 40 * 2^-24; with the sum's 21 roundings:
below 64 * 2^-24 = 3.9e-6 relative.  In the gradient those factors meet terms
of up to sum |g_j| (divided, for renormalised sigmoids, by their sum once and
in the inner product once more): 8e-6 of that."""
import numpy as np
import pytest

from oracle import steps

pytestmark = pytest.mark.gpu

SIG, SOFT = steps.SIGMOID, steps.SOFTMAX


@pytest.fixture(scope="module")
def cns():
    import torch
    import counted_notify_sync_gb300 as c
    c.build()
    torch.cuda.set_device(0)
    return c


def ttype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def grid_inputs(tokens, experts, seed, masked=0.0):
    """Logits in eighths of [-3, 3] and biases in 1/64 + 1/999: sums that are equal or well apart."""
    rng = np.random.RandomState(seed)
    x = rng.randint(-24, 25, size=(tokens, experts)) / 8.0
    b = (rng.randint(0, 4, size=experts) * (1 / 64 + 1 / 999)).astype(np.float32)
    if masked:
        x[rng.rand(tokens, experts) < masked] = -np.inf
        x[rng.rand(tokens) < masked] = -np.inf
    return x, b


def check(cns, x, bias, dtype, capacity=None, stride=None, stream=None, **kw):
    """Route x (float64 values that dtype holds) and compare everything with the oracle; returns the plan."""
    import torch
    t, e = x.shape
    k = kw.pop("top_k")
    logits = torch.from_numpy(x).to(ttype(dtype))
    assert np.array_equal(logits.double().numpy(), x), "values that the type does not hold"
    if stride:
        wide = torch.full((t, stride), 77.0, dtype=ttype(dtype), device="cuda")
        wide[:, 1:1 + e] = logits.cuda()
        logits = wide[:, 1:1 + e]
    else:
        logits = logits.cuda()
    b = None if bias is None else torch.from_numpy(bias).cuda()
    r = cns.new_route(capacity or t, e, k, scores=True, **kw)
    for v in (r.ids, r.weights, r.offsets, r.order, r.places, r.scores):
        v.fill_(-7)
    cns.run_route(r, logits, bias=b, sync=True, stream=stream)
    kw.setdefault("score", SOFT)
    ids, w, s = steps.route(x, bias, top_k=k, **kw)
    assert np.array_equal(r.ids[:t].cpu().numpy(), ids)
    rtol = 9.6e-7 if kw["score"] == SIG else 3.9e-6
    np.testing.assert_allclose(r.weights[:t].cpu().double().numpy(), w, rtol=rtol, atol=1e-30)
    np.testing.assert_allclose(r.scores[:t].cpu().double().numpy(), s, rtol=rtol, atol=1e-30)
    offsets, order, places = steps.plan(ids, e)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy()[:t * k], order)
    assert np.array_equal(r.places[:t].cpu().numpy(), places)
    if capacity:                                                   # nothing beyond the call's tokens
        assert (r.ids[t:] == -7).all() and (r.order[t * k:] == -7).all() and (r.weights[t:] == -7).all()
    return r


def values_apart(x, bias, groups, group_top):
    """Whether the choice values of each row, and its groups' worths, are equal or 4e-6 apart."""
    s = 1.0 / (1.0 + np.exp(-x)) + (0 if bias is None else bias.astype(np.float64))
    s[x == -np.inf] = -9.0
    rows = [s]
    if groups > 1:
        rows.append(np.sort(s.reshape(len(s), groups, -1), -1)[..., -group_top:].sum(-1))
    gaps = [np.diff(np.sort(r, -1), axis=-1) for r in rows]
    return all(((g < 1e-12) | (g > 4e-6)).all() for g in gaps)


@pytest.mark.parametrize("tokens", [1, 2, 31, 33, 200, 1000, 5003])
@pytest.mark.parametrize("experts,top_k", [(1, 1), (8, 2), (33, 5), (64, 6), (100, 3), (160, 8), (256, 8), (384, 8), (512, 32)])
def test_softmax_by_logit(cns, tokens, experts, top_k):
    if tokens * experts > 1_000_000:
        pytest.skip("the oracle's rows are Python")
    rng = np.random.RandomState(tokens + experts)
    x = rng.randn(tokens, experts).astype(np.float16).astype(np.float64)
    check(cns, x, None, "f16", top_k=top_k, score=SOFT, renorm=bool(tokens & 1), scale=1.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,experts,top_k,groups,top_groups,group_top", [
    (700, 64, 4, 1, 0, 1), (300, 256, 8, 8, 4, 2), (301, 160, 6, 8, 3, 1), (64, 384, 8, 4, 2, 2), (40, 96, 3, 32, 5, 2),
    (77, 24, 6, 4, 4, 2), (50, 12, 1, 12, 1, 2), (9, 512, 32, 2, 1, 2)])
@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_with_bias_and_groups(cns, dtype, tokens, experts, top_k, groups, top_groups, group_top, renorm):
    x, b = grid_inputs(tokens, experts, seed=experts + tokens, masked=0.1)
    assert values_apart(x.copy(), b, groups, group_top)
    check(cns, x, b, dtype, top_k=top_k, score=SIG, groups=groups, top_groups=top_groups, group_top=group_top,
          renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("groups", [1, 4])
def test_masks_that_leave_little_or_nothing(cns, score, groups):
    x, _ = grid_inputs(64, 32, seed=3)
    x[0] = -np.inf                                  # nothing
    x[1, 1:] = -np.inf                              # one expert
    x[2, :30] = -np.inf                             # two, the last ones
    x[3, ::2] = -np.inf
    x[4] = np.finfo(np.float32).min                 # the type's lowest value is a number
    x[5, 8:] = np.finfo(np.float32).min
    x[6, 8:] = -np.inf                              # one group
    check(cns, x, None, "f32", top_k=5, score=score, groups=groups, top_groups=2 if groups > 1 else 1)


def test_bias_of_minus_infinity_masks_an_expert(cns):
    x, b = grid_inputs(100, 16, seed=8)
    b[3] = -np.inf
    b[7] = -np.inf
    r = check(cns, x, b, "f32", top_k=15, score=SIG)
    assert not np.isin(r.ids.cpu().numpy(), [3, 7]).any() and (r.ids[:, 14] == -1).all()


def test_nan_and_infinite_logits(cns):
    import torch
    x = torch.zeros(4, 8, device="cuda")
    x[0, 5] = float("nan")
    x[1, 2] = float("inf")
    x[2, 6] = -float("nan")
    for score in (SIG, SOFT):
        r = cns.new_route(4, 8, 2, score=score)
        cns.run_route(r, x, sync=True)
        assert r.ids[0, 0] == 5 and r.ids[2, 0] == 6 and r.ids[1, 0] == 2          # NaN ranks first
        assert torch.isnan(r.weights[0, 0]) and torch.isnan(r.weights[2, 0])
        if score == SIG:
            assert abs(r.weights[1, 0].item() - 2 / 3) < 1e-6
        assert r.ids.min() >= 0 and r.ids.max() < 8
        np.testing.assert_allclose(r.weights[3].cpu().numpy(), [0.5, 0.5])


def test_negative_zero_is_zero(cns):
    import torch
    x = torch.full((1, 40), -0.0, device="cuda")
    x[0, 30] = 0.0
    r = cns.new_route(1, 40, 3)
    cns.run_route(r, x, sync=True)
    assert r.ids[0].tolist() == [0, 1, 2]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts", [7, 64, 100])
def test_strided_rows_and_spare_capacity(cns, dtype, experts):
    x, b = grid_inputs(130, experts, seed=experts)
    for stride in (experts + 1, experts + 3, 2 * experts + 2):
        check(cns, x, b, dtype, top_k=3, score=SIG, stride=stride, capacity=200)


@pytest.mark.parametrize("experts,top_k", [(40, 3), (256, 8), (384, 8), (500, 20)])
@pytest.mark.parametrize("spread", [3, 12, 60, 500])
def test_logits_a_rounding_apart(cns, experts, top_k, spread):
    """Rows whose leading logits are neighbouring floats, `spread` of them: fewer and more than what a token's
    choice is settled among, equals too."""
    rng = np.random.RandomState(experts + spread)
    x = rng.randn(64, experts).astype(np.float32)
    for r in range(64):
        at = rng.permutation(experts)[:spread]
        x[r, at] = np.float32(5.0) + np.float32(2.0 ** -21) * rng.randint(0, max(2, spread // 2), size=at.size).astype(np.float32)
    x[5] = x[5, 0]                                   # all equal
    for groups in (1, 4) if experts % 4 == 0 else (1,):
        check(cns, x.astype(np.float64), None, "f32", top_k=top_k, score=SOFT, groups=groups,
              top_groups=3 if groups > 1 else 1)


@pytest.mark.parametrize("experts,top_k", [(64, 8), (256, 8), (384, 6), (512, 16)])
@pytest.mark.parametrize("spread", [3, 12, 60, 500])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (8, 2), (4, 1)])
def test_scores_a_rounding_apart(cns, experts, top_k, spread, groups, group_top):
    """The same for scores with a bias, against the definition in 32 bits on the device: 1 / (1 + exp(-l)), plus
    the bias, sorted with equals in order."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(experts + spread)
    x = torch.randn(200, experts, generator=gen, device="cuda")
    pick = torch.rand(200, experts, generator=gen, device="cuda").argsort(-1)[:, :spread]
    near = 1.5 + 1e-6 * torch.rand(200, pick.shape[1], generator=gen, device="cuda")
    x.scatter_(1, pick, near)
    b = 0.3 * torch.randn(experts, generator=gen, device="cuda")
    b[torch.rand(experts, generator=gen, device="cuda") < 0.7] = 0.125
    top_groups = max(1, groups // 2)
    v = 1.0 / (1.0 + torch.exp(-x)) + b
    if groups > 1:
        worth = v.view(200, groups, -1).sort(dim=-1, descending=True).values[..., :group_top].sum(-1)
        keep = worth.sort(dim=-1, descending=True, stable=True).indices[:, :top_groups]
        stays = torch.zeros(200, groups, dtype=torch.bool, device="cuda").scatter_(1, keep, True)
        v = torch.where(stays.repeat_interleave(experts // groups, 1), v, torch.full_like(v, -float("inf")))
    want = v.sort(dim=-1, descending=True, stable=True).indices[:, :top_k]
    r = cns.new_route(200, experts, top_k, score=SIG, groups=groups, top_groups=top_groups, group_top=group_top)
    cns.run_route(r, x, bias=b, sync=True)
    assert torch.equal(r.ids.long(), want)


@pytest.mark.parametrize("bias", [3e30, -5e7, float("nan"), 0.0])
def test_biases_beyond_the_fast_path(cns, bias):
    import torch
    x, _ = grid_inputs(90, 48, seed=2)
    b = torch.zeros(48, device="cuda")
    b[7] = bias
    xs = torch.from_numpy(x).float().cuda()
    r = cns.new_route(90, 48, 5, score=SIG)
    cns.run_route(r, xs, bias=b, sync=True)
    v = 1.0 / (1.0 + torch.exp(-xs)) + b
    assert torch.equal(r.ids.long(), v.sort(dim=-1, descending=True, stable=True).indices[:, :5])


@pytest.mark.parametrize("experts,top_k,groups,group_top", [(64, 6, 1, 1), (256, 8, 8, 2), (160, 4, 8, 2), (512, 20, 1, 1)])
@pytest.mark.parametrize("bias", [True, False])
def test_softmax_by_score(cns, experts, top_k, groups, group_top, bias):
    """Softmax scores chosen with a bias, or with groups worth two.  The softmax's sum rounds with its order, so
    the choice is held to its definition in 64 bits within 1e-6 of the values: in order, and none left out that
    is above."""
    import torch
    if not bias and group_top == 1:
        pytest.skip("chosen by logit")
    rng = np.random.RandomState(experts)
    x = (2 * rng.randn(400, experts)).astype(np.float32)
    x[rng.rand(400, experts) < 0.05] = -np.inf
    x[3] = -np.inf
    b = (0.02 * rng.randn(experts)).astype(np.float32) if bias else None
    top_groups = max(1, groups // 2)
    r = cns.new_route(400, experts, top_k, score=SOFT, groups=groups, top_groups=top_groups, group_top=group_top)
    cns.run_route(r, torch.from_numpy(x).cuda(), bias=None if b is None else torch.from_numpy(b).cuda(), sync=True)
    ids, w = r.ids.cpu().numpy(), r.weights.cpu().double().numpy()
    assert (ids[3] == -1).all() and (w[3] == 0).all()
    for t in range(400):
        if t == 3:
            continue
        s = steps.scores(x[t].astype(np.float64), SOFT)
        v = s + (0 if b is None else b.astype(np.float64))
        v[x[t] == -np.inf] = -np.inf
        assert len(set(ids[t])) == top_k and ids[t].min() >= 0
        if groups > 1:
            worth = np.array([np.sort(g[g > -np.inf])[-2:].sum() for g in v.reshape(groups, -1)])
            used = np.unique(ids[t] // (experts // groups))
            assert len(used) <= top_groups
            # the groups used are worth as much as the best ones, and nothing better in them was left out
            bound = np.sort(worth)[-top_groups]
            assert (worth[used] >= bound - 2e-6).all()
            open_ = [g for g in range(groups) if worth[g] > bound + 2e-6] + list(used)
            inside = np.isin(np.arange(experts) // (experts // groups), open_)
        else:
            inside = np.ones(experts, dtype=bool)
        chosen = v[ids[t]]
        assert (np.diff(chosen) <= 1e-6).all()
        rest = inside.copy()
        rest[ids[t]] = False
        assert not rest.any() or v[rest].max() <= chosen[-1] + 1e-6
        q = steps.scores(x[t][ids[t]].astype(np.float64), SOFT)
        np.testing.assert_allclose(w[t], q, rtol=3.9e-6)


@pytest.mark.parametrize("low", [-50.0, -87.5, -88.5, -100.0, -1e10, -3.4028234663852886e38])
@pytest.mark.parametrize("groups", [1, 4])
def test_low_logits_with_high_biases(cns, low, groups):
    """Scores of next to nothing that a bias lifts among the chosen: masked is only -inf."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    x = torch.randn(150, 128, generator=gen, device="cuda")
    x[torch.rand(150, 128, generator=gen, device="cuda") < 0.3] = low
    x[torch.rand(150, 128, generator=gen, device="cuda") < 0.2] = -float("inf")
    b = torch.rand(128, generator=gen, device="cuda") * 1.5
    v = 1.0 / (1.0 + torch.exp(-x)) + b
    v = torch.where(x == -float("inf"), torch.full_like(v, -float("inf")), v)
    if groups > 1:
        best = v.view(150, groups, -1).sort(dim=-1, descending=True).values[..., :2]
        worth = torch.where(best == -float("inf"), torch.zeros_like(best), best).sum(-1)
        keep = worth.sort(dim=-1, descending=True, stable=True).indices[:, :2]
        stays = torch.zeros(150, groups, dtype=torch.bool, device="cuda").scatter_(1, keep, True)
        v = torch.where(stays.repeat_interleave(128 // groups, 1), v, torch.full_like(v, -float("inf")))
    r = cns.new_route(150, 128, 8, score=SIG, groups=groups, top_groups=2 if groups > 1 else 1,
                      group_top=2 if groups > 1 else 1)
    cns.run_route(r, x, bias=b, sync=True)
    assert torch.equal(r.ids.long(), v.sort(dim=-1, descending=True, stable=True).indices[:, :8])


def test_infinite_logits_with_biases(cns):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(12)
    x = torch.randn(60, 64, generator=gen, device="cuda")
    x[torch.rand(60, 64, generator=gen, device="cuda") < 0.05] = float("inf")
    b = torch.rand(64, generator=gen, device="cuda")
    v = 1.0 / (1.0 + torch.exp(-x)) + b
    r = cns.new_route(60, 64, 8, score=SIG)
    cns.run_route(r, x, bias=b, sync=True)
    assert torch.equal(r.ids.long(), v.sort(dim=-1, descending=True, stable=True).indices[:, :8])


def test_no_tokens(cns):
    import torch
    r = cns.new_route(16, 8, 2)
    r.offsets.fill_(-1)
    cns.run_route(r, torch.empty(0, 8, device="cuda"), sync=True)
    assert (r.offsets == 0).all()


@pytest.mark.parametrize("tokens,experts", [(20_000, 8), (70_001, 5), (16_384, 256), (30_000, 64)])
def test_plan_of_many_tokens(cns, tokens, experts):
    """The plan against numpy's stable sort of the ids that came back."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens)
    x = torch.randn(tokens, experts, generator=gen, device="cuda")
    x[torch.rand(tokens, experts, generator=gen, device="cuda") < 0.3] = -float("inf")
    k = min(8, experts)
    r = cns.new_route(tokens, experts, k)
    cns.run_route(r, x, sync=True)
    flat = r.ids.cpu().numpy().reshape(-1)
    key = np.where(flat < 0, experts, flat)
    order = np.argsort(key, kind="stable").astype(np.int32)
    count = np.bincount(key, minlength=experts + 1)[:experts]
    assert np.array_equal(r.offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(count)]))
    order[count.sum():] = -1
    assert np.array_equal(r.order.cpu().numpy(), order)
    places = np.full(flat.size, -1, dtype=np.int32)
    places[order[:count.sum()]] = np.arange(count.sum())
    assert np.array_equal(r.places.cpu().numpy().reshape(-1), places)
    first = [v.clone() for v in (r.ids, r.weights, r.offsets, r.order, r.places)]
    for _ in range(3):                              # the same again, whatever the timing
        cns.run_route(r, x, sync=True)
        assert all(torch.equal(a, b) for a, b in zip(first, (r.ids, r.weights, r.offsets, r.order, r.places)))


def test_one_expert_takes_everything(cns):
    import torch
    x = torch.zeros(9001, 64, device="cuda")
    x[:, 63] = 1.0
    r = cns.new_route(9001, 64, 1)
    cns.run_route(r, x, sync=True)
    assert (r.ids == 63).all() and r.offsets[63] == 0 and r.offsets[64] == 9001
    assert torch.equal(r.order.cpu(), torch.arange(9001, dtype=torch.int32))


def test_without_a_plan(cns):
    x, b = grid_inputs(50, 64, seed=1)
    import torch
    r = cns.new_route(50, 64, 4, score=SIG, plan=False)
    cns.run_route(r, torch.from_numpy(x).float().cuda(), bias=torch.from_numpy(b).cuda(), sync=True)
    ids, w, _ = steps.route(x, b, top_k=4, score=SIG)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    np.testing.assert_allclose(r.weights.cpu().numpy(), w, rtol=9.6e-7)


def test_streams_graphs_and_shared_workspaces(cns):
    import torch
    shapes = [(1, 64, 4), (3000, 64, 4), (40, 256, 8), (9000, 128, 2), (200, 8, 1)]
    need = max(cns.cns_route_workspace_bytes(t, e, k)[1] for t, e, k in shapes)
    ws = cns.new_step_workspace(need)
    s = torch.cuda.Stream()
    runs = []
    for i, (t, e, k) in enumerate(shapes):
        x = torch.randn(t, e, device="cuda")
        runs.append((cns.new_route(t, e, k, workspace=ws), x))
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    for r, x in runs:
        cns.run_route(r, x, stream=s)
    s.synchronize()
    with torch.cuda.graph(g, stream=s):
        for r, x in runs:
            cns.run_route(r, x, stream=s)
    for _, x in runs:
        x.copy_(torch.randn_like(x))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for (t, e, k), (r, x) in zip(shapes, runs):
        top = x.cpu().double().numpy()
        want = np.argsort(-top, -1, kind="stable")[:, :k]
        assert np.array_equal(r.ids.cpu().numpy(), want)
        offsets, order, places = steps.plan(want, e)
        assert np.array_equal(r.order.cpu().numpy(), order) and np.array_equal(r.places.cpu().numpy(), places)


def test_calls_on_several_streams_at_once(cns):
    """Whole-GPU grids from three streams, each with its own workspace: none waits for another's."""
    import torch
    shapes = [(6000, 64, 4), (9000, 256, 8), (400, 128, 8)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    runs = [(cns.new_route(t, e, k), torch.randn(t, e, device="cuda")) for t, e, k in shapes]
    g = torch.randn(5_000_000, device="cuda")
    clip = cns.new_grad_clip([g], 1.0, outs=[torch.empty_like(g)])
    torch.cuda.synchronize()
    for _ in range(30):
        for (r, x), s in zip(runs, streams):
            cns.run_route(r, x, stream=s)
        cns.run_grad_clip(clip, stream=streams[3])
    torch.cuda.synchronize()
    for (r, x), (t, e, k) in zip(runs, shapes):
        assert cns.syncall_read_workspace(r.workspace)[3] == 0
        want = np.argsort(-x.cpu().numpy(), -1, kind="stable")[:, :k]
        assert np.array_equal(r.ids.cpu().numpy(), want)
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip((r.offsets, r.order, r.places), steps.plan(want, e)))
    assert cns.syncall_read_workspace(clip.workspace)[3] == 0
    assert abs(clip.norm.item() / float(torch.linalg.vector_norm(g.double())) - 1) < 4.1e-6


@pytest.mark.parametrize("tokens,experts,top_k", [(20, 64, 4), (700, 96, 6), (5000, 128, 8)])
def test_calls_follow_what_is_before_them_in_the_stream(cns, tokens, experts, top_k):
    """Grids are launched before the kernel ahead of them has ended: its results, and no older ones, are read."""
    import torch
    slow = torch.randn(2048, 2048, device="cuda")
    xs = [torch.randn(tokens, experts, device="cuda") for _ in range(12)]
    dws = [torch.randn(tokens, top_k, device="cuda") for _ in range(12)]
    x, dw, dx = torch.zeros_like(xs[0]), torch.zeros_like(dws[0]), torch.zeros_like(xs[0])
    r = cns.new_route(tokens, experts, top_k)
    clip = cns.new_grad_clip([dx], 0.5, outs=[torch.empty_like(dx)])
    def step(k):
        x.copy_(xs[k])
        dw.copy_(dws[k])
        cns.run_route(r, x)
        cns.run_route_backward(r, x, dw, dlogits=dx)
        norm = cns.run_grad_norm(clip).clone()
        cns.run_grad_clip(clip)
        return [t.clone() for t in (r.ids, r.weights, r.offsets, r.order, r.places, dx, clip.tensors[1][0])] + [norm]
    alone = []
    for k in range(12):
        alone.append(step(k))
        torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(6):
            slow @ slow                                            # lets the host run ahead
        together = [step(k) for k in range(12)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for one, two in zip(alone, together) for a, b in zip(one, two))


def test_a_workspace_shared_with_clipping(cns):
    """Routings and clippings in turn on one workspace: each leaves it as the other needs it."""
    import torch
    ws = cns.new_step_workspace(max(cns.cns_route_workspace_bytes(6000, 96, 4)[1], cns.cns_grad_workspace_bytes(2)[1]))
    xs = [torch.randn(n, 96, device="cuda") for n in (6000, 700, 3000)]
    routes = [cns.new_route(x.shape[0], 96, 4, workspace=ws) for x in xs]
    g = torch.randn(1_000_000, device="cuda")
    clip = cns.new_grad_clip([g], 1e30, outs=[torch.empty_like(g)], workspace=ws)
    for turn in range(7):
        for k, (r, x) in enumerate(zip(routes, xs)):
            r.order.fill_(-7)
            cns.run_route(r, x)
            if (turn + k) % 3 == 0:
                cns.run_grad_clip(clip)
            want = steps.plan(np.argsort(-x.cpu().numpy(), -1, kind="stable")[:, :4], 96)
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip((r.offsets, r.order, r.places), want))


def test_a_failed_workspace_is_refused_until_it_is_initialised(cns):
    import torch
    x = torch.randn(9000, 64, device="cuda")
    r = cns.new_route(9000, 64, 4)
    r.workspace[32] = cns.CNS_ERR_TIMEOUT
    r.workspace[33] = 1
    with pytest.raises(cns.CnsError) as e:
        cns.run_route(r, x, sync=True)
    assert e.value.code == cns.CNS_ERR_TIMEOUT
    cns.check(cns.cns_step_workspace_init(r.workspace, r.workspace.numel() * 4))
    cns.run_route(r, x, sync=True)
    assert r.offsets[64] == 9000 * 4


def test_python_refusals(cns):
    import torch
    r = cns.new_route(8, 16, 2)
    for bad in (torch.zeros(9, 16, device="cuda"), torch.zeros(8, 15, device="cuda"), torch.zeros(8, 16),
                torch.zeros(8, 32, device="cuda")[:, ::2], torch.zeros(1, 16, device="cuda").expand(8, 16)):
        with pytest.raises(ValueError):
            cns.run_route(r, bad)
    with pytest.raises(TypeError):
        cns.run_route(r, torch.zeros(8, 16, dtype=torch.float64, device="cuda"))
    x = torch.zeros(8, 16, device="cuda")
    with pytest.raises(ValueError):
        cns.run_route(r, x, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        cns.run_route(r, x, bias=torch.zeros(16, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        cns.run_route_backward(r, x, torch.zeros(8, 3, device="cuda"))
    with pytest.raises(ValueError):
        cns.run_route_backward(r, x, torch.zeros(8, 2, device="cuda"), dlogits=torch.zeros(8, 16, dtype=torch.float16, device="cuda"))
    with pytest.raises(cns.CnsError):
        cns.new_route(8, 1000, 2)
    with pytest.raises(cns.CnsError):
        cns.run_route(cns.new_route(8, 16, 2, groups=3), x)


# --- the gradient -----------------------------------------------------------------------------------------------

ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("with_scores", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (3, 7, 3), (65, 64, 2), (200, 160, 6), (33, 256, 8), (20, 512, 32), (40, 100, 1)])
def test_gradient_against_the_formula(cns, dtype, score, renorm, with_scores, tokens, experts, top_k):
    import torch
    rng = np.random.RandomState(tokens + experts)
    x = torch.from_numpy(rng.randn(tokens, experts) * 2).to(ttype(dtype))
    if experts > top_k + 4:
        x[torch.from_numpy(rng.rand(tokens, experts) < 0.05)] = -float("inf")
    xd = x.double().numpy()
    ids = np.array([rng.permutation(experts)[:top_k] for _ in range(tokens)], dtype=np.int32)
    for t in range(tokens):                         # a routing never chooses a masked expert
        ids[t][xd[t][ids[t]] == -np.inf] = -1
    dw = rng.randn(tokens, top_k).astype(np.float32)
    ds = rng.randn(tokens, experts).astype(np.float32) if with_scores else None
    scale = 2.5
    r = cns.new_route(tokens, experts, top_k, score=score, renorm=renorm, scale=scale, plan=False)
    got = cns.run_route_backward(r, x.cuda(), torch.from_numpy(dw).cuda(), ids=torch.from_numpy(ids).cuda(),
                                 dscores=None if ds is None else torch.from_numpy(ds).cuda())
    want = steps.route_backward(xd, ids, dw, ds, score=score, renorm=renorm, scale=scale)
    s = np.array([steps.scores(row, score) for row in xd])
    reach = scale * np.abs(np.where(ids >= 0, dw, 0)).sum(-1)
    if renorm and score == SIG:
        reach = reach / np.maximum(np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0).sum(-1), 1e-20) * 2
    if with_scores:
        reach = reach + np.abs(ds).sum(-1)
    err = np.abs(got.cpu().double().numpy() - want)
    allowed = 8e-6 * reach[:, None] + (0 if dtype == "f32" else ULP[dtype] * np.abs(want) + 2.0 ** -24)
    assert (err <= allowed).all(), (err / allowed).max()
    if not with_scores and (renorm or score == SIG):
        touched = np.zeros((tokens, experts), dtype=bool)
        for t in range(tokens):
            touched[t, ids[t][ids[t] >= 0]] = True
        assert (got.cpu().numpy(force=True) if dtype == "f32" else got.cpu().float().numpy())[~touched].max(initial=0.0) == 0.0


@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences_of_the_forward_call(cns, score, renorm):
    """Central differences of sum(dw * weights) through cns_route itself.  With h = 1/64 the truncation is
    below h^2 / 6 * |third derivative| (at most 1 times sum |dw| * scale, the sums here at least 1) and the
    forward call's error 4e-6 * sum |dw| / h: 5e-4 of sum |dw| * scale covers both."""
    import torch
    rng = np.random.RandomState(9)
    t, e, k, scale, h = 5, 12, 3, 1.5, 1 / 64
    # the chosen three stand far above the others, so that no difference changes the choice
    x = rng.randint(-8, 8, size=(t, e)) / 8.0
    for row in x:
        row[rng.permutation(e)[:k]] += 3.0
    x = x + np.arange(e) / 16
    dw = torch.from_numpy(rng.randn(t, k).astype(np.float32)).cuda()
    r = cns.new_route(t, e, k, score=score, renorm=renorm, scale=scale)
    base = torch.from_numpy(x).float().cuda()
    cns.run_route(r, base, sync=True)
    ids = r.ids.clone()
    got = cns.run_route_backward(r, base, dw, ids=ids).cpu().double().numpy()
    dwn = dw.cpu().double().numpy()

    def loss(z):
        cns.run_route(r, z, sync=True)
        w = torch.zeros(t, e, device="cuda", dtype=torch.float64).scatter_(1, r.ids.long(), r.weights.double())
        assert torch.equal(r.ids.sort(-1).values, ids.sort(-1).values)
        return (w.gather(1, ids.long()).cpu().numpy() * dwn).sum(-1)

    for c in range(e):
        d = torch.zeros(t, e, device="cuda")
        d[:, c] = h
        slope = (loss(base + d) - loss(base - d)) / (2 * h)
        assert (np.abs(slope - got[:, c]) <= 5e-4 * np.abs(dwn).sum(-1) * scale).all()


def test_gradient_strides_streams_and_stray_ids(cns):
    import torch
    x = torch.randn(300, 64, device="cuda")
    wide, out = torch.full((300, 70), 3.0, device="cuda"), torch.full((300, 67), 5.0, device="cuda")
    wide[:, 3:67] = x
    r = cns.new_route(300, 64, 4, score=SIG)
    cns.run_route(r, x, sync=True)
    dw = torch.randn(300, 4, device="cuda")
    want = cns.run_route_backward(r, x, dw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = cns.run_route_backward(r, wide[:, 3:67], dw, dlogits=out[:, 1:65], stream=s)
    s.synchronize()
    assert torch.equal(got, want) and (out[:, 0] == 5).all() and (out[:, 65:] == 5).all()
    stray = r.ids.clone()
    stray[7] = torch.tensor([64, -5, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    got = cns.run_route_backward(r, x, dw, ids=stray)
    assert (got[7] == 0).all() and torch.equal(got[8:], want[8:])
