"""The routing's gradient at experts that were not chosen, by the size of each value itself.

Rows hold their largest logit, 0, last, and all others 12 to 80 below it on a grid of 1/8: l - top is exact, and the
softmax's sum is 1 and at most 512 e^-12 = 3.2e-3 beside it.

Bounds, in units of u = 2^-24.  expf is within 2 units in the last place: 4.
  The sum: 1, then at most 5 additions across lanes; the small terms' own roundings are below
2 * 3.2e-3 * 100 = 1: 6 in all.
  A chosen score p: 4 of expf, 6 of the sum, 1 of the quotient: 11.
  softmax, not renormalised: the gradient is -p_e * sum_i p_i g_i.  g = scale * dw rounds once, p g once, and
terms of one sign are added at most 5 times: the inner sum is within 11 + 2 + 5 = 18.  p_e takes expf 4, the sum 6, its
reciprocal 1 and the product 1; the product with the inner sum 1: 13.  Together 31.
  softmax with dL/dscores = 1 at the largest and -1 elsewhere: p_e (h_e - mean) with mean = sum_i p_i h_i, which is
1 - 6.4e-3 at least: within 4 + 6 + 5 (its additions) + 1 (quotient) + 1 (the small terms) = 17, so h_e - mean, near
-2, within 10; with dweights the chosen ones' inner sum comes on top.  13 + 10 and a spare: 24.
  sigmoid with dL/dscores: s (1 - s) h = r (ex r) h: expf 4, 1 + ex 1 + 4 ex / (1 + ex) (2 at most), r 1, twice that of
r, and three products: 4 + 2 (2 + 1 + 1) + 3 = 15."""
import numpy as np
import pytest

from oracle import steps

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def cns():
    import torch
    import counted_notify_sync_gb300 as c
    c.build()
    torch.cuda.set_device(0)
    return c


# 8 lanes a token with rows in registers and read again, 32 lanes, elements one at a time
SHAPES = [(160, 6), (256, 8), (384, 8), (512, 20), (99, 4)]


def rows(tokens, experts, top_k, seed):
    """Logits, and ids that hold the largest and top_k - 1 others."""
    rng = np.random.RandomState(seed)
    x = -rng.randint(96, 641, size=(tokens, experts)) / 8.0
    x[:, -1] = 0.0
    ids = np.array([[experts - 1, *rng.permutation(experts - 1)[:top_k - 1]] for _ in range(tokens)], dtype=np.int32)
    return x, ids


def gradient(cns, x, ids, dw, ds=None, **kw):
    import torch
    r = cns.new_route(*x.shape, ids.shape[1], plan=False, **kw)
    d = cns.run_route_backward(r, torch.from_numpy(x).float().cuda(), torch.from_numpy(dw).cuda(),
                               ids=torch.from_numpy(ids).cuda(),
                               dscores=None if ds is None else torch.from_numpy(ds).cuda())
    return d.cpu().double().numpy()


def unchosen(ids, experts):
    free = np.ones((len(ids), experts), dtype=bool)
    np.put_along_axis(free, ids.astype(np.int64), False, 1)
    return free


@pytest.mark.parametrize("experts,top_k", SHAPES)
def test_softmax_that_is_not_renormalised(cns, experts, top_k):
    x, ids = rows(400, experts, top_k, seed=experts)
    dw = (1.0 + np.random.RandomState(1).rand(400, top_k)).astype(np.float32)
    got = gradient(cns, x, ids, dw, score=steps.SOFTMAX, renorm=False, scale=2.5)
    want = steps.route_backward(x, ids, dw, score=steps.SOFTMAX, renorm=False, scale=2.5)
    free = unchosen(ids, experts)
    off = np.abs(got - want)[free] / np.abs(want)[free]
    assert off.max() <= 31 * U, off.max() / U


@pytest.mark.parametrize("experts,top_k", SHAPES)
@pytest.mark.parametrize("renorm", [False, True])
def test_softmax_scores(cns, experts, top_k, renorm):
    x, ids = rows(400, experts, top_k, seed=experts + 1)
    dw = np.zeros((400, top_k), dtype=np.float32)
    ds = -np.ones(x.shape, dtype=np.float32)
    ds[:, -1] = 1.0
    got = gradient(cns, x, ids, dw, ds, score=steps.SOFTMAX, renorm=renorm)
    want = steps.route_backward(x, ids, dw, ds, score=steps.SOFTMAX, renorm=renorm, scale=1.0)
    free = unchosen(ids, experts)
    off = np.abs(got - want)[free] / np.abs(want)[free]
    assert off.max() <= 24 * U, off.max() / U


@pytest.mark.parametrize("experts,top_k", SHAPES)
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_sigmoid_scores(cns, experts, top_k, sign):
    x, ids = rows(400, experts, top_k, seed=experts + 2)
    x = sign * x
    dw = np.zeros((400, top_k), dtype=np.float32)
    ds = np.random.RandomState(2).randn(*x.shape).astype(np.float32)
    got = gradient(cns, x, ids, dw, ds, score=steps.SIGMOID, renorm=False)
    # s (1 - s) without cancellation: e^-|x| / (1 + e^-|x|)^2
    ex = np.exp(-np.abs(x))
    want = ex / (1.0 + ex) ** 2 * ds.astype(np.float64)
    free = unchosen(ids, experts)
    off = np.abs(got - want)[free] / np.abs(want)[free]
    assert off.max() <= 15 * U, off.max() / U


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", [steps.SIGMOID, steps.SOFTMAX])
def test_what_no_gradient_reaches_is_zero(cns, dtype, score):
    """Exactly, and of either sign."""
    import torch
    x = torch.randn(300, 160, device="cuda").to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype])
    ids = torch.rand(300, 160, device="cuda").argsort(-1)[:, :6].int().contiguous()
    r = cns.new_route(300, 160, 6, score=score, plan=False)
    d = cns.run_route_backward(r, x, torch.randn(300, 6, device="cuda"), ids=ids, dlogits=torch.full_like(x, 7.0))
    free = torch.ones(300, 160, dtype=torch.bool, device="cuda").scatter_(1, ids.long(), False)
    assert (d[free].abs().max() == 0) and (d[~free] != 0).any()
