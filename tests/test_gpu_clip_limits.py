"""Clipping at its limits.  Where the quotient max_norm / (norm + eps) has no value: an unlimited norm (max_norm = inf, the default),
a norm that overflowed, and zero over zero: only a norm of NaN makes NaN of numbers.  And layouts that are alike
though their strides are not."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def cns():
    import torch
    import counted_notify_sync_gb300 as c
    c.build()
    torch.cuda.set_device(0)
    return c


@pytest.mark.parametrize("norm_type", [0, 1])
@pytest.mark.parametrize("n", [100, 3_000_000])
@pytest.mark.parametrize("other", [False, True])
def test_without_a_limit_nothing_changes(cns, norm_type, n, other):
    import torch
    for poison in (INF, -INF, 3e20):                # of 3e20 the squares overflow: the L2 norm is inf
        g = torch.randn(n, device="cuda")
        g[n // 3] = poison
        before = g.clone()
        out = torch.zeros_like(g) if other else g
        norm = cns.run_grad_clip(cns.new_grad_clip([g], norm_type=norm_type, outs=[out] if other else None), sync=True)
        assert norm.item() == (INF if norm_type == 0 else np.float32(abs(poison)))
        assert torch.equal(out.view(torch.int32), before.view(torch.int32))


@pytest.mark.parametrize("max_norm", [INF, 1.0, 0.0])
def test_a_nan_shows_whatever_the_limit(cns, max_norm):
    import torch
    g = torch.ones(5000, device="cuda")
    g[7] = NAN
    assert torch.isnan(cns.run_grad_clip(cns.new_grad_clip([g], max_norm), sync=True))
    assert torch.isnan(g).all()


def test_a_limit_and_a_norm_of_zero(cns):
    import torch
    g = torch.zeros(5000, device="cuda")
    assert cns.run_grad_clip(cns.new_grad_clip([g], 0.0, eps=0.0), sync=True).item() == 0.0
    assert (g == 0).all()


def test_a_finite_limit_makes_an_infinite_norm_zeros(cns):
    import torch
    for limit in (0.0, 1.0, 3e38):
        g = torch.ones(5000, device="cuda")
        g[:10] = 3e20
        out = torch.ones_like(g)
        assert cns.run_grad_clip(cns.new_grad_clip([g], limit, outs=[out]), sync=True).item() == INF
        assert (out == 0).all()


def test_strides_along_axes_of_one_do_not_matter(cns):
    """A 1 x 1 convolution's weights, channels last and not, lie the same way."""
    import torch
    g = torch.as_strided(torch.randn(40 * 24, device="cuda"), (40, 24, 1, 1), (24, 1, 24, 24))
    out = torch.empty((40, 24, 1, 1), device="cuda")
    assert g.stride() != out.stride()
    norm = cns.run_grad_clip(cns.new_grad_clip([g], 1.0, outs=[out]), sync=True).cpu()
    assert torch.equal(out.cpu(), g.cpu() * (torch.tensor(1.0) / (norm + torch.tensor(1e-6))))
    with pytest.raises(ValueError, match="strides"):
        cns.new_grad_clip([torch.zeros(6, 4, device="cuda").t()], 1.0, outs=[torch.zeros(4, 6, device="cuda")])
