"""y = h * r * gain in this order: h * r is no larger than the root of the width, so a y that 32 bits can hold is not
lost to a product on the way, however large or small h and the gain are."""
import numpy as np
import pytest

from oracle import steps
from test_gpu_rms_norm import HALF, TINY, U, check_scales, check_values, cns, host, matrix, scale_values, types  # noqa: F401

pytestmark = pytest.mark.gpu

# (rows' type, size of h, size of the gain, eps): the products h * gain are past 2^128, or below 2^-126
FAR = [("f32", 1e18, 1e21, 1e-6), ("f32", 1e-15, 1e-27, 0.0), ("f32", 3e17, 1e34, 0.0), ("bf16", 1e18, 1e21, 1e-6),
       ("bf16", 1e-15, 1e-27, 0.0), ("f16", 6e4, 1e35, 1e-6), ("f16", 1e-4, 1e-36, 0.0), ("f32", 5e16, 3e22, 0.0),
       ("bf16", 5e16, 3e22, 0.0)]


@pytest.mark.parametrize("dtype,size,gain_size,eps", FAR)
@pytest.mark.parametrize("width", [7, 128, 1000, 4096, 16384, 20480])
def test_large_and_small_products(cns, dtype, size, gain_size, eps, width):  # noqa: F811
    import torch
    rng = np.random.RandomState(width)
    x = torch.from_numpy((rng.choice([-1.0, 1.0], (5, width)) * rng.uniform(0.5, 1.0, (5, width)) * size).astype(np.float32)).to(types()[dtype]).cuda()
    gain = torch.from_numpy((rng.uniform(0.5, 1.0, width) * gain_size).astype(np.float32)).cuda()
    want = steps.rms_norm(host(x), host(gain), eps)
    squares = (host(x) ** 2).sum(-1)
    assert (np.abs(squares / np.finfo(np.float32).max - 1) > 1e-3).all()
    want[squares > np.finfo(np.float32).max] = 0.0     # r is 0 where 32 bits do not hold the sum of the squares
    assert np.isfinite(want.astype(np.float32)).all()
    for block, power in ((None, False), (0, False), (0, True), (32, False), (128, True)):
        # where the rows' type has no number for y, its 8-bit form has
        n = cns.new_rms_norm(width, eps=eps, y=dtype != "f16" or block is None, scale_block=block,
                             scale_type=cns.CNS_SCALE_E8M0 if power else cns.CNS_SCALE_F32)
        _, y, q, s = cns.run_rms_norm(n, x, gain)
        if dtype != "f16":
            assert (np.abs(host(y) - want) <= (41 * U + HALF[dtype] * (1 + 1e-5)) * np.abs(want) + TINY[dtype]).all()
        if block is not None:
            check_scales(scale_values(s), want, block, power)
            check_values(host(q.float()), scale_values(s), want, block)


@pytest.mark.parametrize("width", [64, 4096, 20480])
def test_a_row_whose_squares_overflow_is_zeros(cns, width):  # noqa: F811
    """r is 0 then, and y = h * r * gain, whatever h * gain would be."""
    import torch
    x = torch.full((3, width), 1e20, device="cuda")
    x[1] = 1.0
    gain = torch.full((width,), 1e25, device="cuda")
    for block in (0, 32):
        n = cns.new_rms_norm(width, scale_block=block)
        _, y, q, s = cns.run_rms_norm(n, x, gain)
        for row in (0, 2):
            assert (y[row] == 0).all() and (q[row].float() == 0).all() and (s[row] == 2.0 ** -126).all()
        assert ((y[1] / 1e25 - 1).abs() < 1e-5).all()
