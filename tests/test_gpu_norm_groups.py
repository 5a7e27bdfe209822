"""The norm's gradient where several groups of 64 or 96 threads share a CTA (513 to 1536 columns of 16 bits, 257 to 768 of
32): every group's rows against the definition in 64 bits, and the same bits whichever results a call asks for."""
import numpy as np
import pytest

from oracle import steps
from test_gpu_rms_norm import EPS, HALF, TINY, U, cns, host, matrix  # noqa: F401  (cns: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width,dtype", [(513, "bf16"), (776, "f16"), (1024, "bf16"), (1025, "f16"), (1400, "bf16"), (1536, "f16"),
                                         (257, "f32"), (512, "f32"), (513, "f32"), (700, "f32"), (768, "f32")])
@pytest.mark.parametrize("rows", [1, 2, 5, 17, 3001])
def test_each_groups_rows(cns, width, dtype, rows):  # noqa: F811
    """The tolerances are those of test_gpu_rms_norm: 200 roundings of dx's parts, one of its type; a rounding a row and
    44 of each product of dgain."""
    import torch
    rng = np.random.RandomState(width + rows)
    h, dy, dh = (matrix(rng, rows, width, dtype, 0, 0, k) for k in (2.0, 1.0, 0.5))
    n = cns.new_rms_norm(width, eps=EPS)
    for gain, use_dh in ((None, False), (None, True), (matrix(rng, 1, width, "f32")[0], True)):
        also = dh if use_dh else None
        want, want_gain, size, size_gain = steps.rms_norm_backward(host(h), None if gain is None else host(gain), host(dy),
                                                                   None if also is None else host(also), EPS)
        dgain = torch.empty(width, device="cuda")
        dx, got = cns.run_rms_norm_backward(n, h, gain, dy, dh=also, dgain=dgain)
        assert got is dgain
        assert (np.abs(host(dx) - want) <= 200 * U * size + HALF[dtype] * np.abs(want) * (1 + 1e-5) + TINY[dtype]).all()
        assert (np.abs(host(dgain) - want_gain) <= (rows + 44) * U * size_gain).all()
        # without the gain's gradient, with or without a gain
        alone, none = cns.run_rms_norm_backward(n, h, gain, dy, dh=also, dgain=False)
        assert none is None and torch.equal(alone, dx)
        again, dgain_again = cns.run_rms_norm_backward(n, h, gain, dy, dh=also, dgain=torch.empty_like(dgain))
        assert torch.equal(again, dx) and torch.equal(dgain_again, dgain)
