"""The norm's 8-bit output with scales in 32 bits, bit for bit: s = max(m / 448, 2^-126) and q = e4m3(y / s), both
quotients rounded to 32 bits, m and y the 32-bit values that the norm computes.

y is known exactly in two ways: rows of ones with eps 0 have r = 1, so that y is the gain, whatever 32-bit number that is;
and of rows in 32 bits the y that comes back is the one that the scales and values are made of."""
import numpy as np
import pytest

from oracle import steps
from test_gpu_rms_norm import check_scales, check_values, cns, host, matrix  # noqa: F401  (cns: a fixture)

pytestmark = pytest.mark.gpu

MIDDLES = (steps.E4M3[:-1] + steps.E4M3[1:]) / 2      # between neighbouring values: quotients that are ties


def codes(v):
    """e4m3 codes of 32-bit numbers, with their signs."""
    size = np.searchsorted(steps.E4M3, np.abs(steps.e4m3(np.abs(v))))
    return (size + 128 * np.signbit(v)).astype(np.uint8)


def expected(y, block):
    """(scales, codes) of rows of 32-bit numbers."""
    assert y.dtype == np.float32
    rows, width = y.shape
    step = block or width
    pad = np.zeros((rows, -width % step), np.float32)
    parts = np.abs(np.concatenate([y, pad], 1)).reshape(rows, -1, step)
    s = np.maximum(parts.max(-1) / np.float32(448.0), np.float32(2.0 ** -126))
    assert s.dtype == np.float32
    return s, codes(y / np.repeat(s, step, axis=1)[:, :width])


def blocks_of(scales, values):
    """[n, 32]: blocks with 448 * scale first, so that this is their scale, then 31 values each."""
    first = (np.float32(448.0) * scales.astype(np.float32)).reshape(-1, 1)
    return np.concatenate([first, values.astype(np.float32)], 1)


def ties():
    """Scales of few digits and values that are exactly halfway between two results, and their neighbours."""
    rng = np.random.RandomState(1)
    s = np.concatenate([np.arange(1, 2000, 2), rng.randint(1, 2 ** 16, 1000)]).astype(np.float64) * \
        2.0 ** rng.randint(-40, 40, 2000)
    v = s[:, None] * rng.choice(MIDDLES, (2000, 31))
    v = v.astype(np.float32)
    by = rng.randint(-1, 2, v.shape)
    v = np.where(by == 0, v, np.nextafter(v, np.where(by < 0, -np.inf, np.inf).astype(np.float32)))
    return blocks_of(s, v * rng.choice([-1.0, 1.0], v.shape))


def near_ties():
    """Scales close to those of few digits, values closest to a tie: quotients next to where 32 bits round to the tie."""
    rng = np.random.RandomState(2)
    off = np.concatenate([rng.randint(-9, 10, 2000), rng.randint(-600, 601, 2000)])
    s = (rng.randint(8, 17, 4000) * 2.0 ** 20 + off) * 2.0 ** rng.randint(-60, 20, 4000)
    s = s.astype(np.float32).astype(np.float64)
    v = (s[:, None] * rng.choice(MIDDLES, (4000, 31)) * (1 + rng.choice([0, 2.0 ** -25, -2.0 ** -25, 2.0 ** -24, -2.0 ** -24], (4000, 31))))
    v = v.astype(np.float32)
    by = rng.randint(-1, 2, v.shape)
    v = np.where(by == 0, v, np.nextafter(v, np.where(by < 0, -np.inf, np.inf).astype(np.float32)))
    return blocks_of(s, v * rng.choice([-1.0, 1.0], v.shape))


def all_exponents():
    """Largest values from the least subnormal to the largest number, zeros of both signs among the others."""
    rng = np.random.RandomState(3)
    m = np.ldexp(1 + rng.rand(6000), rng.randint(-150, 128, 6000)).astype(np.float32)
    m[:254] = np.ldexp(np.float32(1.75), np.arange(-127, 127))
    v = (m[:, None].astype(np.float64) * 2.0 ** (-12 * rng.rand(6000, 31)) * rng.choice([-1.0, 1.0], (6000, 31))).astype(np.float32)
    v = np.where(np.abs(v) > m[:, None], m[:, None], v)
    v[::7, 3], v[::7, 4] = 0.0, -0.0
    m[100:103] = 0.0
    v[100:103] *= 0.0
    return np.concatenate([m[:, None], v], 1)


def hand_picked():
    """y = 175 with s = 7: 25, halfway between 24 and 26, so 24."""
    b = np.zeros((8, 32), np.float32)
    for i, (s, y) in enumerate([(7, 175), (7, -175), (7, 161), (11, 187), (13, 299), (19, 475), (1537, 1537 * 27), (3, 51)]):
        b[i, 0], b[i, 1], b[i, 2] = 448 * s, y, -y
    return b


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("what", [hand_picked, ties, near_ties, all_exponents])
def test_quotients_are_rounded_once(cns, what, shift, dtype):  # noqa: F811
    """Rows of ones: y is the gain."""
    import torch
    blocks = what()
    for width in (64, 1024, 8192):
        flat = blocks.reshape(-1)
        flat = np.concatenate([flat, np.zeros(-len(flat) % width, np.float32)])
        n = cns.new_rms_norm(width, eps=0.0, scale_block=32)
        x = matrix(np.random.RandomState(0), 1, width, dtype, 0, shift)
        x.fill_(1.0)
        for at in range(0, len(flat), width)[:24] if width < 8192 else range(0, len(flat), width):
            y = flat[at:at + width]
            gain = torch.from_numpy(y).cuda()
            _, back, q, s = cns.run_rms_norm(n, x, gain)
            if dtype == "f32":
                assert np.array_equal(back.cpu().numpy().view(np.uint32)[0], y.view(np.uint32))
            want_s, want_q = expected(y.reshape(1, -1), 32)
            assert np.array_equal(s.cpu().numpy().view(np.uint32), want_s.view(np.uint32))
            assert np.array_equal(q.view(torch.uint8).cpu().numpy(), want_q)


@pytest.mark.parametrize("width", [24, 64, 100, 520, 1000, 2049, 4096, 8192, 9000, 20480])
@pytest.mark.parametrize("block", [0, 32, 64, 128])
@pytest.mark.parametrize("residual", [False, True])
def test_scales_and_values_are_those_of_y(cns, width, block, residual):  # noqa: F811
    """Rows in 32 bits with gains of few digits, whose quotients often are ties."""
    import torch
    rng = np.random.RandomState(width + block)
    x, more = matrix(rng, 33, width, "bf16").float(), matrix(rng, 33, width, "bf16").float()
    gain = matrix(rng, 1, width, "bf16")[0].float()
    n = cns.new_rms_norm(width, scale_block=block)
    _, y, q, s = cns.run_rms_norm(n, x, gain, residual=more if residual else None)
    want_s, want_q = expected(y.cpu().numpy(), block)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), want_s.view(np.uint32))
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), want_q)
    # without y another number of threads may take a row, so r may differ in its last bits: the tolerances of test_gpu_rms_norm
    n = cns.new_rms_norm(width, y=False, scale_block=block)
    h, none, q, s = cns.run_rms_norm(n, x, gain, residual=more if residual else None)
    want = steps.rms_norm(host(h), host(gain), 1e-6)
    assert none is None
    check_scales(host(s), want, block, False)
    check_values(host(q.float()), host(s), want, block)
