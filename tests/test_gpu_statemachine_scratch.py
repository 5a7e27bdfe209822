"""cns_statemachine_run on scratch that holds anything: its link words are told from what else was in that memory."""
import numpy as np
import pytest

import cns_inputs as ci
import oracle
from tests.gpu_helpers import from_dev_u32, to_dev_u32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cns():
    import torch
    import counted_notify_sync_gb300 as c
    c.build()
    torch.cuda.set_device(0)
    return c


def adds(n):
    """A stream of adds alone: every tile's counts depend on the tile before it."""
    ops = np.zeros((n, 4), dtype=np.uint32)
    ops[:, 1] = 1
    ops[:, 2] = np.random.RandomState(n).randint(1, 1 << 20, size=n)
    return ops


def words(scratch):
    return scratch.cpu().numpy().view(np.uint64)


@pytest.mark.parametrize("make", [ci.notify_ops, adds])
@pytest.mark.parametrize("n", [5000, 200_000, 1_300_000])
def test_what_earlier_calls_and_others_left(cns, make, n):
    import torch
    ops = make(n)
    want_t, want_f = oracle.cnt_statemachine(ops, 3)
    d = to_dev_u32(ops)
    sb = cns.cns_statemachine_scratch_bytes(n)
    scratch = torch.zeros(sb // 4, dtype=torch.int32, device="cuda")

    def run(content=None):
        if content is not None:
            scratch.copy_(torch.from_numpy(np.ascontiguousarray(content).view(np.int32)))
        trace, final = torch.zeros((n, 2), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        cns.check(cns.cns_statemachine_run(d, n, 3, trace, final, scratch, sb, None))
        torch.cuda.synchronize()
        np.testing.assert_array_equal(from_dev_u32(trace), want_t)
        assert int(from_dev_u32(final)[0]) == want_f

    def last_line():
        """The line that a call leaves behind (its last tile's)."""
        w = words(scratch).reshape(-1, 16)
        used = np.nonzero(w.any(axis=1))[0]
        assert used.size
        return w[used[-1]]

    run()
    lines = sb // 128
    for step in (0, 1, 2):
        # every line as the last call's, and as calls after it would have it if they counted up
        scratch.zero_()
        run()
        line = last_line().copy()
        there = line != 0
        line[there] = ((line[there] >> np.uint64(32)) + np.uint64(step)) << np.uint64(32) | np.uint64(0x4136cb55)
        run(np.tile(line, lines))
    # exchanges of other workspaces ({count of calls, float}), traces ({count, outcome}), ones
    for high in range(1, 9):
        run(np.full(lines * 16, high << 32 | 0x4136cb55, dtype=np.uint64))
    run(np.full(lines * 16, (1 << 64) - 1, dtype=np.uint64))


def test_after_a_clipping_in_the_same_memory(cns):
    """Workspaces that torch hands out again as scratch."""
    import torch
    ops = ci.notify_ops(1_000_000)
    want_t, want_f = oracle.cnt_statemachine(ops, 0)
    d = to_dev_u32(ops)
    g = torch.randn(300_000, device="cuda")
    for _ in range(12):
        handles = [cns.new_grad_clip([g], 1e30) for _ in range(6)]
        for h in handles:
            for _ in range(12):
                cns.run_grad_clip(h)
        torch.cuda.synchronize()
        del handles, h
        trace, final = cns.run_statemachine(d, 0)
        np.testing.assert_array_equal(from_dev_u32(trace), want_t)
        assert int(from_dev_u32(final)[0]) == want_f
