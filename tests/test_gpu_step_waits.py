"""The exchange's bounded wait (step_device.cuh) by one CTA whose partners never send: it gives up, says so in the
workspace's status, and the workspace refuses calls until it is initialised again."""
import ctypes
import os
import subprocess
import time

import numpy as np
import pytest

from counted_notify_sync_gb300 import builder

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def cns():
    import torch
    import counted_notify_sync_gb300 as c
    c.build()
    torch.cuda.set_device(0)
    return c


@pytest.fixture(scope="module")
def step_wait(tmp_path_factory):
    """step_wait(header, sent, ctas, tag, timeout in ms): (gave up, the values)."""
    import torch
    so = tmp_path_factory.mktemp("waits") / "step_waits.so"
    subprocess.run([os.path.join(builder.cuda_home(), "bin", "nvcc"), *builder.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-shared", "-cudart", "shared", "-I", builder.INCLUDE, "-I", builder.CSRC, "-o", str(so),
                    os.path.join(HERE, "fused", "step_waits.cu")], check=True)
    fn = ctypes.CDLL(str(so)).step_wait
    fn.argtypes = [ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_void_p,
                   ctypes.c_void_p]

    def call(ws, sent, ctas, tag, ms):
        out = torch.zeros(161, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        assert fn(ws.data_ptr(), sent, ctas, tag, int(ms * 1e6), out.data_ptr(), None) == 0
        got = out.cpu().numpy()
        return bool(got[0]), got[1:1 + ctas]

    return call


def test_a_wait_ends_when_all_have_sent(cns, step_wait):
    for ctas in (1, 31, 33, 152, 160):
        ws = cns.new_step_workspace(1)
        stop, values = step_wait(ws, ctas, ctas, 5, 500)
        assert not stop and np.array_equal(values, 100 + np.arange(ctas))
        assert cns.syncall_read_workspace(ws)[3] == 0


@pytest.mark.parametrize("sent,ctas", [(0, 1), (1, 2), (151, 152), (32, 33)])
def test_a_wait_for_what_nobody_sends_gives_up(cns, step_wait, sent, ctas):
    import torch
    g = torch.ones(3_000_000, device="cuda")
    plan = cns.new_grad_clip([g], 1.0)
    at = time.monotonic()
    stop, _ = step_wait(plan.workspace, sent, ctas, 9, 20)
    assert stop and 0.015 < time.monotonic() - at < 2
    assert cns.syncall_read_workspace(plan.workspace)[3] == cns.CNS_ERR_TIMEOUT
    with pytest.raises(cns.CnsError) as e:
        cns.run_grad_clip(plan, sync=True)
    assert e.value.code == cns.CNS_ERR_TIMEOUT and (g == 1).all()
    cns.check(cns.cns_step_workspace_init(plan.workspace, plan.workspace.numel() * 4))
    assert abs(cns.run_grad_clip(plan, sync=True).item() / 3e6 ** 0.5 - 1) < 4.1e-6


def test_a_wait_ends_early_when_another_one_gave_up(cns, step_wait):
    ws = cns.new_step_workspace(1)
    ws[32], ws[33] = cns.CNS_ERR_TIMEOUT, 1
    at = time.monotonic()
    stop, _ = step_wait(ws, 0, 2, 3, 900)
    assert stop and time.monotonic() - at < 0.5


def test_words_of_other_calls_are_not_taken(cns, step_wait):
    """Boxes that show an older tag are waited for."""
    ws = cns.new_step_workspace(1)
    assert not step_wait(ws, 4, 4, 7, 500)[0]
    assert step_wait(ws, 3, 4, 8, 20)[0]
