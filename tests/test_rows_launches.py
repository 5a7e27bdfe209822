"""What rows to their experts and back and the norm ask of the CUDA runtime: their host code against a stand-in for the
runtime's calls, in a process of its own.  No GPU."""
import json
import os
import subprocess
import sys

import pytest

from counted_notify_sync_gb300 import builder

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PRELUDE = """
import ctypes, json, sys
from counted_notify_sync_gb300 import _native as n
fake = ctypes.CDLL(sys.argv[1])
class Call(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("failed", ctypes.c_int), ("what", ctypes.c_void_p),
                ("n", ctypes.c_uint64), ("stream", ctypes.c_void_p)]
LAUNCH, ATTRIBUTE = 0, 1
A = [(i + 1) << 40 for i in range(12)]
def calls_of(f, s, fail=0):
    fake.fake_reset(fail)
    rc = f(s)
    got = (Call * 64)()
    return rc, [(c.kind, c.failed, c.what, c.n, c.stream) for c in got[:fake.fake_calls(got, 64)]]
def dispatch(fail=0, **kw):
    return calls_of(n.cns_dispatch, n.Dispatch(**{**dict(x_dev=A[0], rows_dev=A[1], places_dev=A[2], stream=0x50, tokens=100,
                    rows=400, row_bytes=64, top_k=4), **kw}), fail)
def combine(fail=0, **kw):
    return calls_of(n.cns_combine, n.Combine(**{**dict(rows_dev=A[0], places_dev=A[1], y_dev=A[2], stream=0x50, tokens=100,
                    rows=400, width=64, top_k=4, dtype=1), **kw}), fail)
def combine_grad(fail=0, **kw):
    return calls_of(n.cns_combine_backward, n.CombineGrad(**{**dict(rows_dev=A[0], dy_dev=A[1], places_dev=A[2], drows_dev=A[3],
                    dweights_dev=A[4], stream=0x50, tokens=100, rows=400, width=64, top_k=4, dtype=1), **kw}), fail)
def norm(fail=0, **kw):
    return calls_of(n.cns_rms_norm, n.RmsNorm(**{**dict(x_dev=A[0], y_dev=A[1], stream=0x50, rows=100, width=64, dtype=1,
                    eps=1e-6), **kw}), fail)
def norm_grad(fail=0, **kw):
    return calls_of(n.cns_rms_norm_backward, n.RmsNormGrad(**{**dict(h_dev=A[0], dy_dev=A[1], dx_dev=A[2], dgain_dev=A[3],
                    workspace_dev=A[4], workspace_bytes=1 << 40, stream=0x50, rows=100, width=64, dtype=1, eps=1e-6), **kw}), fail)
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    builder.build()
    so = tmp_path_factory.mktemp("fake") / "cudart_calls.so"
    subprocess.run(["gcc", "-std=gnu11", "-O1", "-shared", "-fPIC", "-I", os.path.join(builder.cuda_home(), "include"),
                    "-o", str(so), os.path.join(ROOT, "tests", "fakes", "cudart_calls.c")], check=True)

    def script(body):
        p = subprocess.run([sys.executable, "-c", PRELUDE + body, str(so)], cwd=ROOT, capture_output=True, text=True,
                           timeout=120, env=dict(os.environ, LD_PRELOAD=str(so)))
        assert p.returncode == 0, p.stderr
        return json.loads(p.stdout)

    return script


def test_one_launch_each_on_the_calls_stream(run):
    got = run("print(json.dumps([dispatch(), dispatch(scales_dev=A[5], row_scales_dev=A[6], scale_bytes=16), combine(), "
              "combine_grad(), norm(), norm_grad(dgain_dev=None), norm_grad(rows=1000), norm_grad(rows=3)]))")
    for i, (rc, calls) in enumerate(got):
        assert rc == 0
        assert [c[0] for c in calls] == [0] * (2 if i == 6 else 1)         # the gain's gradient is joined by a second grid,
        # where more than one CTA has a part of it
        assert all(c[4] == 0x50 for c in calls)


def test_nothing_to_do_launches_nothing(run):
    got = run("print(json.dumps([dispatch(tokens=0), dispatch(rows=0), combine(tokens=0), combine_grad(tokens=0), norm(rows=0), "
              "norm_grad(rows=0, dgain_dev=None)]))")
    assert all(rc == 0 and calls == [] for rc, calls in got)
    # without rows the base still is the result, the weights' gradient 0, the gain's gradient 0
    got = run("print(json.dumps([combine(rows=0), combine_grad(rows=0), norm_grad(rows=0)]))")
    assert all(rc == 0 and len(calls) == 1 for rc, calls in got)


def test_a_refused_launch_is_reported(run):
    got = run("print(json.dumps([dispatch(1), combine(1), combine_grad(1), norm(1), norm_grad(1, rows=1000), norm_grad(2, rows=1000)]))")
    assert all(rc != 0 for rc, _ in got)
    assert [len(calls) for _, calls in got] == [1, 1, 1, 1, 1, 2]          # no join of parts that are not there


def test_a_kernel_is_allowed_the_same_shared_memory_by_every_call(run):
    """The limit is the kernel's, and calls of other threads set it between this one's setting and its launch."""
    limits = run("""
limits = {}
for dtype in (0, 1, 2):
    for width in list(range(8, 2100, 24)) + [4096, 4104, 5000, 8192, 8193, 9000, 16384, 16385, 20480, 32768]:
        for extra in (None, A[5]):
            for rows in (1, 100000):
                got = [norm(rows=rows, width=width, dtype=dtype, residual_dev=extra, h_dev=extra and A[6]),
                       norm_grad(rows=rows, width=width, dtype=dtype, dh_dev=extra)]
                for rc, calls in got:
                    assert rc == 0, (dtype, width)
                    allowed = {}
                    for kind, _, what, size, _ in calls:
                        if kind == ATTRIBUTE:
                            limits.setdefault(what, []).append(size)
                            allowed[what] = size
                        if kind == LAUNCH:
                            assert size + 512 <= max(allowed.get(what, 0), 48 << 10), (dtype, width, size)
print(json.dumps([sorted(set(v)) for v in limits.values()]))
""")
    assert limits and all(len(v) == 1 and v[0] <= 226 << 10 for v in limits), limits
