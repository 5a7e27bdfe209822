"""What the training-step operators ask of the CUDA runtime, and what they leave when it refuses: their host code
against a stand-in for the runtime's calls, in a process of its own.  No GPU."""
import json
import os
import subprocess
import sys

import pytest

from counted_notify_sync_gb300 import builder

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# run in the process with the stand-in: `route` makes one call (its code, the runtime's calls)
PRELUDE = """
import ctypes, json, sys
from counted_notify_sync_gb300 import _native as n
fake = ctypes.CDLL(sys.argv[1])
class Call(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("failed", ctypes.c_int), ("what", ctypes.c_void_p),
                ("n", ctypes.c_uint64), ("stream", ctypes.c_void_p)]
LAUNCH, ATTRIBUTE, MEMSET = 0, 1, 2
HEADER = 1 << 20
def route(tokens, experts, top_k, fail=0, **kw):
    r = n.Route(logits_dev=1 << 32, ids_dev=2 << 32, weights_dev=3 << 32, offsets_dev=4 << 32, order_dev=5 << 32,
                places_dev=6 << 32, workspace_dev=7 << 32, workspace_bytes=1 << 30, tokens=tokens, experts=experts,
                top_k=top_k, dtype=0, score=1, renorm=1, scale=1.0, stream=0x50)
    for k, v in kw.items():
        setattr(r, k, v)
    fake.fake_reset(fail)
    rc = n.cns_route(r)
    got = (Call * 64)()
    return rc, [(c.kind, c.failed, c.what, c.n, c.stream) for c in got[:fake.fake_calls(got, 64)]]
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    lib = builder.build()
    so = tmp_path_factory.mktemp("fake") / "cudart_calls.so"
    subprocess.run(["gcc", "-std=gnu11", "-O1", "-shared", "-fPIC", "-I", os.path.join(builder.cuda_home(), "include"),
                    "-o", str(so), os.path.join(ROOT, "tests", "fakes", "cudart_calls.c")], check=True)
    assert os.path.exists(lib)

    def script(body):
        p = subprocess.run([sys.executable, "-c", PRELUDE + body, str(so)], cwd=ROOT, capture_output=True, text=True,
                           timeout=120, env=dict(os.environ, LD_PRELOAD=str(so)))
        assert p.returncode == 0, p.stderr
        return json.loads(p.stdout)

    return script


def test_a_plan_that_is_refused_leaves_the_workspace_as_it_was(run):
    """The first grid adds to the blocks' sums, which the second one clears.  If the runtime refuses that one, the
    sums are cleared behind the first, on its stream; a refusal of the first leaves nothing to clear."""
    rc, calls = run("print(json.dumps(route(5000, 64, 4, fail=2)))")
    assert rc == -7 or rc != 0
    launches = [i for i, c in enumerate(calls) if c[0] == 0]
    assert [calls[i][1] for i in launches] == [0, 1]
    after = [c for c in calls[launches[-1] + 1:] if c[0] == 2]
    sums = 4 * 10 * 512                             # 10 blocks of CTAs, 512 experts
    at = (7 << 32) + 233472 - sums                  # the end of the header
    assert after == [[2, 0, at, sums, 0x50]]
    rc, calls = run("print(json.dumps(route(5000, 64, 4, fail=1)))")
    assert rc != 0 and [c[0] for c in calls] == [0]
    rc, calls = run("print(json.dumps(route(5000, 64, 4)))")
    assert rc == 0 and [c[0] for c in calls] == [0, 0]


def test_a_kernel_is_allowed_the_same_shared_memory_by_every_call(run):
    """The limit is the kernel's, and calls of other threads set it between this one's setting and its launch: a
    smaller call must not lower it."""
    limits = run("""
limits = {}
for score in (0, 1):
    for groups, top_groups, group_top in ((1, 1, 1), (4, 2, 1), (4, 2, 2)):
        for experts in (512, 480, 420, 384, 360, 320, 256, 128, 64, 8):
            for tokens in (1, 4, 32, 33, 5000):
                for plan in (True, False):
                    kw = {} if plan else dict(offsets_dev=None, order_dev=None, places_dev=None)
                    rc, calls = route(tokens, experts, 2, score=score, groups=groups, top_groups=top_groups,
                                      group_top=group_top, **kw)
                    assert rc == 0
                    allowed = {}
                    for kind, _, what, size, _ in calls:
                        if kind == ATTRIBUTE:
                            limits.setdefault(what, []).append(size)
                            allowed[what] = size
                        if kind == LAUNCH:
                            assert size <= allowed.get(what, 48 << 10)
print(json.dumps([sorted(set(v)) for v in limits.values()]))
""")
    assert limits and all(len(v) == 1 and v[0] <= 227 << 10 for v in limits), limits
