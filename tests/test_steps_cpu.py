"""The device-wide steps without a GPU: the 64-bit oracle pinned by hand-worked rows, by brute force and by
differences, and the entry points' refusals, which come before any CUDA call."""
import ctypes
import itertools
import os
import subprocess

import numpy as np
import pytest

import counted_notify_sync_gb300 as cns
from counted_notify_sync_gb300 import _native
from oracle import steps

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INF = np.inf


@pytest.fixture(scope="module")
def built():
    cns.build()
    return _native.lib()


# --- the oracle ----------------------------------------------------------------------------------------------

def test_route_by_hand():
    x = np.array([[1.0, 3.0, 2.0, 3.0], [-INF, 0.0, -INF, -INF], [-INF] * 4])
    ids, w, s = steps.route(x, top_k=2, score=steps.SOFTMAX, renorm=True, scale=2.0)
    assert ids.tolist() == [[1, 3], [1, -1], [-1, -1]]        # equals: the lower index first; masked: none
    np.testing.assert_allclose(w, [[1.0, 1.0], [2.0, 0.0], [0.0, 0.0]])
    assert s[2].tolist() == [0.0] * 4
    # groups of two: their best logits are 3 and 3, the first group wins
    ids, _, _ = steps.route(x[:1], top_k=2, score=steps.SOFTMAX, groups=2, top_groups=1)
    assert ids.tolist() == [[1, 0]]
    # two best of each: 3 + 2 against 1 + 3 in scores
    ids, _, _ = steps.route(x[:1], top_k=2, score=steps.SIGMOID, groups=2, top_groups=1, group_top=2)
    assert ids.tolist() == [[3, 2]]
    # the bias takes part in the choice only
    ids, w, s = steps.route(x[:1], np.array([5.0, 0, 0, 0]), top_k=1, score=steps.SIGMOID, renorm=False)
    assert ids.tolist() == [[0]] and abs(w[0, 0] - 1 / (1 + np.exp(-1.0))) < 1e-15


def test_choose_against_brute_force():
    rng = np.random.RandomState(3)
    for _ in range(200):
        v = rng.randint(0, 5, size=6).astype(np.float64)
        v[rng.rand(6) < 0.2] = -INF
        k = rng.randint(1, 7)
        got = steps.choose(v, k)
        # the best ordered pick: lexicographically largest (value, -index) sequence
        picks = [p for p in itertools.permutations([i for i in range(6) if v[i] != -INF], min(k, int((v != -INF).sum())))]
        best = max(picks, key=lambda p: [(v[i], -i) for i in p])
        assert got == list(best) + [-1] * (k - len(best))


def test_plan_by_hand():
    offsets, order, places = steps.plan(np.array([[2, 0], [0, -1], [2, 1]]), 4)
    assert offsets.tolist() == [0, 2, 3, 5, 5]
    assert order.tolist() == [1, 2, 5, 0, 4, -1]
    assert places.tolist() == [[3, 0], [1, -1], [4, 2]]


@pytest.mark.parametrize("score", [steps.SIGMOID, steps.SOFTMAX])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("with_scores", [False, True])
def test_route_gradient_against_differences(score, renorm, with_scores):
    """Central differences of L = sum(dw * w) + sum(ds * scores), the chosen experts held fixed."""
    rng = np.random.RandomState(5)
    t, e, k, scale = 3, 7, 3, 1.7
    x = rng.randn(t, e)
    ids = np.array([rng.permutation(e)[:k] for _ in range(t)])
    ids[1, 2] = -1
    dw, ds = rng.randn(t, k), (rng.randn(t, e) if with_scores else None)

    def loss(z):
        total = 0.0
        for r in range(t):
            s = steps.scores(z[r], score)
            total += (dw[r] * steps.weights(z[r], s, ids[r], score, renorm, scale)).sum()
            total += (ds[r] * s).sum() if with_scores else 0.0
        return total

    got = steps.route_backward(x, ids, dw, ds, score=score, renorm=renorm, scale=scale)
    h = 1e-5
    for r in range(t):
        for c in range(e):
            d = np.zeros_like(x)
            d[r, c] = h
            assert abs((loss(x + d) - loss(x - d)) / (2 * h) - got[r, c]) < 1e-8


# --- layout and refusals ----------------------------------------------------------------------------------------

def test_structs_match_c_layout(tmp_path):
    fields = {"cns_route_t": (_native.Route, ["logits_dev", "scores_dev", "workspace_bytes", "stream", "tokens", "experts",
                                              "scale", "device_status"]),
              "cns_route_grad_t": (_native.RouteGrad, ["dlogits_dev", "tokens", "experts", "scale"]),
              "cns_tensor_t": (_native.Tensor, ["data_dev", "elems", "dtype", "reserved"]),
              "cns_grad_clip_t": (_native.GradClip, ["outs", "count", "norm_dev", "stream", "max_norm", "eps",
                                                     "device_status"])}
    lines = "".join(f'printf("{n} %zu\\n", sizeof({n}));' +
                    "".join(f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for f in fs) for n, (_, fs) in fields.items())
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text(f"#include <stdio.h>\n#include <stddef.h>\n#include \"cns.h\"\nint main(void) {{ {lines} return 0; }}\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    lay = dict(line.split() for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for n, (s, fs) in fields.items():
        assert int(lay[n]) == ctypes.sizeof(s), n
        for f in fs:
            assert int(lay[f"{n}.{f}"]) == getattr(s, f).offset, (n, f)


def good_route(**kw):
    r = _native.Route(logits_dev=0x10000, ids_dev=0x20000, weights_dev=0x30000, offsets_dev=0x40000, order_dev=0x50000,
                      places_dev=0x60000, workspace_dev=0x80000, workspace_bytes=1 << 30, tokens=8, experts=64, top_k=4,
                      dtype=0, score=0, groups=8, top_groups=4, group_top=2, renorm=1, scale=1.0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


INVALID, NULL = cns.CNS_ERR_INVALID_VALUE, cns.CNS_ERR_NULL_PTR


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), INVALID), (dict(tokens=2 ** 31 // 4), INVALID), (dict(experts=0), INVALID),
    (dict(experts=513), INVALID), (dict(top_k=0), INVALID), (dict(top_k=33), INVALID), (dict(dtype=3), INVALID),
    (dict(score=2), INVALID), (dict(groups=7), INVALID), (dict(groups=33), INVALID), (dict(top_groups=9), INVALID),
    (dict(group_top=3), INVALID), (dict(renorm=2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(top_k=9, top_groups=1), INVALID),                       # nine of a group of eight
    (dict(logits_stride=63), INVALID), (dict(logits_dev=0x10002), INVALID), (dict(bias_dev=0x70002), INVALID),
    (dict(workspace_bytes=1024), INVALID), (dict(workspace_dev=0x80040), INVALID),
    (dict(offsets_dev=None), INVALID),                            # order without offsets
    (dict(logits_dev=None), NULL), (dict(ids_dev=None), NULL), (dict(weights_dev=None), NULL),
    (dict(order_dev=None), NULL), (dict(workspace_dev=None), NULL),
])
def test_route_refusals(built, change, code):
    assert cns.cns_route(good_route(**change)) == code


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), INVALID), (dict(experts=513), INVALID), (dict(top_k=0), INVALID), (dict(dtype=-1), INVALID),
    (dict(score=5), INVALID), (dict(renorm=-1), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(logits_stride=1), INVALID), (dict(dlogits_stride=63), INVALID), (dict(dlogits_dev=0x10000), INVALID),
    (dict(dweights_dev=0x30001), INVALID), (dict(logits_dev=None), NULL), (dict(ids_dev=None), NULL),
    (dict(dweights_dev=None), NULL), (dict(dlogits_dev=None), NULL),
])
def test_route_backward_refusals(built, change, code):
    g = _native.RouteGrad(logits_dev=0x10000, ids_dev=0x20000, dweights_dev=0x30000, dlogits_dev=0x40000, tokens=8,
                          experts=64, top_k=4, dtype=0, score=0, renorm=1, scale=1.0)
    for k, v in change.items():
        setattr(g, k, v)
    assert cns.cns_route_backward(g) == code


def good_clip(tensors=((0x10000, 16, 0),), outs=None, **kw):
    g = _native.GradClip(norm_dev=0x20000, workspace_dev=0x80000, workspace_bytes=1 << 30, max_norm=1.0, eps=1e-6)
    g.table = (_native.Tensor * len(tensors))(*[_native.Tensor(*t) for t in tensors])
    g.grads, g.count = g.table, len(tensors)
    if outs is not None:
        g.out_table = (_native.Tensor * len(outs))(*[_native.Tensor(*t) for t in outs])
        g.outs = g.out_table
    for k, v in kw.items():
        setattr(g, k, v)
    return g


@pytest.mark.parametrize("make,code", [
    (lambda: good_clip(count=-1), INVALID), (lambda: good_clip(count=cns.CNS_GRAD_MAX_TENSORS + 1), INVALID),
    (lambda: good_clip(norm_type=2), INVALID), (lambda: good_clip(max_norm=-1.0), INVALID),
    (lambda: good_clip(max_norm=float("nan")), INVALID), (lambda: good_clip(eps=float("inf")), INVALID),
    (lambda: good_clip(eps=-1e-6), INVALID), (lambda: good_clip(workspace_bytes=4096), INVALID),
    (lambda: good_clip(workspace_dev=0x80010), INVALID), (lambda: good_clip(norm_dev=0x20001), INVALID),
    (lambda: good_clip([(0x10001, 16, 1)]), INVALID), (lambda: good_clip([(0x10000, -1, 0)]), INVALID),
    (lambda: good_clip([(0x10000, 16, 7)]), INVALID), (lambda: good_clip([(0x10000, 16, 0, 1)]), INVALID),
    (lambda: good_clip([(0x10000, 16, 0)], outs=[(0x20000, 15, 0)]), INVALID),
    (lambda: good_clip([(0x10000, 16, 0)], outs=[(0x10000, 16, 1)]), INVALID),      # in place, in another type
    (lambda: good_clip([(None, 16, 0)]), NULL), (lambda: good_clip(norm_dev=None), NULL),
    (lambda: good_clip(workspace_dev=None), NULL),
])
def test_grad_clip_refusals(built, make, code):
    assert cns.cns_grad_clip(make()) == code


def test_null_structs_and_workspace_sizes(built):
    L = _native.lib()
    assert L.cns_route(None) == NULL and L.cns_route_backward(None) == NULL
    assert L.cns_grad_norm(None) == NULL and L.cns_grad_clip(None) == NULL
    assert cns.cns_route_workspace_bytes(8, 64, 4, out=False)[0] == NULL
    assert cns.cns_grad_workspace_bytes(8, out=False)[0] == NULL
    assert cns.cns_route_workspace_bytes(8, 600, 4)[0] == INVALID
    assert cns.cns_grad_workspace_bytes(-1)[0] == INVALID
    rc, n = cns.cns_grad_workspace_bytes(0)
    assert rc == 0 and n >= cns.CNS_STEP_WORKSPACE_HEADER_BYTES
    assert cns.cns_grad_workspace_bytes(1000)[1] > n
    assert cns.cns_step_workspace_init(None, 1 << 20) == NULL
    assert cns.cns_step_workspace_init(0x80000, 4096) == INVALID
    assert cns.cns_step_workspace_init(0x80010, 1 << 20) == INVALID
