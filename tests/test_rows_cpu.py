"""Rows to their experts and back and the root-mean-square norm without a GPU: the 64-bit oracle pinned by hand-worked
rows and by differences, the entry points' refusals, which come before any CUDA call, and the Python side's."""
import ctypes
import os
import struct
import subprocess

import numpy as np
import pytest

import counted_notify_sync_gb300 as cns
from counted_notify_sync_gb300 import _native
from oracle import steps

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, NULL = cns.CNS_ERR_INVALID_VALUE, cns.CNS_ERR_NULL_PTR


@pytest.fixture(scope="module")
def built():
    cns.build()
    return _native.lib()


# --- the oracle ----------------------------------------------------------------------------------------------

PLACES = np.array([[2, 0], [-1, 1], [3, 7], [-1, -1]])


def test_rows_by_hand():
    x = np.arange(8.0).reshape(4, 2)
    rows = steps.dispatch(x, PLACES, np.full((5, 2), -9.0))
    assert rows.tolist() == [[0, 1], [2, 3], [0, 1], [4, 5], [-9, -9]]       # 7 is outside; row 4 has no place
    w = np.array([[2.0, 3.0], [5.0, 7.0], [11.0, 13.0], [1.0, 1.0]])
    y, _ = steps.combine(rows, PLACES, w, base=np.ones((4, 2)))
    assert y.tolist() == [[1, 6], [15, 22], [45, 56], [1, 1]]
    assert steps.combine(rows, PLACES)[0].tolist() == [[0, 2], [2, 3], [4, 5], [0, 0]]
    drows, dw, _ = steps.combine_backward(rows, x, PLACES, w, drows=np.full((5, 2), -9.0))
    assert drows.tolist() == [[0, 3], [14, 21], [0, 2], [44, 55], [-9, -9]]
    assert dw.tolist() == [[1, 1], [0, 13], [41, 0], [0, 0]]


def test_row_gradients_against_differences():
    rng = np.random.RandomState(2)
    rows, w, dy = rng.randn(5, 3), rng.rand(4, 2), rng.randn(4, 3)
    drows, dw, _ = steps.combine_backward(rows, dy, PLACES, w)
    loss = lambda r, v: (steps.combine(r, PLACES, v)[0] * dy).sum()  # noqa: E731
    step = 1e-5
    for at in np.ndindex(rows.shape):
        d = np.zeros_like(rows)
        d[at] = step
        assert abs((loss(rows + d, w) - loss(rows - d, w)) / (2 * step) - drows[at]) < 1e-8
    for at in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[at] = step
        assert abs((loss(rows, w + d) - loss(rows, w - d)) / (2 * step) - dw[at]) < 1e-8
    # a dispatch's gradient is a combine without weights
    x, g = rng.randn(4, 3), rng.randn(5, 3)
    dx, _ = steps.combine(g, PLACES)
    for at in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[at] = step
        moved = lambda z: (steps.dispatch(z, PLACES, np.zeros((5, 3))) * g).sum()  # noqa: E731
        assert abs((moved(x + d) - moved(x - d)) / (2 * step) - dx[at]) < 1e-8


def test_norm_by_hand_and_against_differences():
    y = steps.rms_norm([[3.0, 4.0, 0.0, 0.0]], [1.0, 2.0, 3.0, 4.0], eps=0.0)
    np.testing.assert_allclose(y, [[1.2, 3.2, 0.0, 0.0]])
    np.testing.assert_allclose(steps.rms_norm([[0.0, 0.0]], eps=1e-6), 0.0)
    rng = np.random.RandomState(4)
    h, gain, dy, dh = rng.randn(3, 5), rng.rand(5) + 0.5, rng.randn(3, 5), rng.randn(3, 5)
    dx, dgain, _, _ = steps.rms_norm_backward(h, gain, dy, dh, eps=0.1)
    loss = lambda z, v: (steps.rms_norm(z, v, 0.1) * dy).sum() + (z * dh).sum()  # noqa: E731
    step = 1e-5
    for at in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[at] = step
        assert abs((loss(h + d, gain) - loss(h - d, gain)) / (2 * step) - dx[at]) < 1e-8
    for at in range(5):
        d = np.zeros(5)
        d[at] = step
        assert abs((loss(h, gain + d) - loss(h, gain - d)) / (2 * step) - dgain[at]) < 1e-8


def test_eight_bits_by_hand():
    assert steps.E4M3[-1] == 448.0 and steps.E4M3[1] == 2.0 ** -9 and steps.E4M3[8] == 2.0 ** -6
    assert steps.e4m3([1.0, -1.0625, 1.1875, 1.06, 500.0, 2.0 ** -10, 3 * 2.0 ** -10, 0.0]).tolist() == \
        [1.0, -1.0, 1.25, 1.0, 448.0, 0.0, 2.0 ** -8, 0.0]
    y = np.array([[448.0, 1.0, -7.0, 3.5, 449.0, 0.0]])
    assert steps.scales(y, 2)[0].tolist() == [1.0, 7 / 448, 449 / 448]
    assert steps.scales(y, 2, power=True)[0].tolist() == [1.0, 2.0 ** -6, 2.0]
    assert steps.scales(y, 4, power=True)[0].tolist() == [1.0, 2.0]
    assert steps.scales(np.zeros((1, 2)), 0)[0].tolist() == [2.0 ** -126]
    assert steps.scales(np.zeros((1, 2)), 0, power=True)[0].tolist() == [2.0 ** -127]
    assert np.isnan(steps.scales(np.array([[1.0, np.inf]]), 0)).all()


# --- layout and refusals ----------------------------------------------------------------------------------------

STRUCTS = {"cns_dispatch_t": _native.Dispatch, "cns_combine_t": _native.Combine, "cns_combine_grad_t": _native.CombineGrad,
           "cns_rms_norm_t": _native.RmsNorm, "cns_rms_norm_grad_t": _native.RmsNormGrad}


def test_structs_match_c_layout(tmp_path):
    lines = "".join(f'printf("{n} %zu\\n", sizeof({n}));' +
                    "".join(f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for f, _ in s._fields_) for n, s in STRUCTS.items())
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text(f"#include <stdio.h>\n#include <stddef.h>\n#include \"cns.h\"\nint main(void) {{ {lines} return 0; }}\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    lay = dict(line.split() for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for n, s in STRUCTS.items():
        assert int(lay[n]) == ctypes.sizeof(s), n
        for f, _ in s._fields_:
            assert int(lay[f"{n}.{f}"]) == getattr(s, f).offset, (n, f)


def make(kind, good, changes):
    s = kind(**good)
    for k, v in changes.items():
        setattr(s, k, v)
    return s


DISPATCH = dict(x_dev=0x10000, rows_dev=0x20000, places_dev=0x30000, tokens=8, rows=32, row_bytes=64, top_k=4)
SCALES = dict(scales_dev=0x40000, row_scales_dev=0x50000, scale_bytes=16)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), INVALID), (dict(tokens=2 ** 29), INVALID), (dict(rows=-1), INVALID), (dict(top_k=0), INVALID),
    (dict(top_k=33), INVALID), (dict(row_bytes=0), INVALID), (dict(row_bytes=cns.CNS_ROWS_MAX_BYTES + 1), INVALID),
    (dict(x_stride=63), INVALID), (dict(rows_stride=63), INVALID), (dict(rows_stride=2 ** 40), INVALID),
    (dict(places_dev=0x30002), INVALID), (dict(rows_dev=0x10000), INVALID), (dict(reserved=1), INVALID),
    (dict(row_scales_dev=0x50000), INVALID), (dict(scale_bytes=4), INVALID), (dict(SCALES, scale_bytes=0), INVALID),
    (dict(SCALES, scales_stride=15), INVALID), (dict(SCALES, row_scales_stride=-16), INVALID),
    (dict(SCALES, row_scales_dev=0x40000), INVALID), (dict(SCALES, row_scales_dev=None), NULL),
    (dict(x_dev=None), NULL), (dict(rows_dev=None), NULL), (dict(places_dev=None), NULL),
])
def test_dispatch_refusals(built, change, code):
    assert cns.cns_dispatch(make(_native.Dispatch, DISPATCH, change)) == code


COMBINE = dict(rows_dev=0x10000, places_dev=0x20000, weights_dev=0x30000, y_dev=0x40000, tokens=8, rows=32, width=64, top_k=4,
               dtype=1)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), INVALID), (dict(rows=-1), INVALID), (dict(top_k=33), INVALID), (dict(width=0), INVALID),
    (dict(width=cns.CNS_ROWS_MAX_BYTES // 4 + 1), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID),
    (dict(rows_stride=63), INVALID), (dict(base_stride=63), INVALID), (dict(y_stride=-1), INVALID),
    (dict(rows_dev=0x10001), INVALID), (dict(y_dev=0x40001), INVALID), (dict(base_dev=0x50001), INVALID),
    (dict(weights_dev=0x30002), INVALID), (dict(places_dev=0x20001), INVALID), (dict(y_dev=0x10000), INVALID),
    (dict(base_dev=0x40000, y_stride=128), INVALID), (dict(dtype=0, y_dev=0x40002), INVALID), (dict(reserved=2), INVALID),
    (dict(rows_dev=None), NULL), (dict(places_dev=None), NULL), (dict(y_dev=None), NULL),
])
def test_combine_refusals(built, change, code):
    assert cns.cns_combine(make(_native.Combine, COMBINE, change)) == code


COMBINE_GRAD = dict(rows_dev=0x10000, dy_dev=0x20000, places_dev=0x30000, weights_dev=0x40000, drows_dev=0x50000,
                    dweights_dev=0x60000, tokens=8, rows=32, width=64, top_k=4, dtype=2)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), INVALID), (dict(rows=-1), INVALID), (dict(top_k=0), INVALID), (dict(width=0), INVALID),
    (dict(dtype=5), INVALID), (dict(rows_stride=63), INVALID), (dict(dy_stride=63), INVALID),
    (dict(drows_stride=1), INVALID), (dict(drows_dev=0x10000), INVALID), (dict(drows_dev=0x20000), INVALID),
    (dict(dweights_dev=0x40000), INVALID), (dict(dweights_dev=0x60002), INVALID), (dict(dy_dev=0x20001), INVALID),
    (dict(rows_dev=0x10001), INVALID), (dict(drows_dev=0x50001), INVALID), (dict(weights_dev=0x40001), INVALID),
    (dict(places_dev=0x30002), INVALID), (dict(reserved=-1), INVALID), (dict(rows_dev=None), NULL),
    (dict(dy_dev=None), NULL), (dict(places_dev=None), NULL), (dict(drows_dev=None, dweights_dev=None), NULL),
])
def test_combine_backward_refusals(built, change, code):
    assert cns.cns_combine_backward(make(_native.CombineGrad, COMBINE_GRAD, change)) == code


NORM = dict(x_dev=0x10000, residual_dev=0x20000, gain_dev=0x30000, h_dev=0x40000, y_dev=0x50000, q_dev=0x60000,
            scales_dev=0x70000, rows=8, width=256, dtype=1, gain_dtype=0, scale_block=128, eps=1e-6)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(rows=2 ** 31), INVALID), (dict(width=0), INVALID),
    (dict(width=cns.CNS_NORM_MAX_WIDTH + 1), INVALID), (dict(dtype=3), INVALID), (dict(gain_dtype=-1), INVALID),
    (dict(scale_block=16), INVALID), (dict(scale_block=256), INVALID), (dict(scale_block=-1), INVALID),
    (dict(scale_type=2), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(x_stride=255), INVALID),
    (dict(x_stride=cns.CNS_ROWS_MAX_STRIDE + 1), INVALID), (dict(residual_stride=1), INVALID),
    (dict(h_stride=255), INVALID), (dict(y_stride=255), INVALID), (dict(q_stride=255), INVALID),
    (dict(scales_stride=1), INVALID), (dict(x_dev=0x10001), INVALID), (dict(gain_dev=0x30002), INVALID),
    (dict(scales_dev=0x70001), INVALID), (dict(y_dev=0x10000), INVALID), (dict(y_dev=0x20000), INVALID),
    (dict(y_dev=0x40000), INVALID), (dict(h_dev=0x10000, x_stride=512), INVALID),
    (dict(h_dev=0x20000, h_stride=512), INVALID), (dict(residual_dev=None), INVALID), (dict(q_dev=None), INVALID),
    (dict(x_dev=None), NULL), (dict(h_dev=None), NULL), (dict(scales_dev=None), NULL),
    (dict(y_dev=None, q_dev=None, scales_dev=None), NULL),
])
def test_rms_norm_refusals(built, change, code):
    assert cns.cns_rms_norm(make(_native.RmsNorm, NORM, change)) == code


NORM_GRAD = dict(h_dev=0x10000, gain_dev=0x20000, dy_dev=0x30000, dh_dev=0x40000, dx_dev=0x50000, dgain_dev=0x60000,
                 workspace_dev=0x70000, workspace_bytes=8 * 256 * 4, rows=8, width=256, dtype=1, gain_dtype=1, eps=1e-6)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(width=0), INVALID), (dict(dtype=7), INVALID), (dict(gain_dtype=3), INVALID),
    (dict(eps=-1.0), INVALID), (dict(h_stride=255), INVALID), (dict(dy_stride=255), INVALID), (dict(dh_stride=255), INVALID),
    (dict(dx_stride=255), INVALID), (dict(h_dev=0x10001), INVALID), (dict(dgain_dev=0x60002), INVALID),
    (dict(workspace_dev=0x70008), INVALID), (dict(workspace_bytes=8 * 256 * 4 - 1), INVALID), (dict(dx_dev=0x10000), INVALID),
    (dict(dx_dev=0x30000, dx_stride=512), INVALID), (dict(dx_dev=0x40000, dh_stride=512), INVALID),
    (dict(h_dev=None), NULL), (dict(dy_dev=None), NULL), (dict(dx_dev=None), NULL), (dict(workspace_dev=None), NULL),
])
def test_rms_norm_backward_refusals(built, change, code):
    assert cns.cns_rms_norm_backward(make(_native.RmsNormGrad, NORM_GRAD, change)) == code


def test_null_structs_and_workspace_sizes(built):
    L = _native.lib()
    for f in (L.cns_dispatch, L.cns_combine, L.cns_combine_backward, L.cns_rms_norm, L.cns_rms_norm_backward):
        assert f(None) == NULL
    assert cns.cns_rms_norm_workspace_bytes(8, 64, out=False)[0] == NULL
    for rows, width in ((-1, 64), (8, 0), (8, cns.CNS_NORM_MAX_WIDTH + 1), (2 ** 31, 8)):
        assert cns.cns_rms_norm_workspace_bytes(rows, width)[0] == INVALID
    assert cns.cns_rms_norm_workspace_bytes(0, 64) == (0, 0)
    # no more parts than rows, and a bound whatever the rows
    assert cns.cns_rms_norm_workspace_bytes(3, 1000) == (0, 3 * 4000)
    assert cns.cns_rms_norm_workspace_bytes(10 ** 9, 64) == cns.cns_rms_norm_workspace_bytes(10 ** 6, 64)


# --- the Python side: arguments, devices, threads ---------------------------------------------------------------

@pytest.fixture
def handles(monkeypatch):
    """A route and a norm on CPU tensors (whose device index is -1), and the calls that reach the library."""
    import torch
    for t, code in ((torch.float32, 0), (torch.bfloat16, 1), (torch.float16, 2)):
        monkeypatch.setitem(cns._CODES, t, code)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    r = _native.Route()
    r.places, r.weights = torch.zeros((8, 2), dtype=torch.int32), torch.zeros(8, 2)
    r.ids, r.places_dev, r.weights_dev = r.places.clone(), r.places.data_ptr(), r.weights.data_ptr()
    r.capacity, r.index, r.others, r.types = 8, -1, True, (torch.int32, torch.float32)
    r.experts, r.top_k, r.tokens = 16, 2, 8
    n = _native.RmsNorm(width=16, scale_block=32, eps=1e-6)
    n.index, n.others, n.has_y, n.has_q, n.blocks = -1, True, True, False, 1
    n.types = (torch.float8_e4m3fn, torch.float32, torch.float32)
    calls = []

    def entry(name, kind):
        form = struct.Struct("=" + "".join({ctypes.c_void_p: "Q", ctypes.c_uint64: "Q", ctypes.c_int64: "q", ctypes.c_int32: "i",
                                            ctypes.c_float: "f"}[t] for _, t in kind._fields_))
        return lambda b: calls.append((name, kind.from_buffer_copy(b))) or 0, form.pack

    r.call_dispatch, r.call_combine = entry("cns_dispatch", _native.Dispatch), entry("cns_combine", _native.Combine)
    r.call_combine_backward = entry("cns_combine_backward", _native.CombineGrad)
    n.call, n.call_backward = entry("cns_rms_norm", _native.RmsNorm), entry("cns_rms_norm_backward", _native.RmsNormGrad)
    return r, n, calls


def test_arguments_that_python_refuses(handles):
    import torch
    r, n, calls = handles
    x, rows, y = torch.zeros(8, 16), torch.zeros(16, 16), torch.zeros(8, 16)
    bad = [
        lambda: cns.run_dispatch(r, x.t(), rows=rows),                             # columns apart
        lambda: cns.run_dispatch(r, x[:1].expand(8, 16), rows=rows),               # rows that overlap
        lambda: cns.run_dispatch(r, x, rows=rows[:, :8]), lambda: cns.run_dispatch(r, x, rows=rows.half()),
        lambda: cns.run_dispatch(r, torch.zeros(9, 16), rows=rows),                # more tokens than were routed
        lambda: cns.run_dispatch(r, x, rows=rows, places=r.places[:7]),
        lambda: cns.run_dispatch(r, x, rows=rows, places=r.places.long()),
        lambda: cns.run_dispatch(r, x, rows=rows, row_scales=torch.zeros(16, 1)),
        lambda: cns.run_dispatch(r, x, rows=rows, scales=torch.zeros(7, 1), row_scales=torch.zeros(16, 1)),
        lambda: cns.run_dispatch(r, x, rows=rows, scales=torch.zeros(8, 1), row_scales=torch.zeros(16, 2)),
        lambda: cns.run_combine(r, rows, places=r.places, y=y),                    # places without weights
        lambda: cns.run_combine(r, rows, weights=r.weights.half(), y=y),
        lambda: cns.run_combine(r, rows, base=y.half(), y=y), lambda: cns.run_combine(r, rows, y=y[:, :8]),
        lambda: cns.run_combine_backward(r, None, y, drows=rows, dweights=torch.zeros(8, 2)),
        lambda: cns.run_combine_backward(r, rows[:, :8], y, drows=rows),
        lambda: cns.run_combine_backward(r, rows, y, drows=rows[:8], dweights=torch.zeros(8, 2)),
        lambda: cns.run_rms_norm(n, torch.zeros(8, 15), y=y), lambda: cns.run_rms_norm(n, x, torch.zeros(15), y=y),
        lambda: cns.run_rms_norm(n, x, h=y), lambda: cns.run_rms_norm(n, x, y=y, q=y.to(torch.float8_e4m3fn)),
        lambda: cns.run_rms_norm(n, x, residual=y[:4], h=y),
        lambda: cns.run_rms_norm_backward(n, x, torch.zeros(16), y, dx=y, dgain=torch.zeros(15)),
        lambda: cns.run_rms_norm_backward(n, x, torch.zeros(16), y.half(), dx=y),
        lambda: cns.new_rms_norm(0), lambda: cns.new_rms_norm(64, scale_block=48), lambda: cns.new_rms_norm(64, y=False),
    ]
    import types
    import unittest.mock
    with unittest.mock.patch.object(cns, "_torch", lambda: types.SimpleNamespace(float32=0, bfloat16=0, float16=0)):
        for call in bad:
            with pytest.raises(ValueError):
                call()
    with pytest.raises(TypeError):
        cns.run_combine(r, rows.double(), y=y.double())
    with pytest.raises(TypeError):
        cns.run_rms_norm(n, x.double(), y=y.double())
    r.places = None
    with pytest.raises(ValueError, match="plan"):
        cns.run_dispatch(r, x, rows=rows)
    assert not calls


def test_packed_calls_reach_the_entry_points(built):
    """The packed form has the structure's layout, and its answer is the entry point's."""
    for name, kind, good in (("cns_dispatch", _native.Dispatch, DISPATCH), ("cns_combine", _native.Combine, COMBINE),
                             ("cns_combine_backward", _native.CombineGrad, COMBINE_GRAD), ("cns_rms_norm", _native.RmsNorm, NORM),
                             ("cns_rms_norm_backward", _native.RmsNormGrad, NORM_GRAD)):
        call, pack = _native.packed_call(name, kind)
        values = [good.get(f, 0) for f, _ in kind._fields_]
        packed = kind.from_buffer_copy(pack(*values))
        for (f, t), v in zip(kind._fields_, values):
            assert (getattr(packed, f) or 0) == (ctypes.c_float(v).value if t is ctypes.c_float else v), f
        whole = kind(*[v if t is not ctypes.c_void_p else v or None for (_, t), v in zip(kind._fields_, values)])
        assert call(pack(*values)) == getattr(cns, name)(whole)
        bad = [-1 if f in ("tokens", "rows") else v for (f, _), v in zip(kind._fields_, values)]
        assert call(pack(*bad)) == INVALID


def test_calls_of_another_device_are_refused(handles, monkeypatch):
    import torch
    r, n, calls = handles
    x, rows, y, w = torch.zeros(8, 16), torch.zeros(16, 16), torch.zeros(8, 16), torch.zeros(8, 2)
    good = [lambda: cns.run_dispatch(r, x, rows=rows), lambda: cns.run_dispatch_backward(r, rows, dx=x),
            lambda: cns.run_combine(r, rows, y=y), lambda: cns.run_combine_backward(r, rows, y, drows=rows.clone(), dweights=w),
            lambda: cns.run_rms_norm(n, x, y=y), lambda: cns.run_rms_norm_backward(n, x, None, y, dx=y)]
    for call in good:
        call()
    assert [c[0] for c in calls] == ["cns_dispatch", "cns_combine", "cns_combine", "cns_combine_backward", "cns_rms_norm",
                                     "cns_rms_norm_backward"]
    assert calls[1][1].weights_dev is None and calls[2][1].weights_dev == r.weights.data_ptr()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for call in good:
        with pytest.raises(ValueError, match="current"):
            call()
    assert len(calls) == 6


def test_strides_and_sizes_that_reach_the_library(handles):
    import torch
    r, n, calls = handles
    wide = torch.zeros(8, 40, dtype=torch.bfloat16)
    rows = torch.zeros(11, 24, dtype=torch.bfloat16)
    cns.run_dispatch(r, wide[:, 4:20], rows=rows[:, :16], scales=torch.zeros(8, 3), row_scales=torch.zeros(11, 5)[:, 1:4])
    d = calls[-1][1]
    assert (d.tokens, d.rows, d.row_bytes, d.x_stride, d.rows_stride) == (8, 11, 32, 80, 48)
    assert (d.scale_bytes, d.scales_stride, d.row_scales_stride, d.top_k) == (12, 0, 20, 2)
    assert d.x_dev == wide.data_ptr() + 8
    cns.run_dispatch(r, wide[:1, 4:20], rows=rows[:, :16])             # one row: no stride
    assert calls[-1][1].x_stride == 0 and calls[-1][1].tokens == 1
    cns.run_combine(r, rows[:, :16], base=wide[:5, :16], y=wide[:5, 16:32])
    c = calls[-1][1]
    assert (c.tokens, c.rows, c.width, c.rows_stride, c.base_stride, c.y_stride, c.dtype) == (5, 11, 16, 24, 40, 40, 1)
    cns.run_combine_backward(r, None, wide[:, :16], drows=rows[:, :16])
    g = calls[-1][1]
    assert g.rows_dev is None and g.dweights_dev is None and (g.rows, g.drows_stride, g.dy_stride) == (11, 24, 40)
    cns.run_combine_backward(r, rows[:, :16], wide[:, :16], drows=False, dweights=torch.zeros(8, 2))
    assert calls[-1][1].drows_dev is None and calls[-1][1].dweights_dev
