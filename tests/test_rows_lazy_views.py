"""Tensors whose elements are not what their memory holds: torch conjugates and negates lazily, and the calls on rows read
memory.  They are refused.  No GPU."""
import pytest

import counted_notify_sync_gb300 as cns
from test_rows_cpu import handles  # noqa: F401  (a fixture)


def test_lazily_conjugated_rows_are_refused(handles):  # noqa: F811
    import torch
    r, _, calls = handles
    z, out = torch.zeros(8, 16, dtype=torch.complex64), torch.zeros(16, 16, dtype=torch.complex64)
    s, s_out = torch.zeros(8, 3, dtype=torch.complex64), torch.zeros(16, 3, dtype=torch.complex64)
    good = dict(rows=out, scales=s, row_scales=s_out)
    for x, given in ((z.conj(), good), (z[:, :8].conj(), dict(good, rows=out[:, :8])), (z, dict(good, rows=out.conj())),
                     (z, dict(good, rows=torch.zeros(16, 24, dtype=torch.complex64)[:, :16].conj())),
                     (z, dict(good, scales=s.conj())), (z, dict(good, row_scales=s_out.conj()))):
        with pytest.raises(ValueError, match="conj"):
            cns.run_dispatch(r, x, **given)
    assert not calls
    cns.run_dispatch(r, z, **good)
    cns.run_dispatch(r, z.conj().resolve_conj(), **good)
    assert [c[1].row_bytes for c in calls] == [128, 128]


def test_lazily_negated_columns_are_refused(handles):  # noqa: F811
    """The imaginary part of a conjugate: one column of it is a matrix of unit stride."""
    import torch
    r, n, calls = handles
    x = torch.zeros(8, 16, dtype=torch.complex64).conj().imag[:, :1]
    assert x.is_neg() and not x.is_contiguous()
    rows, y = torch.zeros(16, 1), torch.zeros(8, 1)
    n.width = 1
    for call in (lambda: cns.run_dispatch(r, x, rows=rows), lambda: cns.run_combine(r, rows, base=x, y=y),
                 lambda: cns.run_combine_backward(r, rows, x, drows=rows.clone(), dweights=torch.zeros(8, 2)),
                 lambda: cns.run_rms_norm(n, x, y=y), lambda: cns.run_rms_norm_backward(n, x, None, y, dx=y.clone())):
        with pytest.raises(ValueError, match="neg"):
            call()
    assert not calls
    cns.run_dispatch(r, x.resolve_neg(), rows=rows)
    assert len(calls) == 1


def test_a_lazily_negated_number_is_refused(handles):  # noqa: F811
    """A single element is contiguous whatever its strides."""
    import torch
    r, n, calls = handles
    neg = torch.zeros(1, 2, dtype=torch.complex64).conj().imag[:, :1]
    assert neg.is_neg() and neg.is_contiguous() and neg.shape == (1, 1)
    one, rows = torch.zeros(1, 1), torch.zeros(2, 1)
    n.width = 1
    bad = [lambda: cns.run_dispatch(r, neg, rows=rows), lambda: cns.run_dispatch(r, one, rows=neg),
           lambda: cns.run_dispatch(r, one, rows=rows, scales=neg, row_scales=rows),
           lambda: cns.run_dispatch_backward(r, neg, dx=one), lambda: cns.run_dispatch_backward(r, rows, dx=neg),
           lambda: cns.run_combine(r, rows, base=neg, y=one), lambda: cns.run_combine(r, rows, y=neg),
           lambda: cns.run_combine_backward(r, rows, neg, drows=rows.clone(), dweights=torch.zeros(1, 2)),
           lambda: cns.run_combine_backward(r, neg, one, drows=False, dweights=torch.zeros(1, 2)),
           lambda: cns.run_rms_norm(n, neg, y=one), lambda: cns.run_rms_norm(n, one, y=neg),
           lambda: cns.run_rms_norm(n, one, neg[0], y=one.clone()), lambda: cns.run_rms_norm_backward(n, neg, None, one, dx=one.clone()),
           lambda: cns.run_rms_norm_backward(n, one, None, neg, dx=one.clone())]
    r.top_k, i32 = 1, torch.zeros(1, 1, dtype=torch.int32)
    wide = torch.zeros(1, 16)
    with pytest.raises(ValueError, match="neg"):
        cns.run_combine(r, wide, weights=neg, places=i32, y=wide.clone())
    r.top_k = 2
    for call in bad:
        with pytest.raises(ValueError, match="neg"):
            call()
    assert not calls
