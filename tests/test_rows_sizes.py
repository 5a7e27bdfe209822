"""The largest sizes that the header allows reach a launch, and what is past the kernels' counts is refused as a size: the
host code against a stand-in for the CUDA runtime.  No GPU."""
from test_rows_launches import run  # noqa: F401  (a fixture)


def test_as_many_tokens_as_the_header_allows(run):  # noqa: F811
    got = run("""
most = 2 ** 31 - 1
print(json.dumps([
    dispatch(tokens=most, rows=most, row_bytes=1, top_k=1), dispatch(tokens=most, rows=most, row_bytes=2, top_k=1),
    dispatch(tokens=most, rows=most, row_bytes=16, top_k=1),
    dispatch(tokens=most, rows=most, row_bytes=1, top_k=1, scales_dev=A[5], row_scales_dev=A[6], scale_bytes=1),
    dispatch(tokens=most // 2, rows=most, row_bytes=33, top_k=2), combine(tokens=most, rows=most, width=1, top_k=1),
    combine(tokens=most, rows=most, width=1, top_k=1, dtype=0), combine(tokens=most, rows=most, width=8, top_k=1),
    combine(tokens=most // 32, rows=most, width=1, top_k=32), combine_grad(tokens=most, rows=most, width=1, top_k=1),
    combine_grad(tokens=most, rows=most, width=8, top_k=1)]))""")
    for i, (rc, calls) in enumerate(got):
        assert rc == 0 and [c[0] for c in calls] == [0], i


def test_more_than_the_kernels_can_count_is_a_size(run):  # noqa: F811
    """Rows of 16 MB at odd addresses and two thousand million tokens: past any memory."""
    got = run("""
most, invalid = 2 ** 31 - 1, n.CNS_ERR_INVALID_VALUE
print(json.dumps([invalid, dispatch(tokens=most, rows=most, row_bytes=(1 << 24) - 1, top_k=1),
                  combine(tokens=most, rows=most, width=(1 << 22) - 1, top_k=1),
                  combine(tokens=most, rows=most, width=(1 << 22) - 1, top_k=1, dtype=0)]))""")
    invalid = got.pop(0)
    for rc, calls in got:
        assert rc == invalid and calls == []
