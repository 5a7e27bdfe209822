"""cns_dispatch, cns_combine and cns_combine_backward on the GPU against the definitions in 64 bits.

Tolerances.  A dispatch moves bytes: none.  A combine's result is at most k products and k + 1 sums in 32 bits, each
off by 2^-24 of at most the sum of the magnitudes, and one rounding to its type.  A row's gradient is one product in 32
bits and one rounding: equal bit for bit.  A weight's gradient sums its products along a path of at most 16 in a
thread's accesses at a time, 5 exchanges, one addition for each stretch of the row (at most 33 at these widths) and 8
warps: under 64 roundings."""
import numpy as np
import pytest

from oracle import steps

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}     # half a step of the type's subnormals


@pytest.fixture(scope="module")
def cns():
    import torch
    import counted_notify_sync_gb300 as c
    c.build()
    torch.cuda.set_device(0)
    return c


def types():
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make_places(rng, tokens, top_k, rows, masked=0.1):
    """Different rows for all places; some without one, a whole token among them, some past the rows' end."""
    p = rng.permutation(max(rows, tokens * top_k))[:tokens * top_k].astype(np.int32).reshape(tokens, top_k)
    if masked and tokens:
        p[rng.rand(tokens, top_k) < masked] = -1
        p[tokens // 2] = -1
        p[0, -1] = 2 ** 31 - 1
        p[-1, 0] = -(2 ** 31)
    return p


def matrix(rng, rows, cols, dtype, pad=0, shift=0):
    """[rows, cols] values of the type within a larger buffer: `pad` columns more from row to row, `shift` before."""
    import torch
    buf = torch.from_numpy(rng.randn(rows * (cols + pad) + shift + 1).astype(np.float32)).to(types()[dtype]).cuda()
    return buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


def host(t):
    return t.double().cpu().numpy()


SHAPES = [
    # tokens, top_k, width, rows more (or fewer) than places
    (1, 1, 1, 0), (1, 8, 4096, 0), (7, 2, 64, 5), (8, 8, 4096, 0), (33, 6, 100, 3), (130, 3, 8, 0), (513, 2, 1000, -200),
    (64, 32, 520, 7), (300, 1, 2048, 0), (5, 4, 8192, 1), (17, 5, 129, 0), (40, 7, 1032, 0), (3, 2, 16392, 0),
    (50, 5, 256, 0), (41, 3, 512, 2), (70, 6, 64, 0), (19, 1, 264, 0), (35, 9, 128, -3),
]


@pytest.mark.parametrize("tokens,top_k,width,more", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (3, 1), (2, 2), (4, 4)])
def test_rows_and_back(cns, tokens, top_k, width, more, dtype, pad, shift):
    import torch
    rng = np.random.RandomState(tokens * 31 + width)
    n = tokens * top_k + more
    r = cns.new_route(tokens, 64, top_k)
    p = make_places(rng, tokens, top_k, n, masked=0.1 if tokens > 1 else 0.0)
    places = torch.from_numpy(p).cuda()
    w = rng.randn(tokens, top_k).astype(np.float32)
    weights = torch.from_numpy(w).cuda()

    # to the experts
    x, _ = matrix(rng, tokens, width, dtype, pad, shift)
    rows, buf = matrix(rng, n, width, dtype, pad, shift)
    before = buf.clone()
    got = cns.run_dispatch(r, x, places=places, rows=rows)
    assert got is rows
    want = before.clone()
    view = want[shift:shift + n * (width + pad)].view(n, width + pad)[:, :width]
    view.copy_(torch.from_numpy(steps.dispatch(host(x), p, host(view))).to(x.dtype))
    assert torch.equal(buf.view(torch.uint8), want.view(torch.uint8))       # what no place names, and the padding, too

    # and back
    base, _ = matrix(rng, tokens, width, dtype, pad, shift)
    for use_w, use_base in ((True, True), (True, False), (False, False)):
        y, ybuf = matrix(rng, tokens, width, dtype, pad, shift)
        ybefore = ybuf.clone()
        if use_w:
            cns.run_combine(r, rows, weights=weights, places=places, base=base if use_base else None, y=y)
        else:
            cns.run_dispatch_backward(r, rows, places=places, dx=y)
        want, size = steps.combine(host(rows), p, w if use_w else None, host(base) if use_base else None)
        tol = (top_k + 2) * 2.0 ** -24 * size + HALF[dtype] * np.abs(want) * (1 + 1e-6) + TINY[dtype]
        assert (np.abs(host(y) - want) <= tol).all()
        y.copy_(ybefore[shift:shift + tokens * (width + pad)].view(tokens, width + pad)[:, :width])
        assert torch.equal(ybuf, ybefore)

    # the gradient
    dy, _ = matrix(rng, tokens, width, dtype, pad, shift)
    drows, dbuf = matrix(rng, n, width, dtype, pad, shift)
    dbefore = dbuf.clone()
    dweights = torch.full((tokens, top_k), 7.0, device="cuda")
    cns.run_combine_backward(r, rows, dy, weights=weights, places=places, drows=drows, dweights=dweights)
    _, want, size = steps.combine_backward(host(rows), host(dy), p, w)
    assert (np.abs(host(dweights) - want) <= 64 * 2.0 ** -24 * size).all()
    wanted = dbefore.clone()
    view = wanted[shift:shift + n * (width + pad)].view(n, width + pad)[:, :width]
    there = np.argwhere((p >= 0) & (p < n))
    if len(there):
        t, j = (torch.from_numpy(there[:, i]).cuda() for i in (0, 1))
        view[places[t, j].long()] = (dy[t].float() * weights[t, j][:, None]).to(dy.dtype)
    assert torch.equal(dbuf.view(torch.uint8), wanted.view(torch.uint8))

    # one of the two alone
    alone = torch.full_like(dweights, 7.0)
    none, _ = cns.run_combine_backward(r, rows, dy, weights=weights, places=places, drows=False, dweights=alone)
    assert none is None and torch.equal(alone, dweights)
    dbuf.copy_(dbefore)
    _, none = cns.run_combine_backward(r, None, dy, weights=weights, places=places, drows=drows)
    assert none is None and torch.equal(dbuf.view(torch.uint8), wanted.view(torch.uint8))


@pytest.mark.parametrize("tokens,top_k,width,block", [(1, 8, 4096, 128), (9, 3, 130, 32), (600, 6, 2048, 128), (50, 4, 33, 8)])
@pytest.mark.parametrize("scale", ["f32", "bytes"])
def test_eight_bit_rows_with_their_scales(cns, tokens, top_k, width, block, scale):
    import torch
    rng = np.random.RandomState(width)
    n, cols = tokens * top_k + 3, -(-width // block)
    r = cns.new_route(tokens, 32, top_k)
    p = make_places(rng, tokens, top_k, n)
    places = torch.from_numpy(p).cuda()
    x = torch.from_numpy(rng.randint(0, 256, (tokens, width)).astype(np.uint8)).cuda()
    s = torch.from_numpy(rng.randint(0, 256, (tokens, cols)).astype(np.uint8)).cuda()
    if scale == "f32":
        s = torch.from_numpy(rng.rand(tokens, cols).astype(np.float32)).cuda()
    rows, row_scales = torch.zeros(n, width, dtype=x.dtype, device="cuda"), torch.zeros(n, cols, dtype=s.dtype, device="cuda")
    for kind in (torch.uint8, torch.float8_e4m3fn, torch.int8):
        rows.zero_()
        row_scales.zero_()
        a, b = cns.run_dispatch(r, x.view(kind), places=places, rows=rows.view(kind), scales=s, row_scales=row_scales)
        assert np.array_equal(a.view(torch.uint8).cpu().numpy(), steps.dispatch(x.cpu().numpy(), p, np.zeros((n, width), np.uint8)))
        assert np.array_equal(b.cpu().numpy(), steps.dispatch(s.cpu().numpy(), p, np.zeros((n, cols), s.cpu().numpy().dtype)))
    a, b = cns.run_dispatch(r, x, places=places, scales=s)
    assert a.shape == (tokens * top_k, width) and b.shape == (tokens * top_k, cols) and b.dtype == s.dtype
    there = np.array(sorted(v for v in p.reshape(-1) if 0 <= v < tokens * top_k))
    if len(there):
        assert torch.equal(a[there], rows[there].view(a.dtype)) and torch.equal(b[there], row_scales[there])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_what_is_not_there_takes_no_part(cns, dtype):
    """NaN in rows and weights that no valid place uses; no tokens; no rows; all places masked."""
    import torch
    t = types()[dtype]
    r = cns.new_route(4, 8, 2)
    p = torch.tensor([[0, -1], [-1, -1], [3, 9], [1, 2]], dtype=torch.int32, device="cuda")
    rows = torch.ones(6, 24, dtype=t, device="cuda")
    rows[4:] = float("nan")
    w = torch.tensor([[2.0, np.nan], [np.nan, np.nan], [3.0, np.inf], [0.5, 0.25]], device="cuda")
    y = cns.run_combine(r, rows, weights=w, places=p)
    assert y.tolist() == [[2.0] * 24, [0.0] * 24, [3.0] * 24, [0.75] * 24]
    dy = torch.ones(4, 24, dtype=t, device="cuda")
    dy[1] = float("nan")
    drows, dw = cns.run_combine_backward(r, rows, dy, weights=w, places=p, drows=torch.zeros_like(rows))
    assert drows.tolist() == [[v] * 24 for v in (2.0, 0.5, 0.25, 3.0, 0.0, 0.0)]
    assert dw.tolist() == [[24.0, 0.0], [0.0, 0.0], [24.0, 0.0], [24.0, 24.0]]
    # an infinity or a NaN that does take part shows
    rows[0, 3] = float("inf")
    rows[1, 4] = float("nan")
    y = cns.run_combine(r, rows, weights=w, places=p)
    assert y[0, 3] == float("inf") and torch.isnan(y[3, 4]) and y[0, 4] == 2.0
    # nothing at all
    none = torch.empty(0, 24, dtype=t, device="cuda")
    assert cns.run_combine(r, none, weights=w, places=p, base=dy * 0 + 5)[0].tolist() == [5.0] * 24
    assert cns.run_dispatch(r, dy, places=p, rows=none).shape == (0, 24)
    drows, dw = cns.run_combine_backward(r, none, dy, weights=w, places=p)
    assert drows.shape == (0, 24) and dw.tolist() == [[0.0, 0.0]] * 4
    e = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    assert cns.run_combine(r, rows, weights=w[:0], places=e, y=none).shape == (0, 24)
    assert cns.run_dispatch(r, none, places=e).shape == (0, 24)
    drows, dw = cns.run_combine_backward(r, rows, none, weights=w[:0], places=e, drows=torch.zeros_like(rows))
    assert dw.shape == (0, 2) and drows.count_nonzero() == 0


def test_in_place_base_and_defaults(cns):
    """The routing's own places and weights, and the result in the residual's place."""
    import torch
    torch.manual_seed(1)
    t, e, k, width = 700, 32, 4, 320
    r = cns.new_route(1000, e, k)
    x = torch.randn(t, width, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn(t, e, device="cuda")
    logits[5] = -float("inf")
    cns.run_route(r, logits)
    rows = cns.run_dispatch(r, x)
    starts = r.offsets.tolist()
    assert starts[-1] == (t - 1) * k and rows.shape == (t * k, width)
    token = torch.div(r.order[:starts[-1]].long(), k, rounding_mode="floor")
    assert torch.equal(rows[:starts[-1]], x[token])
    base = torch.randn_like(x)
    y = cns.run_combine(r, rows, base=base)
    same = base.clone()
    assert cns.run_combine(r, rows, base=same, y=same) is same and torch.equal(same, y)
    assert torch.equal(y[5], base[5])
    dx = cns.run_dispatch_backward(r, rows)
    # four equal rows a token: their sum is exact but for the last rounding
    want = (4 * x.float()).to(x.dtype)
    want[5] = 0
    assert torch.equal(dx, want)
    drows, dw = cns.run_combine_backward(r, rows, base)
    assert torch.equal(drows[:starts[-1]], (base[token].float() * r.weights[:t].reshape(-1)[r.order[:starts[-1]].long(), None])
                       .to(x.dtype))
    assert dw.shape == (t, k) and dw[5].tolist() == [0.0] * k
    with pytest.raises(ValueError, match="tokens"):
        cns.run_dispatch(r, torch.zeros(t + 1, width, device="cuda"))


def test_offsets_past_32_bits(cns):
    """Rows whose distance takes their last ones past 2^32 bytes, and past 2^31 elements."""
    import torch
    step, n, width, k = 2 ** 27 + 8, 20, 264, 2
    buf = torch.empty(step * n, dtype=torch.bfloat16, device="cuda")
    rows = buf.as_strided((n, width), (step, 1))
    rows.zero_()
    t = n // k
    r = cns.new_route(t, 8, k)
    p = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).view(t, k).contiguous()
    x = torch.randn(t, width, device="cuda", dtype=torch.bfloat16)
    cns.run_dispatch(r, x, places=p, rows=rows)
    assert torch.equal(rows, x.repeat_interleave(k, 0).flip(0))
    w = torch.rand(t, k, device="cuda")
    y = cns.run_combine(r, rows, weights=w, places=p)
    want = x.double() * w.double().sum(1, keepdim=True)
    assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 8 * 2.0 ** -24 * x.double().abs() * 2).all()
    drows, dw = cns.run_combine_backward(r, rows, x, weights=w, places=p, drows=rows.clone())
    assert torch.equal(drows, (x.repeat_interleave(k, 0).float() * w.reshape(-1, 1)).to(x.dtype).flip(0))
    square = x.double().square().sum(1, keepdim=True)
    assert ((dw.double() - square).abs() <= 64 * 2.0 ** -24 * square).all()
    cns.run_combine_backward(r, None, x, weights=w, places=p, drows=rows)
    assert torch.equal(rows, drows)
    del buf, rows


def test_many_tokens(cns):
    """More tokens than the CTAs that the GPU holds take at once, in each form of a row."""
    import torch
    torch.manual_seed(9)
    for t, k, width, dtype in ((200_003, 1, 8, torch.bfloat16), (70_001, 3, 72, torch.float16), (30_011, 6, 260, torch.float32),
                               (50_021, 2, 33, torch.bfloat16)):
        r = cns.new_route(t, 16, k, plan=False)
        p = torch.randperm(t * k, device="cuda").to(torch.int32).view(t, k)
        x, w = torch.randn(t, width, device="cuda").to(dtype), torch.rand(t, k, device="cuda")
        rows = cns.run_dispatch(r, x, places=p)
        want = torch.empty_like(rows)
        want[p.reshape(-1).long()] = x.repeat_interleave(k, 0)
        assert torch.equal(rows, want)
        half = torch.finfo(dtype).eps / 2
        y = cns.run_combine(r, rows, weights=w, places=p)
        exact = x.double() * w.double().sum(1, keepdim=True)
        assert ((y.double() - exact).abs() <= (half * (1 + 1e-6) + 8 * 2.0 ** -24) * exact.abs() + 2.0 ** -25).all()
        drows, dw = cns.run_combine_backward(r, rows, x, weights=w, places=p)
        want[p.reshape(-1).long()] = (x.repeat_interleave(k, 0).float() * w.reshape(-1, 1)).to(dtype)
        assert torch.equal(drows, want)
        square = x.double().square().sum(1, keepdim=True)
        assert ((dw.double() - square).abs() <= 64 * 2.0 ** -24 * square).all()


def busy(torch, n=12):
    a = torch.randn(4096, 4096, device="cuda")
    for _ in range(n):
        a @ a


def test_streams_and_new_tensors(cns):
    """New outputs are the call's stream's memory, not what the current stream has still to write."""
    import torch
    t, k, width = 900, 4, 256
    r = cns.new_route(t, 16, k)
    x = torch.randn(t, width, device="cuda")
    cns.run_route(r, torch.randn(t, 16, device="cuda"), sync=True)
    rows = cns.run_dispatch(r, x)
    calls = [lambda s: cns.run_dispatch(r, x, stream=s), lambda s: cns.run_dispatch_backward(r, rows, stream=s),
             lambda s: cns.run_combine(r, rows, stream=s), lambda s: cns.run_combine_backward(r, rows, x, stream=s)[0],
             lambda s: cns.run_combine_backward(r, rows, x, stream=s)[1]]
    want = [c(None) for c in calls]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    for current, given in ((torch.cuda.default_stream(), side), (side, None), (side, other), (side, side)):
        for call, w in zip(calls, want):
            torch.cuda.synchronize()
            with torch.cuda.stream(current):
                late = torch.empty_like(w)
                busy(torch, 4)
                late.fill_(7.0)
                del late
                got = call(given)
            torch.cuda.synchronize()
            assert torch.equal(got, w)


def test_results_do_not_depend_on_timing(cns):
    import torch
    t, k, width = 3001, 6, 520
    r = cns.new_route(t, 64, k)
    cns.run_route(r, torch.randn(t, 64, device="cuda"))
    rows, dy = torch.randn(t * k, width, device="cuda"), torch.randn(t, width, device="cuda")
    y, (drows, dw) = cns.run_combine(r, rows), cns.run_combine_backward(r, rows, dy)
    for _ in range(5):
        assert torch.equal(cns.run_combine(r, rows), y)
        a, b = cns.run_combine_backward(r, rows, dy)
        assert torch.equal(a, drows) and torch.equal(b, dw)
