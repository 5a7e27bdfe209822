"""The device-wide steps of a training step in 64 bits, plain numpy: routing to experts, its gradient, the
global gradient norm and clipping, rows to their experts and back, the root-mean-square norm.  Written from the
definitions in include/cns.h, row by row where a loop is plainer than an array expression; test infrastructure only."""
from __future__ import annotations

import numpy as np

SIGMOID, SOFTMAX = 0, 1


def scores(x, score):
    """Scores of one row of logits (float64); a row without an unmasked logit scores 0."""
    with np.errstate(all="ignore"):
        if score == SIGMOID:
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max() if not np.isnan(x).any() else np.nan
        if top == -np.inf:
            return np.zeros_like(x)
        e = np.exp(x - top)
        return e / e.sum()


def choice_values(x, s, bias, group_top, round32=True):
    """An expert's choice value: its logit, or its score in 32 bits plus its bias; -inf where masked."""
    if bias is None and group_top == 1:
        v = x.copy()
    else:
        b = np.zeros_like(x) if bias is None else np.asarray(bias, dtype=np.float64)
        v = (s.astype(np.float32) + b.astype(np.float32)).astype(np.float64) if round32 else s + b
    v[x == -np.inf] = -np.inf
    return v


def _rank(values):
    """Indices best first: NaN, then falling values, the lower index first among equals."""
    return sorted(range(len(values)), key=lambda i: (0 if np.isnan(values[i]) else 1,
                                                     0.0 if np.isnan(values[i]) else -values[i], i))


def choose(v, top_k, groups=1, top_groups=0, group_top=1):
    """The chosen experts of one row, best first, -1 where none is left."""
    e = len(v)
    allowed = np.ones(e, dtype=bool)
    if groups > 1:
        size = e // groups
        worth = []
        for g in range(groups):
            mine = v[g * size:(g + 1) * size]
            best = [mine[i] for i in _rank(mine)[:group_top] if mine[i] != -np.inf]
            worth.append(np.sum(np.float32(best).astype(np.float64)) if best else -np.inf)
        worth = np.float32(worth)
        for g in _rank(worth)[(top_groups or groups):]:
            allowed[g * size:(g + 1) * size] = False
    order = [i for i in _rank(v) if allowed[i] and v[i] != -np.inf][:top_k]
    return order + [-1] * (top_k - len(order))


def weights(x, s, ids, score, renorm, scale):
    """The weights of one row's places."""
    w = np.zeros(len(ids))
    there = [j for j, i in enumerate(ids) if i >= 0]
    if not there:
        return w
    chosen = np.array([ids[j] for j in there])
    if renorm and score == SOFTMAX:
        w[there] = scores(x[chosen], SOFTMAX)
    else:
        w[there] = s[chosen]
        if renorm:
            w = w / (w.sum() + 1e-20)
    return w * scale


def route(logits, bias=None, *, top_k, score, groups=1, top_groups=0, group_top=1, renorm=True, scale=1.0):
    """(ids, weights, scores) of [tokens][experts] logits."""
    x = np.asarray(logits, dtype=np.float64)
    ids, w, s = [], [], []
    for row in x:
        sc = scores(row, score)
        i = choose(choice_values(row, sc, bias, group_top), top_k, groups, top_groups, group_top)
        ids.append(i)
        w.append(weights(row, sc, i, score, renorm, scale))
        s.append(sc)
    t, e = x.shape
    return (np.array(ids, dtype=np.int32).reshape(t, top_k), np.array(w).reshape(t, top_k), np.array(s).reshape(t, e))


def plan(ids, experts):
    """(offsets, order, places) of chosen experts."""
    flat = np.asarray(ids).reshape(-1)
    lists = [np.nonzero(flat == e)[0] for e in range(experts)]
    offsets = np.concatenate([[0], np.cumsum([len(a) for a in lists])]).astype(np.int32)
    order = np.full(flat.size, -1, dtype=np.int32)
    places = np.full(flat.size, -1, dtype=np.int32)
    at = 0
    for a in lists:
        order[at:at + len(a)] = a
        places[a] = np.arange(at, at + len(a))
        at += len(a)
    return offsets, order, places.reshape(np.asarray(ids).shape)


def route_backward(logits, ids, dweights, dscores=None, *, score, renorm, scale):
    """dL/dlogits with the chosen experts held fixed."""
    x = np.asarray(logits, dtype=np.float64)
    out = np.zeros_like(x)
    for t, row in enumerate(x):
        s = scores(row, score)
        h = np.zeros_like(row) if dscores is None else np.asarray(dscores[t], dtype=np.float64).copy()
        there = [j for j, i in enumerate(ids[t]) if 0 <= i < len(row)]
        chosen = [int(ids[t][j]) for j in there]
        g = np.array([dweights[t][j] for j in there], dtype=np.float64) * scale
        if chosen and renorm and score == SOFTMAX:
            q = scores(row[chosen], SOFTMAX)
            out[t, chosen] += q * (g - (g * q).sum())
        elif chosen:
            if renorm:
                total = s[chosen].sum() + 1e-20
                g = g / total - (g * s[chosen]).sum() / total ** 2
            h[chosen] += g
        if score == SIGMOID:
            out[t] += h * s * (1.0 - s)
        else:
            out[t] += s * (h - (s * h).sum())
    return out


def grad_norm(tensors, inf=False):
    flat = [np.asarray(t, dtype=np.float64).reshape(-1) for t in tensors]
    flat = np.concatenate(flat) if flat else np.zeros(0)
    if inf:
        return np.abs(flat).max() if flat.size else 0.0
    return np.sqrt((flat ** 2).sum())


# --- rows to their experts and back -----------------------------------------------------------------------------

def dispatch(x, places, rows):
    """`rows` with x's rows written to their places; places outside it are passed over."""
    out = np.array(rows)
    for t, row in enumerate(np.asarray(places)):
        for p in row:
            if 0 <= p < len(out):
                out[p] = x[t]
    return out


def combine(rows, places, weights=None, base=None):
    """(y, the sum of the magnitudes that y is the sum of)."""
    rows = np.asarray(rows, dtype=np.float64)
    t, k = np.asarray(places).shape
    y = np.zeros((t, rows.shape[1])) if base is None else np.asarray(base, dtype=np.float64).copy()
    size = np.abs(y)
    for i in range(t):
        for j in range(k):
            p = places[i][j]
            if 0 <= p < len(rows):
                part = (1.0 if weights is None else float(weights[i][j])) * rows[p]
                y[i] += part
                size[i] += np.abs(part)
    return y, size


def combine_backward(rows, dy, places, weights=None, drows=None):
    """(drows, dweights, the sums of the magnitudes that those are sums of); `drows` is what the rows held before."""
    rows, dy = np.asarray(rows, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    out = np.zeros_like(rows) if drows is None else np.array(drows, dtype=np.float64)
    t, k = np.asarray(places).shape
    dweights, size = np.zeros((t, k)), np.zeros((t, k))
    for i in range(t):
        for j in range(k):
            p = places[i][j]
            if 0 <= p < len(rows):
                out[p] = (1.0 if weights is None else float(weights[i][j])) * dy[i]
                dweights[i, j] = (dy[i] * rows[p]).sum()
                size[i, j] = np.abs(dy[i] * rows[p]).sum()
    return out, dweights, size


# --- the root-mean-square norm ------------------------------------------------------------------------------------

def rms_norm(h, gain=None, eps=1e-6):
    """y of the rows of h (the sum with the residual, as it is held)."""
    h = np.asarray(h, dtype=np.float64)
    with np.errstate(all="ignore"):
        y = h / np.sqrt((h ** 2).mean(-1, keepdims=True) + eps)
        return y if gain is None else y * np.asarray(gain, dtype=np.float64)


def rms_norm_backward(h, gain, dy, dh=None, eps=1e-6):
    """(dx, dgain, the sums of the magnitudes that those are sums of)."""
    h, dy = np.asarray(h, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    g = dy if gain is None else dy * np.asarray(gain, dtype=np.float64)
    r = 1.0 / np.sqrt((h ** 2).mean(-1, keepdims=True) + eps)
    dx = r * g - h * r ** 3 * (g * h).mean(-1, keepdims=True)
    size = np.abs(r * g) + np.abs(h) * r ** 3 * np.abs(g * h).mean(-1, keepdims=True)
    if dh is not None:
        dx, size = dx + np.asarray(dh, dtype=np.float64), size + np.abs(np.asarray(dh, dtype=np.float64))
    return dx, (dy * h * r).sum(0), size, np.abs(dy * h * r).sum(0)


def _e4m3_table():
    """The values of the codes 0 .. 126 (127 is NaN): 4 bits of exponent, bias 7, 3 of fraction."""
    return np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


E4M3 = _e4m3_table()


def e4m3(v):
    """The nearest values, ties to the even code, what is larger than the largest to that."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), E4M3[-1])
    high = np.searchsorted(E4M3, a).clip(max=len(E4M3) - 1)
    low = np.maximum(high - 1, 0)
    up, down = E4M3[high] - a, a - E4M3[low]
    code = np.where(up < down, high, np.where(up > down, low, np.where(high % 2 == 0, high, low)))
    return np.sign(v) * E4M3[code]


def scales(y, block, power=False):
    """The scales of the rows' blocks of columns (0: whole rows); NaN for a block with an infinity or a NaN."""
    y = np.abs(np.asarray(y, dtype=np.float64))
    width = y.shape[1]
    step = block or width
    out = []
    for at in range(0, width, step):
        m = y[:, at:at + step].max(-1)
        if power:
            with np.errstate(all="ignore"):
                _, e = np.frexp(m / 448.0)          # m / 448 = c 2^e, c in [1/2, 1)
                s = np.where(m == 0, 2.0 ** -127, np.ldexp(1.0, e))
                s = np.where(s / 2 >= m / 448.0, s / 2, s)
            s = np.maximum(s, 2.0 ** -127)
        else:
            s = np.maximum(m / 448.0, 2.0 ** -126)
        out.append(np.where(np.isfinite(m), s, np.nan))
    return np.stack(out, -1)
