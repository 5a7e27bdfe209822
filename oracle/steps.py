"""The device-wide steps of a training step in 64 bits, plain numpy: routing to experts, its gradient, the
global gradient norm and clipping.  Written from the definitions in include/cns.h, row by row where a loop is
plainer than an array expression; test infrastructure only."""
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
