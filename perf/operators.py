"""What is measured of the device-wide steps of a training step with experts: routing tokens to experts,
the routing's gradient, the global gradient norm over many tensors, and clipping by it.

    listed()      the cases
    draw(rng)     one more case of the same ranges
    prepare(...)  the inputs of a case, and what a program keeps between its steps
    run(state)    one pass: in elementary torch operations where `own` is false, through this repository's
                  entry points where it is true
    exact(...)    the same results from the definitions in 64 bits
    work(case)    bytes and operations that a pass cannot do without

Routing.  A row of logits l[0..E) is one token's.  Its scores s are sigmoid(l) or softmax(l).  An expert's
choice value is its logit, or s + bias where there is a bias or a group is valued by two of its experts
(the bias balances the load: it takes part in the choice, not in the weights).  An expert whose logit is
-inf is masked and never chosen.  With groups, a group of E / groups neighbouring experts is worth the sum of
its `group_top` best choice values, and only the `top_groups` best groups' experts can be chosen.  The
top_k best are chosen in falling order, the lower index first among equals; places that nothing is left for
hold id -1 and weight 0.  The weights are the chosen scores, divided by their sum with `renorm`, times
`scale`.  An entry is one (token, place), numbered token * top_k + place; `order` lists the entries expert by
expert, in rising number within each; offsets[e] is where expert e's entries start; places[entry] is where
an entry stands in `order` (-1 for a place that holds no expert).

Its gradient.  From the weights' gradient to the logits', the chosen experts held fixed.

Norm and clip.  norm = sqrt(sum of squares over all tensors); each tensor times min(1, max_norm / (norm + eps)),
written to the tensors that the optimiser reads.
"""
import math
import random

import numpy as np
import torch

own = False

SIGMOID, SOFTMAX = "sigmoid", "softmax"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
MAX_NORM, EPS = 1.0, 1e-6

MOST_LOGITS = 65536 * 384
MOST_GRADS = 400_000_000


def routing(op, tokens, experts, top_k, score, dtype, groups=1, top_groups=1, group_top=1, bias=False, renorm=True,
            scale=1.0, masked=0.0):
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "score": score, "dtype": dtype,
            "groups": groups, "top_groups": top_groups, "group_top": group_top, "bias": bias, "renorm": renorm,
            "scale": scale, "masked": masked}


def gradients(op, tensors, elems, dtype, out="f32", even=False):
    return {"op": op, "tensors": tensors, "elems": elems, "dtype": dtype, "out": out, "even": even}


def listed():
    return [
        # one decoding step of a small batch: latency is everything
        dict(routing("route", 8, 128, 8, SOFTMAX, "bf16"), name="route-decode-8x128"),
        # a ragged prefill with padded tokens, groups valued by their best expert, an expert count that is
        # no power of two, weights not renormalised
        dict(routing("route", 3001, 160, 6, SOFTMAX, "f32", groups=8, top_groups=3, renorm=False, scale=16.0,
                     masked=0.05), name="route-prefill-3001x160"),
        # a training step's micro-batch with load-balancing bias and groups valued by their two best
        dict(routing("route", 16384, 256, 8, SIGMOID, "f32", groups=8, top_groups=4, group_top=2, bias=True,
                     scale=2.5), name="route-train-16384x256"),
        # the largest: many tokens and experts, logits in 16 bits (ties are common), no groups
        dict(routing("route", 65536, 384, 8, SIGMOID, "bf16", bias=True, scale=2.5), name="route-train-65536x384"),
        # the gradient of a fine-tuning step: few tokens, two of 64 experts
        dict(routing("route_grad", 509, 64, 2, SOFTMAX, "bf16"), name="route-grad-509x64"),
        # the gradient of the training step above
        dict(routing("route_grad", 16384, 256, 8, SIGMOID, "f32", bias=True, scale=2.5),
             name="route-grad-16384x256"),
        # the gradient through the whole softmax (weights not renormalised), an odd number of tokens
        dict(routing("route_grad", 50021, 160, 6, SOFTMAX, "f32", renorm=False, scale=16.0),
             name="route-grad-50021x160"),
        # the norm over an adapter's few small gradients
        dict(gradients("norm", 24, 200_003, "f32"), name="norm-24-0.2M"),
        # the norm over a model's 16-bit gradients
        dict(gradients("norm", 291, 400_000_000, "bf16", even=True), name="norm-291-400M"),
        # clipping an adapter's gradients into the optimiser's 32-bit ones, at odd addresses
        dict(gradients("clip", 38, 1_000_003, "bf16"), name="clip-38-1M"),
        # clipping 32-bit gradients of a size that the chip holds between its two passes
        dict(gradients("clip", 147, 25_000_011, "f32"), name="clip-147-25M"),
        # clipping a model's 16-bit gradients
        dict(gradients("clip", 291, 400_000_000, "bf16", out="bf16", even=True), name="clip-291-400M"),
    ]


def spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "norm", "clip"])
    if op in ("norm", "clip"):
        elems = spread(rng, 100_000, MOST_GRADS)
        dtype = rng.choice(["f32", "bf16", "f16"])
        if dtype == "f32" or op == "clip":
            elems = min(elems, MOST_GRADS // 4)
        return gradients(op, spread(rng, 1, min(600, elems // 64)), elems, dtype,
                         out=rng.choice(["f32", dtype]), even=rng.random() < 0.5)
    groups, size = rng.choice([(1, spread(rng, 8, 384)), (4, spread(rng, 8, 64)), (8, spread(rng, 4, 48))])
    experts = groups * size
    score = rng.choice([SIGMOID, SOFTMAX])
    top_groups = rng.randint(1, groups)
    bias = score == SIGMOID and rng.random() < 0.7
    return routing(op, spread(rng, 1, min(65536, MOST_LOGITS // experts)), experts,
                   rng.randint(1, min(8, top_groups * size)), score, rng.choice(["f32", "bf16", "f16"]),
                   groups=groups, top_groups=top_groups, group_top=2 if bias and groups > 1 else 1, bias=bias,
                   renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                   masked=rng.choice([0.0, 0.0, 0.1]) if op == "route" else 0.0)


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------

def tensor_sizes(case):
    """The element counts of a case's gradients: many small ones (norms, biases) and a few that hold most of
    it (projections, embeddings); multiples of 64 with `even`, else odd ones among them."""
    rng = random.Random(case["tensors"] * 1_000_003 + case["elems"])
    step = 64 if case["even"] else 1
    parts = [10.0 ** rng.uniform(-4, 0) for _ in range(case["tensors"])]
    whole = case["elems"] // step
    scale = (whole - len(parts)) / sum(parts)
    sizes = [1 + int(p * scale) for p in parts]
    sizes[0] += whole - sum(sizes)
    return [n * step for n in sizes]


def make_logits(case, gen):
    """Router logits: unit variance over a token's experts, some experts more popular than others."""
    t, e = case["tokens"], case["experts"]
    x = torch.randn(t, e, generator=gen, device="cuda")
    x = x * 1.2 + 0.5 * torch.randn(e, generator=gen, device="cuda") - 0.5
    x = x.to(TYPES[case["dtype"]])
    if case["masked"] > 0:
        # padded tokens have no expert, and a share of the others may not use some of them
        pad = torch.rand(t, 1, generator=gen, device="cuda") < case["masked"]
        off = torch.rand(t, e, generator=gen, device="cuda") < case["masked"] / 2
        x = torch.where(pad | off, torch.full_like(x, -math.inf), x)
    return x


def inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] in ("norm", "clip"):
        sizes = tensor_sizes(case)
        flat = torch.randn(sum(sizes), generator=gen, device="cuda", dtype=TYPES[case["dtype"]])
        # layers' gradients differ in size by orders of magnitude
        size = torch.exp(torch.empty(len(sizes), device="cuda").uniform_(-6.0, 0.0, generator=gen))
        flat *= size.to(flat.dtype).repeat_interleave(torch.tensor(sizes, device="cuda"), output_size=flat.numel())
        return {"grads": list(flat.split(sizes)), "sizes": sizes, "flat": flat}
    got = {"logits": make_logits(case, gen), "bias": None}
    if case["bias"]:
        got["bias"] = 0.1 * torch.randn(case["experts"], generator=gen, device="cuda")
    if case["op"] == "route_grad":
        got["ids"] = choose(case, got["logits"], got["bias"])[0].to(torch.int32).contiguous()
        got["dweights"] = torch.randn(case["tokens"], case["top_k"], generator=gen, device="cuda")
    return got


def prepare(case, seed):
    s = dict(inputs(case, seed), case=case)
    if own and case["op"] == "clip":
        s["out"] = torch.empty(s["flat"].numel(), dtype=TYPES[case["out"]], device="cuda")
        s["outs"] = list(s["out"].split(s["sizes"]))
    if own:
        import counted_notify_sync_gb300 as cns
        if case["op"] in ("norm", "clip"):
            s["plan"] = cns.new_grad_clip(s["grads"], MAX_NORM, outs=s.get("outs"), eps=EPS)
        else:
            s["plan"] = cns.new_route(
                case["tokens"], case["experts"], case["top_k"],
                score=cns.CNS_SCORE_SIGMOID if case["score"] == SIGMOID else cns.CNS_SCORE_SOFTMAX,
                groups=case["groups"], top_groups=case["top_groups"], group_top=case["group_top"],
                renorm=case["renorm"], scale=case["scale"])
            if case["op"] == "route_grad":
                s["dlogits"] = torch.empty_like(s["logits"])
    return s


# ---------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if not own:
        return PLAIN[case["op"]](case, s)
    import counted_notify_sync_gb300 as cns
    if case["op"] == "route":
        r = cns.run_route(s["plan"], s["logits"], bias=s["bias"])
        return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "order": r.order, "places": r.places}
    if case["op"] == "route_grad":
        return {"dlogits": cns.run_route_backward(s["plan"], s["logits"], s["dweights"], ids=s["ids"],
                                                  dlogits=s["dlogits"])}
    if case["op"] == "norm":
        return {"norm": cns.run_grad_norm(s["plan"])}
    return {"norm": cns.run_grad_clip(s["plan"]), "clipped": s["out"]}


def scores_of(case, x):
    if case["score"] == SIGMOID:
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def choose(case, logits, bias):
    """(ids [T][k], -1 for none; the scores) of the plain form."""
    x = logits.float()
    s = scores_of(case, x)
    value = x if bias is None and case["group_top"] == 1 else s if bias is None else s + bias
    none = torch.full_like(value, -math.inf)
    value = torch.where(x == -math.inf, none, value)
    t, e, g = case["tokens"], case["experts"], case["groups"]
    if g > 1:
        best = value.view(t, g, e // g).sort(dim=-1, descending=True).values[..., :case["group_top"]]
        worth = torch.where(best == -math.inf, torch.zeros_like(best), best).sum(-1)
        worth = torch.where(best[..., 0] == -math.inf, torch.full_like(worth, -math.inf), worth)
        kept = worth.sort(dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        stays = torch.zeros(t, g, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        value = torch.where(stays.repeat_interleave(e // g, 1), value, none)
    best = value.sort(dim=-1, descending=True, stable=True)
    k = case["top_k"]
    ids = torch.where(best.values[:, :k] == -math.inf, torch.full_like(best.indices[:, :k], -1), best.indices[:, :k])
    return ids, s


def plain_route(case, s):
    ids, scores = choose(case, s["logits"], s["bias"])
    there, safe = ids >= 0, ids.clamp(min=0)
    if case["renorm"] and case["score"] == SOFTMAX:
        x = torch.where(there, s["logits"].float().gather(1, safe), torch.full_like(scores[:, :1], -math.inf))
        w = scores_of(case, x)
    else:
        w = torch.where(there, scores.gather(1, safe), torch.zeros_like(scores[:, :1]))
        if case["renorm"]:
            w = w / (w.sum(-1, keepdim=True) + 1e-20)
    w = w * case["scale"]
    # the entries by expert: a stable sort of the experts, those without one last
    e, flat = case["experts"], ids.reshape(-1)
    n = flat.numel()
    flat = torch.where(flat < 0, torch.full_like(flat, e), flat)
    by = flat.sort(stable=True).indices
    count = torch.zeros(e + 1, dtype=torch.int64, device=flat.device).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([torch.zeros_like(count[:1]), count[:e].cumsum(0)])
    number = torch.arange(n, device=flat.device)
    order = torch.where(number < offsets[e], by, torch.full_like(by, -1))
    places = torch.empty_like(by).scatter_(0, by, number)
    places = torch.where(flat == e, torch.full_like(places, -1), places)
    return {"ids": ids.to(torch.int32), "weights": w, "offsets": offsets.to(torch.int32),
            "order": order.to(torch.int32), "places": places.to(torch.int32).view(case["tokens"], -1)}


def plain_route_grad(case, s):
    x, ids = s["logits"].float(), s["ids"].long()
    there, safe = ids >= 0, ids.clamp(min=0)
    g = torch.where(there, s["dweights"] * case["scale"], torch.zeros_like(s["dweights"]))
    if case["score"] == SOFTMAX and not case["renorm"]:
        p = scores_of(case, x)
        gp = (g * p.gather(1, safe)).sum(-1, keepdim=True)
        return {"dlogits": (p * (torch.zeros_like(x).scatter_add_(1, safe, g) - gp)).to(s["logits"].dtype)}
    lx = torch.where(there, x.gather(1, safe), torch.full_like(g, -math.inf))
    w = scores_of(case, lx)
    if case["score"] == SOFTMAX:
        d = w * (g - (g * w).sum(-1, keepdim=True))
    else:
        if case["renorm"]:
            total = w.sum(-1, keepdim=True) + 1e-20
            g = (g - (g * w).sum(-1, keepdim=True) / total) / total
        d = g * w * (1.0 - w)
    d = torch.where(there, d, torch.zeros_like(d))
    return {"dlogits": torch.zeros_like(x).scatter_add_(1, safe, d).to(s["logits"].dtype)}


def plain_norm(case, s):
    return {"norm": torch.cat(s["grads"]).float().square().sum().sqrt()}


def plain_clip(case, s):
    flat = torch.cat(s["grads"]).float()
    norm = flat.square().sum().sqrt()
    return {"norm": norm, "clipped": (flat * (MAX_NORM / (norm + EPS)).clamp(max=1.0)).to(TYPES[case["out"]])}


PLAIN = {"route": plain_route, "route_grad": plain_route_grad, "norm": plain_norm, "clip": plain_clip}


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------

def scores_exact(case, x):
    with np.errstate(all="ignore"):
        if case["score"] == SIGMOID:
            return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))
        rows = np.isfinite(x).any(-1, keepdims=True)
        e = np.where(rows, np.exp(x - np.where(rows, x.max(-1, keepdims=True), 0.0)), 0.0)
        return e / np.where(rows, e.sum(-1, keepdims=True), 1.0)


def exact(case, seed):
    got = inputs(case, seed)
    if case["op"] in ("norm", "clip"):
        total = got["flat"].double()
        norm = torch.linalg.vector_norm(total)
        if case["op"] == "norm":
            return {"norm": norm}
        return {"norm": norm, "clipped": total * min(1.0, MAX_NORM / (float(norm) + EPS))}
    x = got["logits"].double().cpu().numpy()
    t, e = x.shape
    k, rows = case["top_k"], np.arange(t)[:, None]
    s = scores_exact(case, x)
    if case["op"] == "route":
        value = x if got["bias"] is None and case["group_top"] == 1 else \
            s + (0.0 if got["bias"] is None else got["bias"].double().cpu().numpy())
        value = np.where(np.isneginf(x), -np.inf, value)
        if case["groups"] > 1:
            best = -np.sort(-value.reshape(t, case["groups"], -1), -1)[..., :case["group_top"]]
            worth = np.where(np.isneginf(best[..., 0]), -np.inf, np.where(np.isneginf(best), 0.0, best).sum(-1))
            out = np.argsort(-worth, -1, kind="stable")[:, case["top_groups"]:]
            value = value.reshape(t, case["groups"], -1).copy()
            value[rows, out] = -np.inf
            value = value.reshape(t, e)
        ids = np.argsort(-value, -1, kind="stable")[:, :k]
        there = ~np.isneginf(value[rows, ids])
        if case["renorm"] and case["score"] == SOFTMAX:
            w = scores_exact(case, np.where(there, x[rows, ids], -np.inf))
        else:
            w = np.where(there, s[rows, ids], 0.0)
            if case["renorm"]:
                w = w / (w.sum(-1, keepdims=True) + 1e-20)
        return {"ids": None, "weights": w * case["scale"], "offsets": None, "order": None, "places": None}
    ids = got["ids"].cpu().numpy().astype(np.int64)
    there = ids >= 0
    ids = np.maximum(ids, 0)
    g = np.where(there, got["dweights"].double().cpu().numpy() * case["scale"], 0.0)
    d = np.zeros_like(x)
    if case["score"] == SOFTMAX:
        p = scores_exact(case, np.where(there, x[rows, ids], -np.inf)) if case["renorm"] else s[rows, ids]
        mean = (g * p).sum(-1, keepdims=True)
        if not case["renorm"]:
            d -= s * mean
            np.add.at(d, (rows, ids), p * g)
        else:
            np.add.at(d, (rows, ids), p * (g - mean))
    else:
        w = np.where(there, s[rows, ids], 0.0)
        if case["renorm"]:
            total = w.sum(-1, keepdims=True) + 1e-20
            g = g / total - (g * w).sum(-1, keepdims=True) / total ** 2
        np.add.at(d, (rows, ids), np.where(there, g * w * (1.0 - w), 0.0))
    return {"dlogits": d}


# ---------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------

def work(case):
    if case["op"] in ("norm", "clip"):
        n = case["elems"] // 64 * 64 if case["even"] else case["elems"]
        if case["op"] == "norm":
            return {"bytes": n * BYTES[case["dtype"]] + 4, "flops": 2 * n}
        return {"bytes": n * (BYTES[case["dtype"]] + BYTES[case["out"]]) + 4, "flops": 3 * n}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    logits = t * e * BYTES[case["dtype"]]
    if case["op"] == "route":
        # the logits and the bias; ids, weights, order and places; the offsets.  A score and a comparison each
        return {"bytes": logits + (4 * e if case["bias"] else 0) + 16 * t * k + 4 * (e + 1), "flops": 4 * t * e}
    # ids and the weights' gradient; the logits' gradient; of the logits the chosen ones, or all of them where
    # the gradient goes through the whole softmax
    whole = case["score"] == SOFTMAX and not case["renorm"]
    read = logits if whole else t * k * BYTES[case["dtype"]]
    return {"bytes": read + 8 * t * k + logits, "flops": 5 * (t * e if whole else t * k)}
