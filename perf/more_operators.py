"""What is measured of the operators around a layer of experts: tokens' rows sorted by expert (dispatch) and
back with their weights (combine), the root-mean-square norm before them with the residual's addition and an output
in 8 bits, and their gradients.

    listed()      the cases
    draw(rng)     one more case of the same ranges
    prepare(...)  the inputs of a case, and what a program keeps between its steps
    run(state)    one pass: in elementary torch operations where `own` is false, through this repository's
                  entry points where it is true
    exact(...)    the same results from the definitions in 64 bits
    work(case)    bytes and operations that a pass cannot do without

The plan of a routing lists its entries (token t, place j; number t * top_k + j) by expert: `order` holds the
entries' numbers, -1 behind the last, `places[t][j]` where an entry stands in it, -1 for a place without an expert.

Dispatch.  rows[places[t][j]] = x[t].  Rows may be 8-bit values with a row of scales each, which move along.
Its gradient.  dx[t] = the sum over j of drows[places[t][j]].
Combine.  y[t] = base[t] + the sum over j of weights[t][j] * rows[places[t][j]], in 32 bits, rounded once.
Its gradient.  drows[places[t][j]] = weights[t][j] * dy[t]; dweights[t][j] = dy[t] . rows[places[t][j]], 0 for a
place without an expert.  In all four, rows that no entry names stay as they were.

Norm.  h = x + residual, rounded to the rows' type; y = h / sqrt(mean(h^2) + eps) * gain in 32 bits, rounded to
that type; for each block of `block` columns (0: the row) of y in 32 bits, m its largest magnitude, a scale s:
max(m / 448, 2^-126) in 32 bits, or the lowest power of two from 2^-127 on that is no less than m / 448; q = y / s
rounded to e4m3.
Its gradient.  With r = 1 / sqrt(mean(h^2) + eps) and g = gain * dy: dx = dh + r * g - h * r^3 * mean(g * h), dgain =
the sum over rows of dy * h * r.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
EXPERTS = 64
EPS = 1e-6

MOST = 16384 * 8 * 4096      # elements of the rows of a case
MOST_NORM = 16384 * 4096


def experts(op, tokens, width, top_k, dtype, masked=0.0, base=False, block=128):
    """`masked`: the share of padded tokens, and of places without an expert among the others."""
    return {"op": op, "tokens": tokens, "width": width, "top_k": top_k, "dtype": dtype, "masked": masked, "base": base,
            "block": block}


def norms(op, tokens, width, dtype, residual=True, y=True, block=-1, power=False):
    """`block`: columns of a scale of the 8-bit output, 0 for one a row, -1 for no such output; `power`: scales that
    are powers of two, in 8 bits.  In the gradient `residual` says that one arrives through the residual too."""
    return {"op": op, "tokens": tokens, "width": width, "dtype": dtype, "residual": residual, "y": y, "block": block,
            "power": power}


def listed():
    return [
        # one decoding step of a small batch: latency is everything
        dict(experts("dispatch", 8, 4096, 8, "bf16"), name="dispatch-decode-8x4096"),
        # a large micro-batch whose experts compute in 8 bits: rows and their scales
        dict(experts("dispatch", 16384, 4096, 8, "e4m3"), name="dispatch-8bit-16384x4096"),
        # the gradient of a ragged batch with padded tokens
        dict(experts("dispatch_grad", 3001, 2048, 6, "f16", masked=0.05), name="dispatch-grad-3001x2048"),
        # the gradient of a training step's micro-batch
        dict(experts("dispatch_grad", 16384, 4096, 8, "bf16"), name="dispatch-grad-16384x4096"),
        # the decoding step's way back, into the residual stream
        dict(experts("combine", 8, 4096, 8, "bf16", base=True), name="combine-decode-8x4096"),
        # many tokens of two experts each in 32 bits, an odd number of them, a width that is no power of two
        dict(experts("combine", 50021, 1000, 2, "f32", masked=0.05, base=True), name="combine-50021x1000"),
        # a fine-tuning step of few tokens
        dict(experts("combine_grad", 509, 1024, 2, "bf16"), name="combine-grad-509x1024"),
        # the largest: the way back of a training step, forward rows read and gradient rows written
        dict(experts("combine_grad", 16384, 4096, 8, "bf16"), name="combine-grad-16384x4096"),
        # the decoding step's norm, for a router in 16 bits and experts in 8
        dict(norms("norm", 8, 4096, "bf16", block=128), name="norm-decode-8x4096"),
        # a large micro-batch's norm, with one power of two for 32 values
        dict(norms("norm", 16384, 4096, "bf16", block=32, power=True), name="norm-16384x4096"),
        # the gradient of a small model's norm in 32 bits, odd sizes
        dict(norms("norm_grad", 777, 1000, "f32", residual=False), name="norm-grad-777x1000"),
        # the gradient of a training step's norm
        dict(norms("norm_grad", 16384, 4096, "bf16"), name="norm-grad-16384x4096"),
    ]


def spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "norm", "norm_grad"])
    width = spread(rng, 64, 8192)
    if rng.random() < 0.85:
        width = (width + 7) // 8 * 8
    if op in ("norm", "norm_grad"):
        dtype = rng.choice(["f32", "bf16", "f16"])
        most = MOST_NORM * 2 // BYTES[dtype]
        block = rng.choice([-1, 0, 32, 64, 128]) if op == "norm" else -1
        return norms(op, spread(rng, 1, min(65536, most // width)), width, dtype, residual=rng.random() < 0.6,
                     y=block < 0 or rng.random() < 0.7, block=block, power=block >= 0 and rng.random() < 0.5)
    dtype = rng.choice(["f32", "bf16", "f16"] + (["e4m3"] if op == "dispatch" else []))
    top_k = rng.randint(1, 8)
    most = MOST // max(2, BYTES[dtype])
    return experts(op, spread(rng, 1, min(65536, most // (width * top_k))), width, top_k, dtype,
                   masked=rng.choice([0.0, 0.0, 0.1]), base=op == "combine" and rng.random() < 0.5,
                   block=rng.choice([32, 128]))


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------

def scales_per_row(case):
    return 1 if case["block"] == 0 else -(-case["width"] // case["block"])


def plan(case, gen):
    """order and places of a routing: some experts more popular than others, padded tokens, places without one."""
    t, k = case["tokens"], case["top_k"]
    liking = torch.randn(t, EXPERTS, generator=gen, device="cuda") + 0.5 * torch.randn(EXPERTS, generator=gen, device="cuda")
    ids = liking.topk(k, dim=1).indices
    if case["masked"] > 0:
        pad = torch.rand(t, 1, generator=gen, device="cuda") < case["masked"]
        off = torch.rand(t, k, generator=gen, device="cuda") < case["masked"] / 2
        ids = torch.where(pad | off, torch.full_like(ids, EXPERTS), ids)
    flat = ids.reshape(-1)
    by = flat.sort(stable=True).indices
    number = torch.arange(t * k, device="cuda")
    there = flat < EXPERTS
    order = torch.where(there[by], by, torch.full_like(by, -1))
    places = torch.where(there, torch.empty_like(by).scatter_(0, by, number), torch.full_like(by, -1))
    return order.to(torch.int32), places.to(torch.int32).view(t, k)


def inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    t, w, dtype = case["tokens"], case["width"], TYPES[case["dtype"]]

    def rows(n, to=dtype):
        if to == torch.float8_e4m3fn:   # values that fill the type's range, as a scaled row's do
            return torch.randn(n, w, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(100).clamp_(-448, 448).to(to)
        return torch.randn(n, w, generator=gen, device="cuda", dtype=to)

    got = {}
    if case["op"] in ("norm", "norm_grad"):
        gain = 1.0 + 0.2 * torch.randn(w, generator=gen, device="cuda")
        got["gain"] = gain.to(dtype)
        # tokens differ in size, and a few columns are far larger than the rest
        size = torch.exp(0.5 * torch.randn(t, 1, generator=gen, device="cuda")).to(dtype)
        loud = torch.where(torch.rand(w, generator=gen, device="cuda") < 0.01, 20.0, 1.0).to(dtype)
        got["x"] = rows(t) * size * loud
        if case["op"] == "norm":
            got["residual"] = rows(t) * size if case["residual"] else None
        else:
            got["dy"] = rows(t)
            got["dh"] = rows(t) if case["residual"] else None
        return got
    got["order"], got["places"] = plan(case, gen)
    n = t * case["top_k"]
    if case["op"] == "dispatch":
        got["x"] = rows(t)
        if case["dtype"] == "e4m3":
            got["scales"] = torch.rand(t, scales_per_row(case), generator=gen, device="cuda") * 0.01 + 0.001
        return got
    got["rows"] = rows(n)
    if case["op"] in ("combine", "combine_grad"):
        weights = torch.rand(t, case["top_k"], generator=gen, device="cuda") + 0.05
        weights = weights / weights.sum(-1, keepdim=True)
        got["weights"] = torch.where(got["places"] < 0, torch.zeros_like(weights), weights)
    if case["op"] == "combine":
        got["base"] = rows(t) if case["base"] else None
    if case["op"] == "combine_grad":
        got["dy"] = rows(t)
    return got


def prepare(case, seed):
    s = dict(inputs(case, seed), case=case)
    if own:
        import counted_notify_sync_gb300 as cns
        t, w = case["tokens"], case["width"]
        if case["op"] in ("norm", "norm_grad"):
            s["plan"] = cns.new_rms_norm(w, eps=EPS, y=case["y"], scale_block=None if case["block"] < 0 else case["block"],
                                         scale_type=cns.CNS_SCALE_E8M0 if case["power"] else cns.CNS_SCALE_F32)
            if case["op"] == "norm_grad":
                s["dx"] = torch.empty_like(s["x"])
                s["dgain"] = torch.empty(w, device="cuda")
                s["workspace"] = torch.empty(cns.cns_rms_norm_workspace_bytes(t, w)[1], dtype=torch.uint8, device="cuda")
            else:
                s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
                s["y"] = torch.empty_like(s["x"]) if case["y"] else None
                s["q"] = s["scales"] = None
                if case["block"] >= 0:
                    s["q"] = torch.empty(t, w, dtype=torch.float8_e4m3fn, device="cuda")
                    s["scales"] = torch.empty(t, scales_per_row(case), device="cuda",
                                              dtype=torch.float8_e8m0fnu if case["power"] else torch.float32)
            return s
        s["plan"] = cns.new_route(t, EXPERTS, case["top_k"])
        n = t * case["top_k"]
        if case["op"] == "dispatch":
            s["rows"] = torch.zeros(n, w, device="cuda", dtype=s["x"].dtype)
            s["row_scales"] = torch.zeros(n, s["scales"].shape[1], device="cuda") if "scales" in s else None
        elif case["op"] == "combine_grad":
            s["drows"] = torch.zeros_like(s["rows"])
            s["dweights"] = torch.empty_like(s["weights"])
        else:
            s["y"] = torch.empty(t, w, device="cuda", dtype=s["rows"].dtype)
    return s


# ---------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](case, s)
    import counted_notify_sync_gb300 as cns
    if op == "dispatch":
        if case["dtype"] == "e4m3":
            rows, scales = cns.run_dispatch(s["plan"], s["x"], places=s["places"], rows=s["rows"], scales=s["scales"],
                                            row_scales=s["row_scales"])
            return {"rows": rows, "scales": scales}
        return {"rows": cns.run_dispatch(s["plan"], s["x"], places=s["places"], rows=s["rows"])}
    if op == "dispatch_grad":
        return {"dx": cns.run_dispatch_backward(s["plan"], s["rows"], places=s["places"], dx=s["y"])}
    if op == "combine":
        return {"y": cns.run_combine(s["plan"], s["rows"], weights=s["weights"], places=s["places"], base=s["base"],
                                     y=s["y"])}
    if op == "combine_grad":
        drows, dweights = cns.run_combine_backward(s["plan"], s["rows"], s["dy"], weights=s["weights"],
                                                   places=s["places"], drows=s["drows"], dweights=s["dweights"])
        return {"drows": drows, "dweights": dweights}
    if op == "norm":
        h, y, q, scales = cns.run_rms_norm(s["plan"], s["x"], s["gain"], residual=s["residual"], h=s["h"], y=s["y"],
                                           q=s["q"], scales=s["scales"])
        return {"h": h if case["residual"] else None, "y": y, "q": q, "scales": scales}
    dx, dgain = cns.run_rms_norm_backward(s["plan"], s["x"], s["gain"], s["dy"], dh=s["dh"], dx=s["dx"],
                                          dgain=s["dgain"], workspace=s["workspace"])
    return {"dx": dx, "dgain": dgain}


def entries(case, s):
    """Token of each row and, with padded places, which rows and places there are."""
    order = s["order"].long()
    token = torch.div(order.clamp(min=0), case["top_k"], rounding_mode="floor")
    if case["masked"] == 0:
        return order, token, None, None
    return order.clamp(min=0), token, (order >= 0).unsqueeze(1), (s["places"] >= 0)


def plain_dispatch(case, s):
    _, token, there, _ = entries(case, s)

    def moved(x):
        x = x.view(torch.uint8) if x.element_size() == 1 else x
        got = x.index_select(0, token)
        return got if there is None else torch.where(there, got, torch.zeros_like(got))

    out = {"rows": moved(s["x"]).view(s["x"].dtype)}
    if "scales" in s:
        out["scales"] = moved(s["scales"])
    return out


def gathered(case, s):
    """[tokens][top_k][width]: each place's row in 32 bits, 0 where there is none."""
    at = s["places"].reshape(-1).long()
    got = s["rows"].index_select(0, at.clamp(min=0)).float()
    if case["masked"] > 0:
        got = torch.where((at >= 0).unsqueeze(1), got, torch.zeros_like(got[:, :1]))
    return got.view(case["tokens"], case["top_k"], case["width"])


def plain_dispatch_grad(case, s):
    return {"dx": gathered(case, s).sum(1).to(s["rows"].dtype)}


def plain_combine(case, s):
    y = (gathered(case, s) * s["weights"].unsqueeze(-1)).sum(1)
    if s["base"] is not None:
        y = y + s["base"].float()
    return {"y": y.to(s["rows"].dtype)}


def plain_combine_grad(case, s):
    order, token, there, _ = entries(case, s)
    dy = s["dy"].float()
    drows = dy.index_select(0, token) * s["weights"].reshape(-1).index_select(0, order).unsqueeze(1)
    if there is not None:
        drows = torch.where(there, drows, torch.zeros_like(drows[:, :1]))
    return {"drows": drows.to(s["dy"].dtype), "dweights": (gathered(case, s) * dy.unsqueeze(1)).sum(-1)}


def plain_norm(case, s):
    x, dtype = s["x"], s["x"].dtype
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(dtype)
    hf = h.float()
    y = hf * torch.rsqrt(hf.square().mean(-1, keepdim=True) + EPS) * s["gain"].float()
    out = {"h": None if s["residual"] is None else h, "y": y.to(dtype) if case["y"] else None, "q": None, "scales": None}
    if case["block"] < 0:
        return out
    t, w = y.shape
    block, n = case["block"] or w, scales_per_row(case)
    if n * block > w:
        y = torch.cat([y, y.new_zeros(t, n * block - w)], 1)
    y = y.view(t, n, block)
    largest = y.abs().amax(-1, keepdim=True)
    if case["power"]:
        part, exponent = torch.frexp(largest)               # largest = part * 2^exponent, part in [1/2, 1); 448 = 7/8 * 2^9
        exponent = (exponent - 9 + (part > 0.875)).clamp(min=-127)
        scale = torch.ldexp(torch.ones_like(largest), exponent)
        out["scales"] = (exponent + 127).to(torch.uint8).view(t, n).view(torch.float8_e8m0fnu)
    else:
        scale = (largest / 448.0).clamp(min=2.0 ** -126)
        out["scales"] = scale.view(t, n)
    out["q"] = (y / scale).view(t, n * block)[:, :w].to(torch.float8_e4m3fn)
    return out


def plain_norm_grad(case, s):
    h, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    unit, g = h * r, dy * s["gain"].float()
    dx = r * (g - unit * (g * unit).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dgain": (dy * unit).sum(0)}


PLAIN = {"dispatch": plain_dispatch, "dispatch_grad": plain_dispatch_grad, "combine": plain_combine,
         "combine_grad": plain_combine_grad, "norm": plain_norm, "norm_grad": plain_norm_grad}


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = inputs(case, seed)
    return exact_norm(case, s) if case["op"] in ("norm", "norm_grad") else exact_experts(case, s)


def exact_experts(case, s):
    op, k, places = case["op"], case["top_k"], s["places"].long()
    t, w, n = case["tokens"], case["width"], case["tokens"] * case["top_k"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if op == "dispatch":
        # one place at a time, to where the plan says
        out = {"rows": torch.zeros(n, w, **f64)}
        if "scales" in s:
            out["scales"] = torch.zeros(n, s["scales"].shape[1], **f64)
        for j in range(k):
            there = torch.nonzero(places[:, j] >= 0).squeeze(1)
            out["rows"][places[there, j]] = s["x"].double()[there]
            if "scales" in s:
                out["scales"][places[there, j]] = s["scales"].double()[there]
        return out
    if op == "combine_grad":
        drows, dweights = torch.zeros(n, w, **f64), torch.zeros(t, k, **f64)
        dy, weights = s["dy"].double(), s["weights"].double()
        for j in range(k):
            there = torch.nonzero(places[:, j] >= 0).squeeze(1)
            at = places[there, j]
            drows[at] = weights[there, j].unsqueeze(1) * dy[there]
            dweights[there, j] = torch.einsum("tw,tw->t", dy[there], s["rows"][at].double())
        return {"drows": drows, "dweights": dweights}
    total = torch.zeros(t, w, **f64)
    for j in range(k):
        there = torch.nonzero(places[:, j] >= 0).squeeze(1)
        part = s["rows"][places[there, j]].double()
        total[there] += part * s["weights"].double()[there, j].unsqueeze(1) if op == "combine" else part
    if op == "dispatch_grad":
        return {"dx": total}
    return {"y": total if s["base"] is None else total + s["base"].double()}


def to_e4m3(v):
    """The nearest value with 4 significant bits, 2^-9 its least step, ties to the even one."""
    size = v.abs()
    exponent = torch.floor(torch.log2(torch.where(size == 0, torch.ones_like(size), size))).clamp(min=-6.0)
    step = torch.pow(2.0, exponent - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def exact_norm(case, s):
    h = s["x"].double()
    gain, w = s["gain"].double(), case["width"]
    if case["op"] == "norm_grad":
        length = torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / w + EPS)
        dy = s["dy"].double()
        inner = torch.einsum("tw,tw,w->t", dy, h, gain).unsqueeze(1)
        dx = gain * dy / length - h * inner / (w * length ** 3)
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dgain": torch.einsum("tw,tw->w", dy, h / length)}
    out = {"h": None, "y": None, "q": None, "scales": None}
    if s["residual"] is not None:
        # the sum of two 32-bit numbers rounded to 32 bits, then to the rows' type: what h is held in
        h = (h + s["residual"].double()).float().to(s["x"].dtype).double()
        out["h"] = h
    y = gain * h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / w + EPS)
    if case["y"]:
        out["y"] = y
    if case["block"] < 0:
        return out
    block = case["block"] or w
    q, scales = torch.empty_like(y), []
    for at in range(0, w, block):
        part = y[:, at:at + block]
        scale = part.abs().max(dim=1, keepdim=True).values / 448.0
        if case["power"]:
            scale = torch.pow(2.0, torch.ceil(torch.log2(scale.clamp(min=2.0 ** -127))))
        else:
            scale = scale.clamp(min=2.0 ** -126)
        q[:, at:at + block] = to_e4m3(part / scale)
        scales.append(scale)
    return dict(out, q=q, scales=torch.cat(scales, 1))


# ---------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------

def work(case):
    t, w, op, b = case["tokens"], case["width"], case["op"], BYTES[case["dtype"]]
    row = t * w * b
    if op == "norm":
        out = row * ((2 if case["residual"] else 0) + (1 if case["y"] else 0)) + row + w * b
        if case["block"] >= 0:
            out += t * w + t * scales_per_row(case) * (1 if case["power"] else 4)
        return {"bytes": out, "flops": 6 * t * w}
    if op == "norm_grad":
        return {"bytes": row * (4 if case["residual"] else 3) + w * (b + 4), "flops": 12 * t * w}
    k = case["top_k"]
    there = 1.0 - 1.5 * case["masked"]                # of the places, those that hold an expert
    rows, places = int(row * k * there), 4 * t * k
    if op == "dispatch":
        scales = 4 * scales_per_row(case) if case["dtype"] == "e4m3" else 0
        return {"bytes": row + rows + places + int(t * scales * (1 + k * there)), "flops": 0}
    if op == "combine_grad":
        return {"bytes": row + 2 * rows + 3 * places, "flops": int(3 * t * w * k * there)}
    return {"bytes": row * (2 if case["base"] else 1) + rows + places * (2 if op == "combine" else 1),
            "flops": int(2 * t * w * k * there)}
