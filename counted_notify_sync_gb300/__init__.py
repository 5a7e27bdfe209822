"""counted_notify_sync_gb300: SYNCALL epoch barrier and CntNotify on GB300, and device-wide steps of a
training step (the norm before a layer of experts, routing to them, the tokens' rows to them and back, gradient
norm and clipping).

The C ABI (include/cns.h, libcns.so) does all the work; this package is the
thin Python side: ``_native`` mirrors the C entry points one to one, and the
helpers below allocate device buffers with PyTorch and marshal arguments.
"""
from __future__ import annotations

from . import _native
from ._native import *  # noqa: F401,F403  (C names and constants)

__all__ = [n for n in dir(_native) if not n.startswith("_")] + [
    "build", "new_workspace", "run_syncall", "run_statemachine", "run_pipeline",
    "new_step_workspace", "new_route", "run_route", "run_route_backward", "run_dispatch", "run_dispatch_backward",
    "run_combine", "run_combine_backward", "new_rms_norm", "run_rms_norm", "run_rms_norm_backward", "new_grad_clip",
    "run_grad_norm", "run_grad_clip",
]


def build(force: bool = False, verbose: bool = False) -> str:
    from .builder import build as _b
    return _b(force=force, verbose=verbose)


def _torch():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("counted_notify_sync_gb300 needs a CUDA device")
    return torch


def new_workspace(device=None, start_value: int = 0, stream=None, die_local: bool = True, mirror: bool = True,
                  participants: int | None = None, elems: int | None = None):
    """An initialised SYNCALL workspace on `device`, usable by every barrier variant.  With die_local (the
    default) it starts on a CNS_SYNCALL_DIE_LOCAL_ALIGN boundary, so that the two copies of each counter sit
    on different dies, and has room for the die-local variant's per-die payload copies: of rows of one uint4
    and up to CNS_SYNCALL_MIRROR_MAX_P participants (CNS_SYNCALL_WORKSPACE_MIRROR_BYTES), or, given
    participants and elems, of that ring (syncall_workspace_bytes).  mirror=False gives
    CNS_SYNCALL_WORKSPACE_DIE_LOCAL_BYTES, die_local=False the minimal CNS_SYNCALL_WORKSPACE_BYTES."""
    torch = _torch()
    if not die_local:
        ws = torch.empty(_native.CNS_SYNCALL_WORKSPACE_BYTES // 4, dtype=torch.int32, device=device or "cuda")
    else:
        nbytes = _native.CNS_SYNCALL_WORKSPACE_MIRROR_BYTES if mirror else _native.CNS_SYNCALL_WORKSPACE_DIE_LOCAL_BYTES
        if mirror and participants is not None and elems is not None:
            rc, need = _native.syncall_workspace_bytes(participants, elems)
            _native.check(rc, "syncall_workspace_bytes")
            nbytes = max(nbytes, need)
        align = _native.CNS_SYNCALL_DIE_LOCAL_ALIGN
        raw = torch.empty((nbytes + align) // 4, dtype=torch.int32, device=device or "cuda")
        skip = (-raw.data_ptr()) % align // 4
        ws = raw[skip:skip + nbytes // 4]   # a view: keeps `raw` alive
    _native.check(_native.syncall_workspace_init(ws, ws.numel() * 4, start_value, stream), "syncall_workspace_init")
    return ws


def run_syncall(mode, core_type, workload, launch_ctas, buf0, buf1, rounds, *, used_cores=0, aiv_ratio=0,
                elems=0, threads=256, cluster_dim=0, timeout_ms=0, workspace=None, cta_status=None,
                stream=None, sync=True, host_in=None, host_out=None, check=True, variant=0, launch_flags=0,
                hard_step=0):
    """Call syncall_run with device buffers (torch tensors); returns the filled SyncallData and the code."""
    d = _native.SyncallData()
    d.workload = workload
    d.launch_ctas = launch_ctas
    d.threads = threads
    d.cluster_dim = cluster_dim
    d.buf0_dev = _native.ptr(buf0)
    d.buf1_dev = _native.ptr(buf1)
    d.elems = elems
    d.workspace_dev = _native.ptr(workspace)
    d.cta_status_dev = _native.ptr(cta_status)
    d.stream = _native.stream_handle(stream)
    d.timeout_ms = timeout_ms
    d.sync = 1 if sync else 0
    d.host_in = _native.ptr(host_in)
    d.host_out = _native.ptr(host_out)
    d.barrier_variant = variant
    d.launch_flags = launch_flags
    d.hard_step = hard_step
    d.workspace_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    rc = _native.syncall_run(mode, core_type, used_cores, aiv_ratio, rounds, d)
    if check and rc != _native.CNS_SUCCESS:
        raise _native.CnsError(rc, "syncall_run")
    return d, rc


def run_statemachine(ops_dev, init: int, stream=None):
    """Apply an [n, 4] int32 device op stream; returns (trace [n, 2] int32, final [1] int32) device tensors."""
    torch = _torch()
    n = ops_dev.shape[0]
    trace = torch.empty((n, 2), dtype=torch.int32, device=ops_dev.device)
    final = torch.empty(1, dtype=torch.int32, device=ops_dev.device)
    sb = _native.cns_statemachine_scratch_bytes(n)
    scratch = torch.empty(max(sb, 8), dtype=torch.uint8, device=ops_dev.device)
    _native.check(_native.cns_statemachine_run(ops_dev if n else None, n, init, trace if n else None, final,
                                               scratch, scratch.numel(), stream), "cns_statemachine_run")
    return trace, final


def run_pipeline(done, ack, tiles: int, tile_words: int, rounds: int, producer_stream, consumer_stream,
                 timeout_s: int = 10, producer_ctas: int = 0, sync: bool = True, buffers=None, areas: int = 1,
                 consumer_wait: int = 0):
    """Run the two-stream counting pipeline; returns (Pipeline struct, code, checksums, released).
    areas = 2 alternates the rounds between two tile areas (the tile buffer then holds both);
    consumer_wait = 1 (CNS_PIPE_WAIT_IN_KERNEL) has the consumer kernel take the wait itself."""
    torch = _torch()
    if buffers is None:
        tiles_buf = torch.empty(max(1, areas) * tiles * tile_words, dtype=torch.int32, device="cuda")
        checksums = torch.empty(rounds, dtype=torch.int32, device="cuda")
        released = torch.empty(rounds, dtype=torch.int32, device="cuda")
    else:
        tiles_buf, checksums, released = buffers
    cfg = _native.Pipeline()
    cfg.done = done
    cfg.ack = ack
    cfg.tiles_dev = _native.ptr(tiles_buf)
    cfg.checksums_dev = _native.ptr(checksums)
    cfg.released_dev = _native.ptr(released)
    cfg.tiles = tiles
    cfg.tile_words = tile_words
    cfg.producer_ctas = producer_ctas
    cfg.rounds = rounds
    cfg.producer_stream = _native.stream_handle(producer_stream)
    cfg.consumer_stream = _native.stream_handle(consumer_stream)
    cfg.timeout_s = timeout_s
    cfg.sync = 1 if sync else 0
    cfg.areas = areas
    cfg.consumer_wait = consumer_wait
    rc = _native.cns_pipeline_run(cfg)
    return cfg, rc, checksums, released


# --- device-wide steps of a training step ------------------------------------------------------------------
#
# Like every call here these run on the stream that they are given (None: the default stream) and return before
# the GPU is done.  A tensor that belongs to another stream needs what it needs for any kernel: the streams
# ordered by an event, and record_stream before it is freed.
#
# A handle (new_route, new_grad_clip) has one workspace and one set of results, so its calls belong to one thread at
# a time, and those of run_route, run_grad_norm and run_grad_clip to streams that are ordered with one another.
# run_route_backward, run_dispatch, run_combine, their gradients and the norm only read the handle: they may be called
# from several threads at once.  A handle's device has to be the current one at each call.

_CODES = {}   # torch dtype -> cns_dtype_t, filled by the first new_route, new_rms_norm or new_grad_clip


def _dtype_codes():
    if not _CODES:
        torch = _torch()
        _CODES.update({torch.float32: _native.CNS_DT_F32, torch.bfloat16: _native.CNS_DT_BF16,
                       torch.float16: _native.CNS_DT_F16})
    return _CODES


def _dtype_code(dtype):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"float32, bfloat16 or float16 expected, got {dtype}")
    return code


def _check_current(index):
    """The library launches on the current device, whatever device the tensors are on.  (Handles say whether there
    is another one at all: asking torch takes half a microsecond.)"""
    import torch
    at = torch.cuda.current_device()
    if at != index:
        raise ValueError(f"made for CUDA device {index}, and device {at} is the current one")


def new_step_workspace(nbytes: int, device=None, stream=None):
    """An initialised workspace of `nbytes` for cns_route, cns_grad_norm and cns_grad_clip.  Calls that follow
    one another on a stream may share one; calls that may overlap need one each.
    Its memory is torch's current stream's and is zeroed on that stream; `stream` and the default stream wait for
    it.  Any other stream that uses the workspace has to wait for the current one first, as for every tensor."""
    torch = _torch()
    nbytes = max(nbytes, _native.CNS_STEP_WORKSPACE_HEADER_BYTES)
    with torch.cuda.device(torch.device(device or "cuda")):
        ws = torch.empty((nbytes + 15) // 16 * 4, dtype=torch.int32, device="cuda")   # torch aligns to 512 bytes
        here = torch.cuda.current_stream()
        _native.check(_native.cns_step_workspace_init(ws, ws.numel() * 4, here), "cns_step_workspace_init")
        handle = _native.stream_handle(stream)
        if handle and handle != here.cuda_stream:
            torch.cuda.ExternalStream(handle).wait_stream(here)
        # (what a capture records reaches the default stream by the replay alone)
        if here.cuda_stream and not torch.cuda.is_current_stream_capturing():
            torch.cuda.default_stream().wait_stream(here)
    return ws


def new_route(tokens: int, experts: int, top_k: int, *, score: int = _native.CNS_SCORE_SOFTMAX, groups: int = 1,
              top_groups: int = 0, group_top: int = 1, renorm: bool = True, scale: float = 1.0, plan: bool = True,
              scores: bool = False, workspace=None, timeout_ms: int = 0, device=None, stream=None):
    """A routing of up to `tokens` tokens (cns_route_t, see cns.h for the rules), with the tensors that
    run_route fills:
      ids [tokens, top_k] int32, weights [tokens, top_k] float32;
      with plan: offsets [experts + 1], order [tokens * top_k], places [tokens, top_k], all int32;
      with scores: scores [tokens, experts] float32.
    They are torch's current stream's, and so is the zeroing of the workspace that this enqueues: see
    new_step_workspace for the streams that are ordered behind it."""
    torch = _torch()
    _dtype_codes()
    r = _native.Route()
    device = torch.device(device or "cuda")
    rc, nbytes = _native.cns_route_workspace_bytes(tokens, experts, top_k)
    _native.check(rc, "new_route")
    i32 = dict(dtype=torch.int32, device=device)
    r.ids = torch.empty((tokens, top_k), **i32)
    r.weights = torch.empty((tokens, top_k), dtype=torch.float32, device=device)
    r.scores = torch.empty((tokens, experts), dtype=torch.float32, device=device) if scores else None
    r.offsets = torch.empty(experts + 1, **i32) if plan else None
    r.order = torch.empty(tokens * top_k, **i32) if plan else None
    r.places = torch.empty((tokens, top_k), **i32) if plan else None
    r.workspace = workspace
    if plan and workspace is None:
        r.workspace = new_step_workspace(nbytes, device, stream)
    r.capacity, r.index, r.others = tokens, r.ids.get_device(), torch.cuda.device_count() > 1
    r.types = (torch.int32, torch.float32)
    r.call_dispatch = _native.packed_call("cns_dispatch", _native.Dispatch)
    r.call_combine = _native.packed_call("cns_combine", _native.Combine)
    r.call_combine_backward = _native.packed_call("cns_combine_backward", _native.CombineGrad)
    b = r.backward = _native.RouteGrad()   # run_route_backward's, but for the call's own tensors
    b.experts, b.top_k, b.score, b.renorm, b.scale = experts, top_k, score, int(renorm), scale
    r.ids_dev, r.weights_dev, r.scores_dev = _native.ptr(r.ids), _native.ptr(r.weights), _native.ptr(r.scores)
    r.offsets_dev, r.order_dev, r.places_dev = _native.ptr(r.offsets), _native.ptr(r.order), _native.ptr(r.places)
    r.workspace_dev = _native.ptr(r.workspace)
    r.workspace_bytes = r.workspace.numel() * r.workspace.element_size() if r.workspace is not None else 0
    r.experts, r.top_k, r.score = experts, top_k, score
    r.groups, r.top_groups, r.group_top = groups, top_groups, group_top
    r.renorm, r.scale, r.timeout_ms = int(renorm), scale, timeout_ms
    return r


def _check_logits(route, logits, what):
    """(rows, elements from row to row) of a [tokens, experts] tensor."""
    shape, stride, e = logits.shape, logits.stride(), route.experts
    if len(shape) == 2 and logits.get_device() == route.index:
        (t, cols), (step, one) = shape, stride
        if cols == e and t <= route.capacity and (one == 1 or e == 1) and (step >= e or t <= 1):
            return t, step if t > 1 else 0
    raise ValueError(f"{what}: [tokens <= {route.capacity}, {e}] on {route.ids.device}, rows apart and of unit stride, "
                     f"expected; got {tuple(shape)}, strides {stride}, on {logits.device}")


def _check_rows(route, x, name, rows, cols, dtype):
    shape = x.shape
    if not (len(shape) == 2 and shape[0] >= rows and shape[1] == cols and x.is_contiguous() and x.dtype == dtype and
            x.get_device() == route.index):
        raise ValueError(f"{name}: contiguous {dtype} [tokens, {cols}] on {route.ids.device} expected")


def run_route(route, logits, bias=None, stream=None, sync: bool = False):
    """Route the rows of `logits` ([tokens, experts], float32, bfloat16 or float16, rows at any stride) on
    `stream` (None: the default stream).  Returns `route`, whose tensors hold the results: the first
    logits.shape[0] rows, and of `order` the first logits.shape[0] * top_k.  They are no part of torch's graph:
    run_route_backward has the gradient (examples/expert_training_step.py joins the two to autograd)."""
    if route.others:
        _check_current(route.index)
    t, route.logits_stride = _check_logits(route, logits, "logits")
    if bias is None:
        route.bias_dev = None
    else:
        if not (bias.is_contiguous() and bias.numel() == route.experts and bias.dtype == route.types[1] and
                bias.get_device() == route.index):
            raise ValueError("bias: contiguous float32 [experts] on the logits' device expected")
        route.bias_dev = bias.data_ptr()
    route.dtype = _dtype_code(logits.dtype)
    route.logits_dev, route.tokens = logits.data_ptr(), t
    route.stream = _native.stream_handle(stream)
    route.sync = 1 if sync else 0
    rc = _native.cns_route(route)
    if rc:
        raise _native.CnsError(rc, "cns_route")
    return route


def _empty_on(stream, like, shape, dtype=None):
    """A tensor whose memory is the stream's that the call runs on: torch hands out what calls of its own stream may
    still be using, which comes before that stream's work alone."""
    import torch
    handle = _native.stream_handle(stream) or 0
    if torch._C._cuda_getCurrentRawStream(like.get_device()) == handle:   # (a Stream object takes some us)
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()):
        return like.new_empty(shape, dtype=dtype)


def run_route_backward(route, logits, dweights, *, ids=None, dscores=None, dlogits=None, stream=None):
    """dL/dlogits of run_route(route, logits): from dL/dweights [tokens, top_k] float32 and, if given,
    dL/dscores [tokens, experts] float32.  `ids` are the chosen experts (default: route.ids); the result goes to
    `dlogits` (default: a new tensor, of `stream`'s memory) in the logits' type."""
    if route.others:
        _check_current(route.index)
    g = _native.RouteGrad.from_buffer_copy(route.backward)   # this call's own: other threads may be filling in theirs
    t, step = _check_logits(route, logits, "logits")
    dtype = logits.dtype
    if step:
        g.logits_stride = step
    if dlogits is None:
        dlogits = _empty_on(stream, logits, (t, route.experts))
    else:
        rows, step = _check_logits(route, dlogits, "dlogits")
        if rows != t or dlogits.dtype != dtype:
            raise ValueError("dlogits: the logits' type and shape expected")
        if step:
            g.dlogits_stride = step
    if ids is None:
        ids = route.ids
    (i32, f32), top_k = route.types, g.top_k
    _check_rows(route, ids, "ids", t, top_k, i32)
    _check_rows(route, dweights, "dweights", t, top_k, f32)
    if dscores is not None:
        _check_rows(route, dscores, "dscores", t, route.experts, f32)
        g.dscores_dev = dscores.data_ptr()
    if stream is not None:
        g.stream = _native.stream_handle(stream)
    g.logits_dev, g.ids_dev, g.dweights_dev = logits.data_ptr(), ids.data_ptr(), dweights.data_ptr()
    g.dlogits_dev, g.tokens, g.dtype = dlogits.data_ptr(), t, _dtype_code(dtype)
    rc = _native.cns_route_backward(g)
    if rc:
        raise _native.CnsError(rc, "cns_route_backward")
    return dlogits


# The calls below check their tensors in place where these are as most are (dense, of the shape, type and device
# expected), and ask a function about the others: with that and packed arguments a combine takes the host 4.6 us, where a
# function for each tensor and a structure filled in took 6.6.

def _matrix(x, name, index, shape, dtype):
    """Elements from row to row (0: packed) of a matrix."""
    if x.shape == shape and x.dtype is dtype and x.get_device() == index:
        if x.is_contiguous():
            return 0
        (rows, cols), (step, one) = shape, x.stride()
        if (one == 1 or cols == 1) and (step >= cols or rows <= 1):
            _no_neg(**{name: x})
            return step if rows > 1 else 0
    raise ValueError(f"{name}: {tuple(shape)} {dtype} on CUDA device {index}, rows apart and of unit stride, expected; got "
                     f"{tuple(x.shape)} {x.dtype}, strides {x.stride()}, on {x.device}")


def _no_neg(**tensors):
    """Refuse tensors that stand for their memory's numbers with the other sign: parts of lazy conjugates, so contiguous
    only with a single element."""
    for name, x in tensors.items():
        if x is not None and x is not False and x.is_neg():
            raise ValueError(f"{name}: a lazily negated tensor; pass its resolve_neg()")


def _no_conj(**tensors):
    """Refuse tensors that stand for the conjugates of what their memory holds."""
    for name, x in tensors.items():
        if x is not None and x.is_conj():
            raise ValueError(f"{name}: a lazily conjugated tensor; pass its resolve_conj()")


def _per_place(route, x, name, tokens, dtype):
    """Address of a value for each place of `tokens` tokens, or of more."""
    if x.is_contiguous() and x.dtype is dtype and x.get_device() == route.index:
        shape = x.shape
        if shape == (tokens, route.top_k) or (len(shape) == 2 and shape[0] > tokens and shape[1] == route.top_k):
            return x.data_ptr()
    raise ValueError(f"{name}: contiguous {dtype} [tokens, {route.top_k}] on {route.ids.device} expected")


def _places(route, places, tokens):
    """Address of the places of `tokens` tokens: given ones, or those of the route's last call."""
    if places is not None:
        return _per_place(route, places, "places", tokens, route.types[0])
    if route.places is None:
        raise ValueError("a route without a plan has no places")
    if tokens > route.tokens:
        raise ValueError(f"{tokens} tokens, and the route's last call had {route.tokens}")
    return route.places_dev or 0


def _weights(route, weights, places, tokens):
    """Address of the weights of `tokens` tokens' places: given ones, or those of the route's last call."""
    if weights is not None:
        return _per_place(route, weights, "weights", tokens, route.types[1])
    if places is not None:
        raise ValueError("places come with their weights")
    return route.weights_dev or 0


def run_dispatch(route, x, *, places=None, rows=None, scales=None, row_scales=None, stream=None):
    """Sort tokens' rows by expert: rows[places[t, j]] = x[t], for `x` [tokens, width] of any type, rows at any
    stride.  `places` [tokens, top_k] int32 are the plan's (default: those of run_route's last call); expert e's rows
    are then rows[offsets[e]:offsets[e + 1]].  `rows` [any number, width] (default: a new tensor of tokens * top_k, of
    `stream`'s memory); places outside it are passed over (a limited capacity), and rows that no place names stay as they
    were, in a new tensor whatever its memory held.  With `scales` [tokens, n], of any type, row_scales[places[t, j]] =
    scales[t] too.  Returns rows, with scales (rows, row_scales), no part of torch's graph: run_dispatch_backward has the
    gradient.  (What memory holds is moved: lazily conjugated or negated tensors are refused, by the calls below too.)"""
    index, shape, dtype, size, top_k = route.index, x.shape, x.dtype, x.element_size(), route.top_k
    if route.others:
        _check_current(index)
    if size >= 4 and dtype.is_complex:
        _no_conj(x=x, rows=rows)
    t, width = shape
    if width == 1:
        _no_neg(x=x, rows=rows)
    x_step = 0 if x.is_contiguous() and x.get_device() == index else _matrix(x, "x", index, shape, dtype) * size
    if places is not None and (places.shape == (t, top_k) and places.dtype is route.types[0] and
                               places.get_device() == index and places.is_contiguous()):
        places_at = places.data_ptr()
    else:
        places_at = _places(route, places, t)
    if rows is None:
        n, rows_step, rows = t * top_k, 0, _empty_on(stream, x, (t * top_k, width))
    else:
        n = rows.shape[0]
        rows_step = 0 if (rows.shape == (n, width) and rows.dtype is dtype and rows.get_device() == index and
                          rows.is_contiguous()) else _matrix(rows, "rows", index, (n, width), dtype) * size
    each = scales_at = row_scales_at = scales_step = row_scales_step = 0
    if scales is not None:
        kind, each, cols = scales.dtype, scales.element_size(), scales.shape[-1]
        if kind.is_complex:
            _no_conj(scales=scales, row_scales=row_scales)
        if cols == 1:
            _no_neg(scales=scales, row_scales=row_scales)
        scales_step = _matrix(scales, "scales", index, (t, cols), kind) * each
        if row_scales is None:
            row_scales = _empty_on(stream, scales, (n, cols))
        row_scales_step = _matrix(row_scales, "row_scales", index, (n, cols), kind) * each
        scales_at, row_scales_at, each = scales.data_ptr(), row_scales.data_ptr(), cols * each
    elif row_scales is not None:
        raise ValueError("row_scales without scales")
    call, pack = route.call_dispatch
    rc = call(pack(x.data_ptr(), rows.data_ptr(), scales_at, row_scales_at, places_at,
                   0 if stream is None else _native.stream_handle(stream), t, n, width * size, each, x_step, rows_step,
                   scales_step, row_scales_step, top_k, 0))
    if rc:
        raise _native.CnsError(rc, "cns_dispatch")
    return rows if scales is None else (rows, row_scales)


def _combine(route, rows, weighted, weights, places, base, y, stream, what):
    """cns_combine, with weights or without; `what` names the rows and the result in errors."""
    index, shape, dtype, top_k, (i32, f32) = route.index, rows.shape, rows.dtype, route.top_k, route.types
    if route.others:
        _check_current(index)
    code = _CODES.get(dtype)
    if code is None:
        code = _dtype_code(dtype)
    n, width = shape
    rows_step = 0 if rows.is_contiguous() and rows.get_device() == index else _matrix(rows, what[0], index, shape, dtype)
    first = y if y is not None else base if base is not None else places
    t = route.tokens if first is None else first.shape[0]
    shape, per = (t, width), (t, top_k)
    if width == 1 or t == top_k == 1:
        _no_neg(weights=weights, base=base, **{what[0]: rows, what[1]: y})
    weights_at = base_at = base_step = y_step = 0
    if weighted:
        if weights is not None and (weights.shape == per and weights.dtype is f32 and weights.get_device() == index and
                                    weights.is_contiguous()):
            weights_at = weights.data_ptr()
        else:
            weights_at = _weights(route, weights, places, t)
    if places is not None and (places.shape == per and places.dtype is i32 and places.get_device() == index and
                               places.is_contiguous()):
        places_at = places.data_ptr()
    else:
        places_at = _places(route, places, t)
    if base is not None:
        base_at = base.data_ptr()
        base_step = 0 if (base.shape == shape and base.dtype is dtype and base.get_device() == index and
                          base.is_contiguous()) else _matrix(base, "base", index, shape, dtype)
    if y is None:
        y = _empty_on(stream, rows, shape)
    elif not (y.shape == shape and y.dtype is dtype and y.get_device() == index and y.is_contiguous()):
        y_step = _matrix(y, what[1], index, shape, dtype)
    call, pack = route.call_combine
    rc = call(pack(rows.data_ptr(), places_at, weights_at, base_at, y.data_ptr(),
                   0 if stream is None else _native.stream_handle(stream), t, n, rows_step, base_step, y_step, width, top_k,
                   code, 0))
    if rc:
        raise _native.CnsError(rc, "cns_combine")
    return y


def run_dispatch_backward(route, drows, *, places=None, dx=None, stream=None):
    """dL/dx of run_dispatch from dL/drows (float32, bfloat16 or float16): dx[t] = the sum over j of
    drows[places[t, j]], in 32 bits, rounded once.  For the tokens of `dx` (default: a new tensor for those of
    `places`, or of run_route's last call)."""
    return _combine(route, drows, False, None, places, None, dx, stream, ("drows", "dx"))


def run_combine(route, rows, *, weights=None, places=None, base=None, y=None, stream=None):
    """Experts' rows back to their tokens: y[t] = base[t] + the sum over j of weights[t, j] * rows[places[t, j]], in 32
    bits, rounded once, for rows [any number, width] in float32, bfloat16 or float16.  `weights` [tokens, top_k] float32
    and `places` default to those of run_route's last call; `base` [tokens, width] (the residual, say) is optional.  The
    result goes to `y` [tokens, width] (default: a new tensor, of `stream`'s memory), which may be `base`."""
    return _combine(route, rows, True, weights, places, base, y, stream, ("rows", "y"))


def run_combine_backward(route, rows, dy, *, weights=None, places=None, drows=None, dweights=None, stream=None):
    """The gradient of run_combine from dL/dy [tokens, width]: (drows, dweights), drows[places[t, j]] = weights[t, j] *
    dy[t], and dweights[t, j] = dy[t] . rows[places[t, j]], 0 for a place without a row.  `drows` (default: a new tensor
    like rows): what no place names stays as it was.  `rows` None: no dweights (None is returned); `drows` False: no
    drows.  The base's gradient is dy."""
    index, shape, dtype, top_k, (i32, f32) = route.index, dy.shape, dy.dtype, route.top_k, route.types
    if route.others:
        _check_current(index)
    code = _CODES.get(dtype)
    if code is None:
        code = _dtype_code(dtype)
    t, width = shape
    dy_step = 0 if dy.is_contiguous() and dy.get_device() == index else _matrix(dy, "dy", index, shape, dtype)
    per = (t, top_k)
    if width == 1 or t == top_k == 1:
        _no_neg(rows=rows, dy=dy, weights=weights, drows=drows, dweights=dweights)
    if weights is not None and (weights.shape == per and weights.dtype is f32 and weights.get_device() == index and
                                weights.is_contiguous()):
        weights_at = weights.data_ptr()
    else:
        weights_at = _weights(route, weights, places, t)
    if places is not None and (places.shape == per and places.dtype is i32 and places.get_device() == index and
                               places.is_contiguous()):
        places_at = places.data_ptr()
    else:
        places_at = _places(route, places, t)
    n, rows_at, rows_step, dweights_at = t * top_k, 0, 0, 0
    if rows is not None:
        n, rows_at = rows.shape[0], rows.data_ptr()
        rows_step = 0 if (rows.shape == (n, width) and rows.dtype is dtype and rows.get_device() == index and
                          rows.is_contiguous()) else _matrix(rows, "rows", index, (n, width), dtype)
        if dweights is None:
            dweights = _empty_on(stream, dy, per, f32)
            dweights_at = dweights.data_ptr()
        elif (dweights.shape == per and dweights.dtype is f32 and dweights.get_device() == index and
              dweights.is_contiguous()):
            dweights_at = dweights.data_ptr()
        else:
            dweights_at = _per_place(route, dweights, "dweights", t, f32)
    elif dweights is not None:
        raise ValueError("dweights without rows")
    elif drows is not None and drows is not False:
        n = drows.shape[0]
    drows_at = drows_step = 0
    if drows is False:
        drows = None
    else:
        if drows is None:
            drows = _empty_on(stream, dy, (n, width))
        elif not (drows.shape == (n, width) and drows.dtype is dtype and drows.get_device() == index and
                  drows.is_contiguous()):
            drows_step = _matrix(drows, "drows", index, (n, width), dtype)
        drows_at = drows.data_ptr()
    call, pack = route.call_combine_backward
    rc = call(pack(rows_at, dy.data_ptr(), places_at, weights_at, drows_at, dweights_at,
                   0 if stream is None else _native.stream_handle(stream), t, n, rows_step, dy_step, drows_step, width, top_k,
                   code, 0))
    if rc:
        raise _native.CnsError(rc, "cns_combine_backward")
    return drows, dweights


def new_rms_norm(width: int, *, eps: float = 1e-6, y: bool = True, scale_block: int | None = None,
                 scale_type: int = _native.CNS_SCALE_F32, device=None):
    """A root-mean-square norm of rows of `width` columns (cns_rms_norm_t, see cns.h for the rules).  Its outputs: `y`
    in the rows' type, and, with scale_block, e4m3 values with scales, one for each block of 32, 64 or 128 columns, or
    one a row (0): float32 (CNS_SCALE_F32) or powers of two in 8 bits (CNS_SCALE_E8M0).  The handle holds no memory of
    the GPU."""
    torch = _torch()
    _dtype_codes()
    if not 1 <= width <= _native.CNS_NORM_MAX_WIDTH:
        raise ValueError(f"width: 1 to {_native.CNS_NORM_MAX_WIDTH} expected, got {width}")
    if scale_block not in (None, 0, 32, 64, 128):
        raise ValueError(f"scale_block: None, 0, 32, 64 or 128 expected, got {scale_block}")
    if not y and scale_block is None:
        raise ValueError("a norm with neither y nor 8-bit values")
    n = _native.RmsNorm()
    device = torch.device(device or "cuda")
    if device.type != "cuda":
        raise ValueError(f"a norm on {device}, a CUDA device expected")
    n.index = torch.cuda.current_device() if device.index is None else device.index
    n.others = torch.cuda.device_count() > 1
    n.has_y, n.has_q = y, scale_block is not None
    n.call = _native.packed_call("cns_rms_norm", _native.RmsNorm)
    n.call_backward = _native.packed_call("cns_rms_norm_backward", _native.RmsNormGrad)
    n.blocks = -(-width // scale_block) if scale_block else 1
    n.types = (torch.float8_e4m3fn, torch.float8_e8m0fnu if scale_type == _native.CNS_SCALE_E8M0 else torch.float32,
               torch.float32)
    n.width, n.scale_block, n.scale_type, n.eps = width, scale_block or 0, scale_type, eps
    return n


def _gain(norm, gain):
    """(address, cns_dtype_t) of a norm's gain."""
    if not (gain.is_contiguous() and gain.numel() == norm.width and gain.get_device() == norm.index):
        raise ValueError(f"gain: contiguous [{norm.width}] on CUDA device {norm.index} expected")
    return gain.data_ptr(), _dtype_code(gain.dtype)


def run_rms_norm(norm, x, gain=None, *, residual=None, h=None, y=None, q=None, scales=None, stream=None):
    """Normalise the rows of `x` ([rows, width], float32, bfloat16 or float16, rows at any stride) on `stream` (None:
    the default stream): h = x + residual, y = h / sqrt(mean(h^2) + eps) * gain, q and scales as new_rms_norm says.
    Returns (h, y, q, scales): h is x without a residual, and what the norm does not have is None.  The results go to
    the tensors given (h may be x or residual), or to new ones, of `stream`'s memory.  They are no part of torch's graph:
    run_rms_norm_backward has the gradient."""
    index, dtype, width = norm.index, x.dtype, norm.width
    if norm.others:
        _check_current(index)
    code = _CODES.get(dtype)
    if code is None:
        code = _dtype_code(dtype)
    t = x.shape[0]
    shape = (t, width)
    if width == 1 or t == norm.blocks == 1:
        _no_neg(x=x, gain=gain, residual=residual, h=h, y=y, scales=scales)
    x_step = 0 if x.shape == shape and x.get_device() == index and x.is_contiguous() else _matrix(x, "x", index, shape, dtype)
    gain_at, gain_code = (0, 0) if gain is None else _gain(norm, gain)
    residual_at = residual_step = h_at = h_step = y_at = y_step = q_at = q_step = scales_at = scales_step = 0
    if residual is not None:
        residual_at = residual.data_ptr()
        if not (residual.shape == shape and residual.dtype is dtype and residual.get_device() == index and
                residual.is_contiguous()):
            residual_step = _matrix(residual, "residual", index, shape, dtype)
        if h is None:
            h = _empty_on(stream, x, shape)
        elif not (h.shape == shape and h.dtype is dtype and h.get_device() == index and h.is_contiguous()):
            h_step = _matrix(h, "h", index, shape, dtype)
        h_at = h.data_ptr()
    elif h is not None:
        raise ValueError("h without a residual is x")
    else:
        h = x
    if norm.has_y:
        if y is None:
            y = _empty_on(stream, x, shape)
        elif not (y.shape == shape and y.dtype is dtype and y.get_device() == index and y.is_contiguous()):
            y_step = _matrix(y, "y", index, shape, dtype)
        y_at = y.data_ptr()
    elif y is not None:
        raise ValueError("y: this norm has none")
    if norm.has_q:
        (e4m3, kind, _), blocks = norm.types, (t, norm.blocks)
        if q is None:
            q = _empty_on(stream, x, shape, e4m3)
        elif not (q.shape == shape and q.dtype is e4m3 and q.get_device() == index and q.is_contiguous()):
            q_step = _matrix(q, "q", index, shape, e4m3)
        if scales is None:
            scales = _empty_on(stream, x, blocks, kind)
        elif not (scales.shape == blocks and scales.dtype is kind and scales.get_device() == index and
                  scales.is_contiguous()):
            scales_step = _matrix(scales, "scales", index, blocks, kind)
        q_at, scales_at = q.data_ptr(), scales.data_ptr()
    elif q is not None or scales is not None:
        raise ValueError("q, scales: this norm has none")
    call, pack = norm.call
    rc = call(pack(x.data_ptr(), residual_at, gain_at, h_at, y_at, q_at, scales_at,
                   0 if stream is None else _native.stream_handle(stream), t, x_step, residual_step, h_step, y_step, q_step,
                   scales_step, width, code, gain_code, norm.scale_block, norm.scale_type, norm.eps))
    if rc:
        raise _native.CnsError(rc, "cns_rms_norm")
    return h, y, q, scales


def run_rms_norm_backward(norm, h, gain, dy, *, dh=None, dx=None, dgain=None, workspace=None, stream=None):
    """The gradient of run_rms_norm from dL/dy and, through the residual's addition, dL/dh (optional), of the h that it
    returned: (dx, dgain).  dx is x's and the residual's, in h's type; dgain is float32 [width].  They go to `dx` (which
    may be dy or dh) and `dgain`, or to new tensors; without a gain, or with dgain False, dgain is None.  `workspace`:
    any tensor of cns_rms_norm_workspace_bytes that no other call uses meanwhile (default: a new one, of `stream`'s
    memory)."""
    index, dtype, width = norm.index, h.dtype, norm.width
    if norm.others:
        _check_current(index)
    code = _CODES.get(dtype)
    if code is None:
        code = _dtype_code(dtype)
    t = h.shape[0]
    shape = (t, width)
    if width == 1:
        _no_neg(h=h, gain=gain, dy=dy, dh=dh, dx=dx, dgain=dgain)
    gain_at, gain_code = (0, 0) if gain is None else _gain(norm, gain)
    h_step = 0 if h.shape == shape and h.get_device() == index and h.is_contiguous() else _matrix(h, "h", index, shape, dtype)
    dy_step = 0 if (dy.shape == shape and dy.dtype is dtype and dy.get_device() == index and
                    dy.is_contiguous()) else _matrix(dy, "dy", index, shape, dtype)
    dh_at = dh_step = dx_step = dgain_at = workspace_at = nbytes = 0
    if dh is not None:
        dh_at = dh.data_ptr()
        if not (dh.shape == shape and dh.dtype is dtype and dh.get_device() == index and dh.is_contiguous()):
            dh_step = _matrix(dh, "dh", index, shape, dtype)
    if dx is None:
        dx = _empty_on(stream, h, shape)
    elif not (dx.shape == shape and dx.dtype is dtype and dx.get_device() == index and dx.is_contiguous()):
        dx_step = _matrix(dx, "dx", index, shape, dtype)
    if dgain is False or (dgain is None and gain is None):
        dgain = None
    else:
        f32 = norm.types[2]
        if dgain is None:
            dgain = _empty_on(stream, h, (width,), f32)
        elif not (dgain.is_contiguous() and dgain.numel() == width and dgain.dtype is f32 and dgain.get_device() == index):
            raise ValueError(f"dgain: contiguous float32 [{width}] on CUDA device {index} expected")
        if workspace is None:
            rc, nbytes = _native.cns_rms_norm_workspace_bytes(t, width)
            _native.check(rc, "cns_rms_norm_workspace_bytes")
            workspace = _empty_on(stream, h, (nbytes // 4,), f32)
        elif workspace.is_contiguous() and workspace.get_device() == index:
            nbytes = workspace.nbytes
        else:
            raise ValueError(f"workspace: contiguous, on CUDA device {index} expected")
        dgain_at, workspace_at = dgain.data_ptr(), workspace.data_ptr()
    call, pack = norm.call_backward
    rc = call(pack(h.data_ptr(), gain_at, dy.data_ptr(), dh_at, dx.data_ptr(), dgain_at, workspace_at, nbytes,
                   0 if stream is None else _native.stream_handle(stream), t, h_step, dy_step, dh_step, dx_step, width, code,
                   gain_code, norm.eps))
    if rc:
        raise _native.CnsError(rc, "cns_rms_norm_backward")
    return dx, dgain


def _dense(t):
    """Whether the tensor's elements fill one stretch of memory, in whatever order of the axes."""
    if t.is_contiguous():
        return True
    at = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1):
        if stride != at:
            return False
        at *= size
    return True


def _same_layout(t, o):
    """Whether equal indices of two tensors of one shape are at equal distances from the start."""
    return t.numel() == 0 or all(a == b or n == 1 for a, b, n in zip(t.stride(), o.stride(), t.shape))


def _tensor_table(tensors, index, what):
    """(cns_tensor_t array, [(first byte, last byte + 1)]) of dense tensors on device `index`."""
    table = (_native.Tensor * max(len(tensors), 1))()
    spans = []
    for i, (t, e) in enumerate(zip(tensors, table)):
        if t.get_device() != index:
            raise ValueError(f"{what}[{i}]: on {t.device}, CUDA device {index} expected")
        if not _dense(t):
            raise ValueError(f"{what}[{i}]: not dense (strides {t.stride()})")
        n, at, code = t.numel(), t.data_ptr(), _dtype_code(t.dtype)
        e.data_dev, e.elems, e.dtype = at, n, code
        spans.append((at, at + n * (4 if code == _native.CNS_DT_F32 else 2)))
    return table, spans


def new_grad_clip(grads, max_norm: float = float("inf"), *, outs=None, eps: float = 1e-6,
                  norm_type: int = _native.CNS_NORM_L2, workspace=None, timeout_ms: int = 0, device=None, stream=None):
    """The gradients of a step (a list of dense tensors, float32, bfloat16 or float16 mixed as they come) and
    where their clipped values go: `outs`, tensors of the same shapes and strides, or in place.  Holds these
    tensors and their addresses: for others make another one.  A program that drops its gradients and lets torch make
    new ones (zero_grad() does, unless set_to_none=False) would go on clipping the old ones.
    `norm` is the float32 scalar that run_grad_norm and run_grad_clip fill.  Enqueues the zeroing of its workspace
    on torch's current stream: see new_step_workspace for the streams that are ordered behind it."""
    torch = _torch()
    _dtype_codes()
    g = _native.GradClip()
    grads, n = list(grads), len(grads)
    device = torch.device(device or (grads[0].device if n else "cuda"))
    if device.type != "cuda":
        raise ValueError(f"gradients on {device}, a CUDA device expected")
    g.norm = torch.empty((), dtype=torch.float32, device=device)
    index, g.others = g.norm.get_device(), torch.cuda.device_count() > 1
    g.index = index
    g.grad_table, spans = _tensor_table(grads, index, "grads")
    g.out_table = None
    if outs is None:
        spans = [(a, b, True, i) for i, (a, b) in enumerate(spans) if b > a]
    else:
        outs = list(outs)
        if len(outs) != n:
            raise ValueError("outs: one for each gradient expected")
        g.out_table, to = _tensor_table(outs, index, "outs")
        for i, (t, o) in enumerate(zip(grads, outs)):
            if t.shape != o.shape or not _same_layout(t, o):
                raise ValueError(f"outs[{i}]: the gradient's shape and strides expected")
        # an output that is its gradient is one tensor
        same = [a == b and t.dtype == o.dtype for a, b, t, o in zip(spans, to, grads, outs)]
        spans = ([(a, b, False, i) for i, ((a, b), s) in enumerate(zip(spans, same)) if b > a and not s] +
                 [(a, b, True, i) for i, (a, b) in enumerate(to) if b > a])
    spans.sort()
    end, written = (0, 0), (0, 0)   # how far the tensors so far reach, and those of them that are written
    for first, last, writes, i in spans:
        if first < written[0] or (writes and first < end[0]):
            raise ValueError(f"tensors {i} and {(written if first < written[0] else end)[1]} overlap")
        end = max(end, (last, i))
        if writes:
            written = max(written, (last, i))
    g.tensors = (grads, outs)   # alive as long as the table
    g.grads = g.grad_table
    if g.out_table is not None:
        g.outs = g.out_table
    g.count, g.max_norm, g.eps, g.norm_type, g.timeout_ms = n, max_norm, eps, norm_type, timeout_ms
    if workspace is None:
        rc, nbytes = _native.cns_grad_workspace_bytes(n)
        _native.check(rc, "new_grad_clip")
        workspace = new_step_workspace(nbytes, device, stream)
    g.workspace = workspace
    g.norm_dev, g.workspace_dev = g.norm.data_ptr(), workspace.data_ptr()
    g.workspace_bytes = workspace.numel() * workspace.element_size()
    return g


def run_grad_norm(plan, stream=None, sync: bool = False):
    """The global norm of new_grad_clip's gradients on `stream` (None: the default stream); returns plan.norm."""
    if plan.others:
        _check_current(plan.index)
    plan.stream = _native.stream_handle(stream)
    plan.sync = 1 if sync else 0
    rc = _native.cns_grad_norm(plan)
    if rc:
        raise _native.CnsError(rc, "cns_grad_norm")
    return plan.norm


def run_grad_clip(plan, stream=None, sync: bool = False):
    """Clip new_grad_clip's gradients by their global norm on `stream`; returns plan.norm, the norm before
    clipping."""
    if plan.others:
        _check_current(plan.index)
    plan.stream = _native.stream_handle(stream)
    plan.sync = 1 if sync else 0
    rc = _native.cns_grad_clip(plan)
    if rc:
        raise _native.CnsError(rc, "cns_grad_clip")
    return plan.norm
