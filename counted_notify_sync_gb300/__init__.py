"""counted_notify_sync_gb300: SYNCALL epoch barrier and CntNotify on GB300, and device-wide steps of a
training step (routing to experts, gradient norm and clipping).

The C ABI (include/cns.h, libcns.so) does all the work; this package is the
thin Python side: ``_native`` mirrors the C entry points one to one, and the
helpers below allocate device buffers with PyTorch and marshal arguments.
"""
from __future__ import annotations

from . import _native
from ._native import *  # noqa: F401,F403  (C names and constants)

__all__ = [n for n in dir(_native) if not n.startswith("_")] + [
    "build", "new_workspace", "run_syncall", "run_statemachine", "run_pipeline",
    "new_step_workspace", "new_route", "run_route", "run_route_backward", "new_grad_clip", "run_grad_norm",
    "run_grad_clip",
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
# run_route_backward only reads the handle: gradients may be taken from several threads at once.  A handle's device
# has to be the current one at each call.

_CODES = {}   # torch dtype -> cns_dtype_t, filled by the first new_route or new_grad_clip


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


def _empty_on(stream, like, shape):
    """A tensor whose memory is the stream's that the call runs on: torch hands out what calls of its own stream may
    still be using, which comes before that stream's work alone."""
    import torch
    handle = _native.stream_handle(stream) or 0
    if torch.cuda.current_stream().cuda_stream == handle:
        return like.new_empty(shape)
    with torch.cuda.stream(torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()):
        return like.new_empty(shape)


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
