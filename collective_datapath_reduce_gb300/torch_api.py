"""Torch-tensor front end over the C ABI, shaped like Purlin's Python API.

purlin 0.6.5 (PyPI page), Python section: `purlin.initialize(group, device,
arch, stream)` returns a handle, `purlin.all_reduce(x, out, handle, stream,
reduction_mode=...)` runs a collective, `purlin.finalize(handle, stream)`
frees the handle.  Here one process owns all ranks, so the "group" is just the
world size and every collective takes one tensor per rank.  Argument
marshalling only: checks shapes and dtypes, passes data pointers and byte
counts to libpurlin_gb.so and raises on a non-OK status.
"""

from __future__ import annotations

import enum
import operator
import threading
import types

import torch

from . import purlin as P


class ReductionMode(enum.IntEnum):
    DETERMINISTIC = P.PL_DETERMINISTIC


class Scores(enum.IntEnum):
    SOFTMAX = P.PL_SCORES_SOFTMAX
    SIGMOID = P.PL_SCORES_SIGMOID


_DTYPES = {torch.float32: P.PL_F32, torch.bfloat16: P.PL_BF16}
_Function = types.FunctionType


class Handle:
    def __init__(self, raw, world, device):
        self.raw, self.world, self.device = raw, world, device
        self.workspaces = {}  # of the operators, by stream
        self.lock = threading.RLock()  # held from taking one of them until the call's launches are queued

    def __repr__(self):
        return f"purlin.Handle(world={self.world}, device={self.device})"


def _stream(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(status, what):
    if status != P.PL_OK:
        raise P.PurlinError(status, what)


def _on(handle):
    """Make the handle's device current for the call (the C ABI requires it)."""
    return torch.cuda.device(handle.device)


def _same(tensors, world, what):
    """One contiguous CUDA (or pinned host) tensor per rank."""
    if len(tensors) != world:
        raise ValueError(f"{what}: expected {world} tensors (one per rank), got {len(tensors)}")
    for t in tensors:
        if not t.is_contiguous():
            raise ValueError(f"{what}: tensors must be contiguous")


def _resident(tensors, what):
    for t in tensors:
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{what}: tensors must be CUDA tensors or pinned host tensors")


def _nbytes(t):
    return t.numel() * t.element_size()


def _sizes(tensors, want, what, side):
    """Each tensor holds exactly want[r] bytes (the library cannot see
    allocation sizes, so a short tensor would be written past its end)."""
    for r, (t, w) in enumerate(zip(tensors, want)):
        if _nbytes(t) != w:
            raise ValueError(f"{what}: {side}[{r}] holds {_nbytes(t)} bytes, the collective needs {w}")


def _one_dtype(tensors, dtype, what):
    if any(t.dtype != dtype for t in tensors):
        raise ValueError(f"{what}: every tensor must have dtype {dtype}")


def _checked(what, handle, xs, outs, in_bytes, out_bytes, reduce=False):
    """Argument checks shared by the collectives, all before any library call:
    one tensor per rank on each side, one dtype (float32 or bfloat16 for the
    reductions), the exact byte size of every input and output, residency."""
    _same(xs, handle.world, what)
    _same(outs, handle.world, what)
    dtype = xs[0].dtype
    _one_dtype(list(xs) + list(outs), dtype, what)
    dt = _DTYPES.get(dtype)
    if reduce and dt is None:
        raise ValueError(f"{what}: float32 or bfloat16 tensors")
    _sizes(xs, in_bytes, what, "inputs")
    _sizes(outs, out_bytes, what, "outputs")
    _resident(list(xs) + list(outs), what)
    return dt


def initialize(world: int, device=None, stream=None) -> Handle:
    """Create a handle for `world` ranks on `device` (default: current device)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        st, raw = P.purlin_initialize(world, None, 0, _stream(stream, device))
    _check(st, "initialize")
    return Handle(raw, world, device)


def finalize(handle: Handle, stream=None) -> None:
    st = P.purlin_finalize(handle.raw, _stream(stream, handle.device))
    handle.raw = None
    handle.workspaces.clear()
    _check(st, "finalize")


def all_reduce(xs, outs, handle: Handle, stream=None, reduction_mode=ReductionMode.DETERMINISTIC):
    """outs[r] = sum over s of xs[s], for every rank r (outs may be xs: in place)."""
    b = _nbytes(xs[0]) if len(xs) else 0
    dt = _checked("all_reduce", handle, xs, outs, [b] * handle.world, [b] * handle.world, reduce=True)
    with _on(handle):
        _check(P.purlin_all_reduce(handle.raw, xs, outs, b, dt, int(reduction_mode),
                                   _stream(stream, handle.device)), "all_reduce")


def reduce_scatter(xs, outs, handle: Handle, stream=None, reduction_mode=ReductionMode.DETERMINISTIC):
    """outs[r] = chunk r (of world equal chunks along dim 0) of the sum of xs."""
    b = _nbytes(xs[0]) if len(xs) else 0
    if len(xs) and xs[0].numel() % handle.world:
        raise ValueError("reduce_scatter: the input length must split into world equal chunks")
    dt = _checked("reduce_scatter", handle, xs, outs, [b] * handle.world, [b // handle.world] * handle.world,
                  reduce=True)
    with _on(handle):
        _check(P.purlin_reduce_scatter(handle.raw, xs, outs, b, dt, int(reduction_mode),
                                       _stream(stream, handle.device)), "reduce_scatter")


def all_gather(xs, outs, handle: Handle, stream=None):
    """outs[r] = concatenation of xs along dim 0, for every rank r."""
    b = _nbytes(xs[0]) if len(xs) else 0
    _checked("all_gather", handle, xs, outs, [b] * handle.world, [handle.world * b] * handle.world)
    with _on(handle):
        _check(P.purlin_all_gather(handle.raw, xs, outs, b, _stream(stream, handle.device)), "all_gather")


def all_to_all(xs, outs, handle: Handle, stream=None):
    """outs[d] chunk s = xs[s] chunk d (world equal chunks along dim 0)."""
    b = _nbytes(xs[0]) if len(xs) else 0
    if len(xs) and xs[0].numel() % handle.world:
        raise ValueError("all_to_all: the length must split into world equal chunks")
    _checked("all_to_all", handle, xs, outs, [b] * handle.world, [b] * handle.world)
    with _on(handle):
        _check(P.purlin_all_to_all(handle.raw, xs, outs, b, _stream(stream, handle.device)), "all_to_all")


def all_gather_v(xs, outs, handle: Handle, stream=None):
    """outs[r] = concatenation of all of xs (each rank's tensor in full), packed in rank order."""
    _same(xs, handle.world, "all_gather_v")
    sizes = [_nbytes(t) for t in xs]
    _checked("all_gather_v", handle, xs, outs, sizes, [sum(sizes)] * handle.world)
    with _on(handle):
        _check(P.purlin_all_gather_v(handle.raw, xs, outs, sizes, _stream(stream, handle.device)), "all_gather_v")


def all_to_all_v(xs, outs, counts, handle: Handle, stream=None):
    """counts[s][d] elements go from rank s to rank d (packed, prefix-sum displacements)."""
    N = handle.world
    if len(counts) != N or any(len(row) != N for row in counts) or any(int(c) < 0 for row in counts for c in row):
        raise ValueError(f"all_to_all_v: counts must be {N} x {N} non-negative element counts")
    es = xs[0].element_size() if len(xs) else 1
    sent = [sum(int(c) for c in counts[s]) * es for s in range(N)]
    received = [sum(int(counts[s][d]) for s in range(N)) * es for d in range(N)]
    _checked("all_to_all_v", handle, xs, outs, sent, received)
    flat = [int(c) * es for row in counts for c in row]
    with _on(handle):
        _check(P.purlin_all_to_all_v(handle.raw, xs, outs, flat, _stream(stream, handle.device)), "all_to_all_v")


def reduce_scatter_v(xs, outs, counts, handle: Handle, stream=None, reduction_mode=ReductionMode.DETERMINISTIC):
    """outs[r] = the counts[r] elements of the sum starting at sum(counts[:r])."""
    N = handle.world
    if len(counts) != N or any(int(c) < 0 for c in counts):
        raise ValueError(f"reduce_scatter_v: counts must be {N} non-negative element counts")
    es = xs[0].element_size() if len(xs) else 1
    total = sum(int(c) for c in counts) * es
    dt = _checked("reduce_scatter_v", handle, xs, outs, [total] * N, [int(c) * es for c in counts], reduce=True)
    with _on(handle):
        _check(P.purlin_reduce_scatter_v(handle.raw, xs, outs, [int(c) * es for c in counts], dt, int(reduction_mode),
                                         _stream(stream, handle.device)), "reduce_scatter_v")


# --------------------------------------- operators around the collectives
#
# Outputs are the caller's, as for the collectives.  Matrices are 2-D tensors
# whose rows are packed (the last stride is 1) and any stride apart; vectors,
# picks and places are contiguous.  Workspaces come from torch's allocator and
# are kept by the handle, one for each stream.  Threads may call the operators
# on one handle at once.

def _values(t, what):
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{what}: float32 or bfloat16 tensors")
    return dt


def _resident_one(t, what):
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{what}: tensors must be CUDA tensors or pinned host tensors")


def _matrix(t, rows, width, dtype, what, name):
    """Checks a rows x width matrix and returns its row stride."""
    if t.shape != (rows, width):
        raise ValueError(f"{what}: {name} must be {rows} x {width}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{what}: {name} must have dtype {dtype}")
    stride, one = t.stride()
    if rows <= 1:
        stride = width
    if (one != 1 and width > 1) or stride < width:
        raise ValueError(f"{what}: {name} must have packed rows")
    if not t.is_cuda:
        _resident_one(t, what)
    return stride


def _packed(t, shape, dtype, what, name):
    if t.shape != shape:
        raise ValueError(f"{what}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{what}: {name} must have dtype {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: {name} must be contiguous")
    if not t.is_cuda:
        _resident_one(t, what)


def _two(t, what, name):
    if t.dim() != 2:
        raise ValueError(f"{what}: {name} must have two dimensions, got {tuple(t.shape)}")
    return t.shape


def _workspace(nbytes, stream, handle):
    """At least nbytes of device memory for a call on `stream`, taken with that
    stream current.  The handle's device is current already."""
    if nbytes == 0:
        return None
    device = handle.device
    index = device.index if device.index is not None else torch.cuda.current_device()
    current = torch._C._cuda_getCurrentRawStream(index)
    key = current if stream is None else _stream(stream, device)
    if key == current:
        return _block(nbytes, key, handle)
    with torch.cuda.stream(torch.cuda.ExternalStream(key, device=device)):
        return _block(nbytes, key, handle)


def _block(nbytes, key, handle):
    """The handle keeps one block for each stream, the largest that a call
    needed, until it is finalised; that stream's calls use it one after the
    other.  It comes from torch's allocator on the same stream, so a block that
    is replaced by a larger one is not handed on before its calls are done.  A
    captured call gets a block of its own, since the graph may replay anywhere:
    the graph's pool hands it on to later calls on the same stream only."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=handle.device)
    kept = handle.workspaces.get(key)
    if kept is None or kept.numel() < nbytes:
        kept = handle.workspaces[key] = torch.empty(nbytes, dtype=torch.uint8, device=handle.device)
    return kept


def _call(fn, what, handle, stream, *args):
    """fn(handle, *args, stream) with the handle's device current.  The guard
    of the device and the stream's object cost more than a small operator does,
    so both are skipped where the device is current already."""
    index = handle.device.index
    if index is None or torch.cuda.current_device() != index:
        with _on(handle):
            _check(fn(handle.raw, *args, _stream(stream, handle.device)), what)
        return
    stream = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream, handle.device)
    _check(fn(handle.raw, *args, stream), what)


def _call_in_workspace(fn, what, handle, stream, nbytes, *args):
    """_call with a workspace and its size behind args.  A call is several
    launches on one block, so no other thread's may come between them.  The
    library's own functions take an address, the binding's a tensor too."""
    if nbytes == 0:
        return _call(fn, what, handle, stream, *args, None, 0)
    index = handle.device.index
    if index is None or torch.cuda.current_device() != index:
        with _on(handle), handle.lock:
            ws = _workspace(nbytes, stream, handle)
            ws = ws if type(fn) is _Function else ws.data_ptr()
            return _check(fn(handle.raw, *args, ws, nbytes, _stream(stream, handle.device)), what)
    key = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream, handle.device)
    with handle.lock:
        ws = _block(nbytes, key, handle) if stream is None else _workspace(nbytes, key, handle)
        ws = ws if type(fn) is _Function else ws.data_ptr()
        _check(fn(handle.raw, *args, ws, nbytes, key), what)


def route_experts(logits, ids, weights, handle: Handle, bias=None, scores=Scores.SOFTMAX, groups=1, kept_groups=1,
                  group_best=1, renormalise=True, scale=1.0, stream=None):
    """ids[t, j], weights[t, j] = token t's j-th best expert and its weight.

    logits: tokens x experts (float32 or bfloat16); ids int32 and weights
    float32, tokens x top_k.  bias (float32, one per expert) orders the experts
    but is not part of the weights.  With groups > 1 only the kept_groups best
    runs of experts take part, each counted by its group_best (1 or 2) best
    experts.  Experts with logit -inf are never picked: missing picks have id
    -1 and weight 0."""
    what = "route_experts"
    T, E = _two(logits, what, "logits")
    k = _two(ids, what, "ids")[1]
    ld = _matrix(logits, T, E, logits.dtype, what, "logits")
    dt = _values(logits, what)
    _packed(ids, (T, k), torch.int32, what, "ids")
    _packed(weights, (T, k), torch.float32, what, "weights")
    if bias is not None:
        _packed(bias, (E,), torch.float32, what, "bias")
    routing = P.make_routing(E, k, scores, groups, kept_groups, group_best, renormalise, scale)
    _call(P.purlin_route_experts, what, handle, stream, logits, ld, dt, bias, T, routing, ids, weights)


def route_experts_grad(logits, ids, grad_weights, grad_logits, handle: Handle, scores=Scores.SOFTMAX, renormalise=True,
                       scale=1.0, stream=None):
    """grad_logits (like logits) = the gradient that grad_weights (like the
    weights) gives, the picks held fixed.  Groups and bias only choose the
    picks, so the gradient does not ask for them."""
    what = "route_experts_grad"
    T, E = _two(logits, what, "logits")
    k = _two(ids, what, "ids")[1]
    ld = _matrix(logits, T, E, logits.dtype, what, "logits")
    dt = _values(logits, what)
    _packed(ids, (T, k), torch.int32, what, "ids")
    _packed(grad_weights, (T, k), torch.float32, what, "grad_weights")
    ldg = _matrix(grad_logits, T, E, logits.dtype, what, "grad_logits")
    routing = P.make_routing(E, k, scores, renormalise=renormalise, scale=scale)
    _call(P.purlin_route_experts_grad, what, handle, stream, logits, ld, dt, T, routing, ids, grad_weights, grad_logits,
          ldg)


def expert_plan(ids, offsets, places, handle: Handle, stream=None):
    """places[t, j] = the row of pick ids[t, j] among all picks sorted by
    expert (equal ones by token and j); offsets[e] .. offsets[e + 1] are expert
    e's rows.  ids and places int32, tokens x top_k; offsets int32, experts + 1
    values.  A pick outside [0, experts) is dropped: its place is ~p, p a row
    past offsets[experts]."""
    what = "expert_plan"
    T, k = _two(ids, what, "ids")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"{what}: offsets must hold experts + 1 values, got {tuple(offsets.shape)}")
    E = offsets.shape[0] - 1
    _packed(ids, (T, k), torch.int32, what, "ids")
    _packed(places, (T, k), torch.int32, what, "places")
    _packed(offsets, (E + 1,), torch.int32, what, "offsets")
    nbytes = P.purlin_expert_plan_bytes(T, k, E)
    _call_in_workspace(P.purlin_expert_plan, what, handle, stream, nbytes, ids, T, k, E, offsets, places)


def dispatch_rows(x, places, rows, handle: Handle, stream=None):
    """rows[places[t, j]] = x[t]; rows of dropped picks are 0.  x: tokens x
    width; rows: (tokens x top_k) x width, of one dtype."""
    what = "dispatch_rows"
    T, D = _two(x, what, "x")
    k = _two(places, what, "places")[1]
    ldx = _matrix(x, T, D, x.dtype, what, "x")
    dt = _values(x, what)
    _packed(places, (T, k), torch.int32, what, "places")
    ldr = _matrix(rows, T * k, D, x.dtype, what, "rows")
    _call(P.purlin_dispatch_rows, what, handle, stream, x, ldx, places, T, k, D, dt, rows, ldr)


def combine_rows(rows, places, weights, y, handle: Handle, stream=None):
    """y[t] = the sum over j of weights[t, j] x rows[places[t, j]].  weights:
    float32, or None for all 1 (the gradient of dispatch_rows)."""
    what = "combine_rows"
    T, k = _two(places, what, "places")
    D = _two(y, what, "y")[1]
    ldr = _matrix(rows, T * k, D, y.dtype, what, "rows")
    dt = _values(y, what)
    _packed(places, (T, k), torch.int32, what, "places")
    if weights is not None:
        _packed(weights, (T, k), torch.float32, what, "weights")
    ldy = _matrix(y, T, D, y.dtype, what, "y")
    _call(P.purlin_combine_rows, what, handle, stream, rows, ldr, places, weights, T, k, D, dt, y, ldy)


def combine_rows_grad(rows, places, weights, grad_y, grad_rows, grad_weights, handle: Handle, stream=None):
    """grad_rows[places[t, j]] = weights[t, j] x grad_y[t], and grad_weights[t,
    j] = the product of rows[places[t, j]] and grad_y[t]."""
    what = "combine_rows_grad"
    T, k = _two(places, what, "places")
    D = _two(grad_y, what, "grad_y")[1]
    dt = _values(grad_y, what)
    ldr = _matrix(rows, T * k, D, grad_y.dtype, what, "rows")
    _packed(places, (T, k), torch.int32, what, "places")
    _packed(weights, (T, k), torch.float32, what, "weights")
    ldy = _matrix(grad_y, T, D, grad_y.dtype, what, "grad_y")
    ldg = _matrix(grad_rows, T * k, D, grad_y.dtype, what, "grad_rows")
    _packed(grad_weights, (T, k), torch.float32, what, "grad_weights")
    _call(P.purlin_combine_rows_grad, what, handle, stream, rows, ldr, places, weights, grad_y, ldy, T, k, D, dt,
          grad_rows, ldg, grad_weights)


def _tokens(tokens, what):
    if tokens.dim() != 1 or tokens.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"{what}: tokens must be a vector of int32 or int64")
    _packed(tokens, tokens.shape, tokens.dtype, what, "tokens")
    return tokens.shape[0], 8 if tokens.dtype is torch.int64 else 4


def embed(table, tokens, out, handle: Handle, first=0, scale=1.0, stream=None):
    """out[i] = scale x table[tokens[i] - first], 0 for a token outside the
    table's range of the vocabulary."""
    what = "embed"
    R, D = _two(table, what, "table")
    n, size = _tokens(tokens, what)
    ldt = _matrix(table, R, D, table.dtype, what, "table")
    dt = _values(table, what)
    ldo = _matrix(out, n, D, table.dtype, what, "out")
    _call(P.purlin_embed, what, handle, stream, table, ldt, R, int(first), tokens, size, n, D, scale, dt, out, ldo)


def embed_grad(grad_out, tokens, grad_table, handle: Handle, first=0, scale=1.0, base=None, stream=None):
    """grad_table[r] = base[r] + scale x the sum of grad_out[i] over the tokens
    with tokens[i] - first == r.  base: like grad_table, or None for 0; base is
    grad_table adds in place and touches only the rows that tokens name.
    grad_out and grad_table may have different dtypes."""
    what = "embed_grad"
    R, D = _two(grad_table, what, "grad_table")
    n, size = _tokens(tokens, what)
    dx, dt = _values(grad_out, what), _values(grad_table, what)
    ldx = _matrix(grad_out, n, D, grad_out.dtype, what, "grad_out")
    ldt = _matrix(grad_table, R, D, grad_table.dtype, what, "grad_table")
    ldb = _matrix(base, R, D, grad_table.dtype, what, "base") if base is not None else 0
    nbytes = P.purlin_embed_grad_bytes(n, R, D)
    _call_in_workspace(P.purlin_embed_grad, what, handle, stream, nbytes, grad_out, ldx, dx, tokens, size, n, D, scale,
                       base, ldb, grad_table, ldt, dt, R, int(first))


# The row operators' calls are short, and the host's: checks ask a contiguous
# tensor of the right shape and type four questions, and the library is called
# with addresses.

def _rows_of(t, shape, dtype, what, name):
    """Checks a matrix of the given shape and returns its row stride."""
    if t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.is_cuda:
        return shape[1]
    return _matrix(t, shape[0], shape[1], dtype, what, name)


def _vector_of(t, shape, dtype, what, name):
    """Checks a packed tensor and returns its address."""
    if not (t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.is_cuda):
        _packed(t, shape, dtype, what, name)
    return t.data_ptr()


_F32 = torch.float32


def layer_norm(x, weight, bias, y, handle: Handle, residual=None, total=None, stats=None, eps=1e-5, stream=None):
    """y = the layer norm of x + residual (rounded to their dtype, which total
    receives), times weight, plus bias.  x, residual, total, y: tokens x width of
    one dtype; weight, bias: width values of one dtype, or None for 1 and 0;
    residual, total, stats may be None.  stats: float32, tokens x 2, each row's
    mean and 1 / deviation, for the gradient.  y and total may each be x or
    residual itself."""
    what = "layer_norm"
    shape, dtype = x.shape, x.dtype
    T, D = shape if len(shape) == 2 else _two(x, what, "x")
    dt = _values(x, what)
    ldx = _rows_of(x, shape, dtype, what, "x")
    ldy = _rows_of(y, shape, dtype, what, "y")
    r, ldr = (None, 0) if residual is None else (residual.data_ptr(), _rows_of(residual, shape, dtype, what, "residual"))
    t, ldt = (None, 0) if total is None else (total.data_ptr(), _rows_of(total, shape, dtype, what, "total"))
    of = weight if weight is not None else bias
    dw, wtype = (P.PL_F32, None) if of is None else (_values(of, what), of.dtype)
    w = None if weight is None else _vector_of(weight, (D,), wtype, what, "weight")
    b = None if bias is None else _vector_of(bias, (D,), wtype, what, "bias")
    s = None if stats is None else _vector_of(stats, (T, 2), _F32, what, "stats")
    _call(P.load().purlin_layer_norm, what, handle, stream, x.data_ptr(), ldx, r, ldr, T, D, dt, w, b, dw, eps, y.data_ptr(),
          ldy, t, ldt, s)


def layer_norm_grad(grad_y, x, stats, weight, grad_x, grad_weight, grad_bias, handle: Handle, grad_total=None,
                    stream=None):
    """grad_x = the gradient of the normalised rows x (layer_norm's total, where
    it had a residual, whose gradient it is too), plus grad_total; grad_weight
    and grad_bias = those of weight and bias, in one dtype, each may be None.
    weight: None for 1.  grad_x may be grad_y, x or grad_total itself."""
    what = "layer_norm_grad"
    shape, dtype = grad_y.shape, grad_y.dtype
    T, D = shape if len(shape) == 2 else _two(grad_y, what, "grad_y")
    dt = _values(grad_y, what)
    ldg = _rows_of(grad_y, shape, dtype, what, "grad_y")
    ldx = _rows_of(x, shape, dtype, what, "x")
    s = _vector_of(stats, (T, 2), _F32, what, "stats")
    t, ldt = (None, 0) if grad_total is None else (grad_total.data_ptr(),
                                                   _rows_of(grad_total, shape, dtype, what, "grad_total"))
    ldo = _rows_of(grad_x, shape, dtype, what, "grad_x")
    of = weight if weight is not None else grad_weight if grad_weight is not None else grad_bias
    dw, wtype = (P.PL_F32, None) if of is None else (_values(of, what), of.dtype)
    w = None if weight is None else _vector_of(weight, (D,), wtype, what, "weight")
    gw = None if grad_weight is None else _vector_of(grad_weight, (D,), wtype, what, "grad_weight")
    gb = None if grad_bias is None else _vector_of(grad_bias, (D,), wtype, what, "grad_bias")
    lib = P.load()
    nbytes = 0 if gw is None and gb is None else lib.purlin_layer_norm_grad_bytes(T, D)
    _call_in_workspace(lib.purlin_layer_norm_grad, what, handle, stream, nbytes, grad_y.data_ptr(), ldg, x.data_ptr(), ldx, s,
                       T, D, dt, w, dw, t, ldt, grad_x.data_ptr(), ldo, gw, gb)


def balance_loss(logits, ids, counts, sums, loss, handle: Handle, scores=Scores.SOFTMAX, scale=1.0, stream=None):
    """counts[e] = how many of the picks are expert e's; sums = the same, then the
    sums of the experts' shares of the scores over the tokens that have picks,
    then the number of these; loss[0] = scale x experts x the mean share of an
    expert's scores times its share of the picks, added up.  logits and ids as in
    route_experts; counts: int32, experts values; sums: float32, 2 x experts + 1;
    loss: one float32, or None where the sums of several ranks are added first
    (all_reduce, then balance_join)."""
    what = "balance_loss"
    T, E = _two(logits, what, "logits")
    k = _two(ids, what, "ids")[1]
    ld = _rows_of(logits, (T, E), logits.dtype, what, "logits")
    dt = _values(logits, what)
    i = _vector_of(ids, (T, k), torch.int32, what, "ids")
    c = _vector_of(counts, (E,), torch.int32, what, "counts")
    s = _vector_of(sums, (2 * E + 1,), _F32, what, "sums")
    of = None if loss is None else _vector_of(loss, (1,), _F32, what, "loss")
    lib = P.load()
    _call_in_workspace(lib.purlin_balance_loss, what, handle, stream, lib.purlin_balance_loss_bytes(T, E), logits.data_ptr(),
                       ld, dt, i, T, k, E, int(scores), scale, c, s, of)


def balance_join(sums, loss, handle: Handle, scale=1.0, stream=None):
    """loss[0] = balance_loss's of the sums, which may be those of all ranks."""
    what = "balance_join"
    if sums.dim() != 1 or sums.shape[0] < 3 or sums.shape[0] % 2 == 0:
        raise ValueError(f"{what}: sums must hold 2 x experts + 1 values, got {tuple(sums.shape)}")
    s = _vector_of(sums, sums.shape, _F32, what, "sums")
    of = _vector_of(loss, (1,), _F32, what, "loss")
    _call(P.load().purlin_balance_join, what, handle, stream, s, sums.shape[0] // 2, scale, of)


def balance_loss_grad(logits, ids, sums, grad_loss, grad_logits, handle: Handle, scores=Scores.SOFTMAX, scale=1.0,
                      base=None, stream=None):
    """grad_logits = base + grad_loss[0] x the gradient of the loss that sums give,
    the picks held fixed.  grad_loss: one float32, or None for 1.  base: like
    grad_logits, or None for 0; base is grad_logits adds in place (to
    route_experts_grad's, say)."""
    what = "balance_loss_grad"
    T, E = shape = _two(logits, what, "logits")
    k = _two(ids, what, "ids")[1]
    dtype = logits.dtype
    ld = _rows_of(logits, shape, dtype, what, "logits")
    dt = _values(logits, what)
    i = _vector_of(ids, (T, k), torch.int32, what, "ids")
    s = _vector_of(sums, (2 * E + 1,), _F32, what, "sums")
    g = None if grad_loss is None else _vector_of(grad_loss, (1,), _F32, what, "grad_loss")
    b, ldb = (None, 0) if base is None else (base.data_ptr(), _rows_of(base, shape, dtype, what, "base"))
    ldg = _rows_of(grad_logits, shape, dtype, what, "grad_logits")
    _call(P.load().purlin_balance_loss_grad, what, handle, stream, logits.data_ptr(), ld, dt, i, T, k, E, int(scores), scale, s,
          g, b, ldb, grad_logits.data_ptr(), ldg)


def _teacher(logits, ids, teacher, what, first, vocabulary, temperature, scale):
    """Checks what the distillation's calls share: (tokens, width, stride, dtype, a
    reference to the C struct, addresses of ids and teacher)."""
    T, R = _two(logits, what, "logits")
    k = _two(ids, what, "ids")[1]
    ld = _rows_of(logits, (T, R), logits.dtype, what, "logits")
    dt = _values(logits, what)
    wide = ids.dtype is torch.int64
    if not wide and ids.dtype is not torch.int32:
        raise ValueError(f"{what}: ids must be int32 or int64")
    i = _vector_of(ids, (T, k), ids.dtype, what, "ids")
    dq = _values(teacher, what)
    t = _vector_of(teacher, (T, k), teacher.dtype, what, "teacher")
    d = P.make_distillation(R, first, first + R if vocabulary is None else vocabulary, k, 8 if wide else 4, dq, temperature,
                            scale)
    return T, R, ld, dt, P.ctypes.byref(d), i, t


def distil_loss(logits, ids, teacher, loss, stats, handle: Handle, temperature=1.0, scale=1.0, stream=None):
    """loss[t] = scale x the Kullback-Leibler divergence of the softmax of
    logits[t] / temperature from that of teacher[t] / temperature over the words
    ids[t]; ids outside the vocabulary are no picks, and a token without picks has
    loss 0.  logits: tokens x vocabulary; ids (int32 or int64) and teacher
    (float32 or bfloat16): tokens x picks; loss: float32, one for each token;
    stats: float32, tokens x 2, for the gradient."""
    what = "distil_loss"
    T, _, ld, dt, d, i, t = _teacher(logits, ids, teacher, what, 0, None, temperature, scale)
    of = _vector_of(loss, (T,), _F32, what, "loss")
    s = _vector_of(stats, (T, 2), _F32, what, "stats")
    _call(P.load().purlin_distil_loss, what, handle, stream, logits.data_ptr(), ld, dt, T, d, i, t, of, s)


def distil_parts(logits, ids, teacher, parts, handle: Handle, first=0, vocabulary=None, temperature=1.0, stream=None):
    """parts (float32, tokens x 4) = what distil_join needs of one range of the
    vocabulary.  logits: tokens x words, those of the words first .. first +
    words; vocabulary: the words of all ranges (None: this is the last)."""
    what = "distil_parts"
    T, _, ld, dt, d, i, t = _teacher(logits, ids, teacher, what, first, vocabulary, temperature, 1.0)
    p = _vector_of(parts, (T, 4), _F32, what, "parts")
    _call(P.load().purlin_distil_parts, what, handle, stream, logits.data_ptr(), ld, dt, T, d, i, t, p)


def distil_join(parts, loss, stats, handle: Handle, temperature=1.0, scale=1.0, stream=None):
    """loss and stats as distil_loss gives them, from the parts of all ranges:
    ranges x tokens x 4, or (ranges x tokens) x 4, as all_gather leaves them."""
    what = "distil_join"
    T = loss.numel()
    ranges = parts.numel() // (4 * T) if T else 1
    if parts.shape[-1:] != (4,) or ranges == 0 or parts.numel() != 4 * T * ranges:
        raise ValueError(f"{what}: parts must be ranges x {T} x 4, got {tuple(parts.shape)}")
    p = _vector_of(parts, parts.shape, _F32, what, "parts")
    of = _vector_of(loss, (T,), _F32, what, "loss")
    s = _vector_of(stats, (T, 2), _F32, what, "stats")
    _call(P.load().purlin_distil_join, what, handle, stream, p, ranges, T, temperature, scale, of, s)


def distil_loss_grad(logits, ids, teacher, stats, grad_loss, grad_logits, handle: Handle, first=0, vocabulary=None,
                     temperature=1.0, scale=1.0, stream=None):
    """grad_logits (like logits, or logits itself) = grad_loss[t] x the gradient of
    loss[t], for a range's logits too, given the whole vocabulary's stats."""
    what = "distil_loss_grad"
    T, R, ld, dt, d, i, t = _teacher(logits, ids, teacher, what, first, vocabulary, temperature, scale)
    s = _vector_of(stats, (T, 2), _F32, what, "stats")
    g = _vector_of(grad_loss, (T,), _F32, what, "grad_loss")
    ldg = _rows_of(grad_logits, (T, R), logits.dtype, what, "grad_logits")
    _call(P.load().purlin_distil_loss_grad, what, handle, stream, logits.data_ptr(), ld, dt, T, d, i, t, s, g,
          grad_logits.data_ptr(), ldg)


_numel, _data_ptr, _is_contiguous = torch.Tensor.numel, torch.Tensor.data_ptr, torch.Tensor.is_contiguous
_dtype_of = operator.attrgetter("dtype")


def clip_grad_norm(grads, outs, max_norm, norm, handle: Handle, scale=1.0, stream=None):
    """norm[0] = |scale| x the 2-norm of all grads together; outs[i] = grads[i] x
    scale x min(1, max_norm / (norm + 1e-6)).  grads: contiguous tensors of any
    shapes and one dtype; outs: as many of the same sizes, or the grads
    themselves (in place), or None for the norm alone; norm: one float32."""
    what = "clip_grad_norm"
    _packed(norm, (1,), torch.float32, what, "norm")
    if outs is not None and len(outs) != len(grads):
        raise ValueError(f"{what}: expected {len(grads)} outputs, got {len(outs)}")
    # whole columns at a time: for many tensors this is what the call takes
    dt, counts = P.PL_F32, list(map(_numel, grads))
    if counts:
        dt = _values(grads[0], what)
        for side in (grads,) if outs is None or outs is grads else (grads, outs):
            # where each tensor lives is checked by the library, for all of them
            if set(map(_dtype_of, side)) != {grads[0].dtype} or not all(map(_is_contiguous, side)):
                raise ValueError(f"{what}: gradients and outputs must be contiguous tensors of one dtype")
        if outs is not None and outs is not grads and list(map(_numel, outs)) != counts:
            raise ValueError(f"{what}: each output must have its gradient's size")
    nbytes = P.purlin_clip_grad_norm_bytes()
    _call_in_workspace(P.purlin_clip_grad_norm, what, handle, stream, nbytes, list(map(_data_ptr, grads)),
                       None if outs is None else list(map(_data_ptr, outs)), counts, dt, scale, max_norm, norm)
