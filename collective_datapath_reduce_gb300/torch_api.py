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

import torch

from . import purlin as P


class ReductionMode(enum.IntEnum):
    DETERMINISTIC = P.PL_DETERMINISTIC


class Scores(enum.IntEnum):
    SOFTMAX = P.PL_SCORES_SOFTMAX
    SIGMOID = P.PL_SCORES_SIGMOID


_DTYPES = {torch.float32: P.PL_F32, torch.bfloat16: P.PL_BF16}


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
    launches on one block, so no other thread's may come between them."""
    if nbytes == 0:
        return _call(fn, what, handle, stream, *args, None, 0)
    index = handle.device.index
    if index is None or torch.cuda.current_device() != index:
        with _on(handle), handle.lock:
            ws = _workspace(nbytes, stream, handle)
            return _check(fn(handle.raw, *args, ws, nbytes, _stream(stream, handle.device)), what)
    key = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream, handle.device)
    with handle.lock:
        ws = _block(nbytes, key, handle) if stream is None else _workspace(nbytes, key, handle)
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


def _vector(t, n, dtype, what, name):
    """Checks a vector of n columns that may be None."""
    if t is not None:
        _packed(t, (n,), dtype, what, name)


def layer_norm(x, weight, bias, y, handle: Handle, residual=None, total=None, stats=None, eps=1e-5, stream=None):
    """y = the layer norm of x + residual (rounded to their dtype, which total
    receives), times weight, plus bias.  x, residual, total, y: tokens x width of
    one dtype; weight, bias: width values of one dtype, or None for 1 and 0;
    residual, total, stats may be None.  stats: float32, tokens x 2, each row's
    mean and 1 / deviation, for the gradient.  y and total may each be x or
    residual itself."""
    what = "layer_norm"
    T, D = _two(x, what, "x")
    dt = _values(x, what)
    ldx = _matrix(x, T, D, x.dtype, what, "x")
    ldy = _matrix(y, T, D, x.dtype, what, "y")
    ldr = _matrix(residual, T, D, x.dtype, what, "residual") if residual is not None else 0
    ldt = _matrix(total, T, D, x.dtype, what, "total") if total is not None else 0
    of = weight if weight is not None else bias
    dw = P.PL_F32 if of is None else _values(of, what)
    _vector(weight, D, of.dtype if of is not None else None, what, "weight")
    _vector(bias, D, of.dtype if of is not None else None, what, "bias")
    if stats is not None:
        _packed(stats, (T, 2), torch.float32, what, "stats")
    _call(P.purlin_layer_norm, what, handle, stream, x, ldx, residual, ldr, T, D, dt, weight, bias, dw, eps, y, ldy, total,
          ldt, stats)


def layer_norm_grad(grad_y, x, stats, weight, grad_x, grad_weight, grad_bias, handle: Handle, grad_total=None,
                    stream=None):
    """grad_x = the gradient of the normalised rows x (layer_norm's total, where
    it had a residual, whose gradient it is too), plus grad_total; grad_weight
    and grad_bias = those of weight and bias, in one dtype, each may be None.
    weight: None for 1.  grad_x may be grad_y, x or grad_total itself."""
    what = "layer_norm_grad"
    T, D = _two(grad_y, what, "grad_y")
    dt = _values(grad_y, what)
    ldg = _matrix(grad_y, T, D, grad_y.dtype, what, "grad_y")
    ldx = _matrix(x, T, D, grad_y.dtype, what, "x")
    _packed(stats, (T, 2), torch.float32, what, "stats")
    ldt = _matrix(grad_total, T, D, grad_y.dtype, what, "grad_total") if grad_total is not None else 0
    ldo = _matrix(grad_x, T, D, grad_y.dtype, what, "grad_x")
    of = weight if weight is not None else grad_weight if grad_weight is not None else grad_bias
    dw, dtype = (P.PL_F32, None) if of is None else (_values(of, what), of.dtype)
    _vector(weight, D, dtype, what, "weight")
    _vector(grad_weight, D, dtype, what, "grad_weight")
    _vector(grad_bias, D, dtype, what, "grad_bias")
    nbytes = P.purlin_layer_norm_grad_bytes(T, D) if grad_weight is not None or grad_bias is not None else 0
    _call_in_workspace(P.purlin_layer_norm_grad, what, handle, stream, nbytes, grad_y, ldg, x, ldx, stats, T, D, dt, weight,
                       dw, grad_total, ldt, grad_x, ldo, grad_weight, grad_bias)


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
    ld = _matrix(logits, T, E, logits.dtype, what, "logits")
    dt = _values(logits, what)
    _packed(ids, (T, k), torch.int32, what, "ids")
    _packed(counts, (E,), torch.int32, what, "counts")
    _packed(sums, (2 * E + 1,), torch.float32, what, "sums")
    if loss is not None:
        _packed(loss, (1,), torch.float32, what, "loss")
    nbytes = P.purlin_balance_loss_bytes(T, E)
    _call_in_workspace(P.purlin_balance_loss, what, handle, stream, nbytes, logits, ld, dt, ids, T, k, E, int(scores), scale,
                       counts, sums, loss)


def balance_join(sums, loss, handle: Handle, scale=1.0, stream=None):
    """loss[0] = balance_loss's of the sums, which may be those of all ranks."""
    what = "balance_join"
    if sums.dim() != 1 or sums.shape[0] < 3 or sums.shape[0] % 2 == 0:
        raise ValueError(f"{what}: sums must hold 2 x experts + 1 values, got {tuple(sums.shape)}")
    _packed(sums, sums.shape, torch.float32, what, "sums")
    _packed(loss, (1,), torch.float32, what, "loss")
    _call(P.purlin_balance_join, what, handle, stream, sums, sums.shape[0] // 2, scale, loss)


def balance_loss_grad(logits, ids, sums, grad_loss, grad_logits, handle: Handle, scores=Scores.SOFTMAX, scale=1.0,
                      base=None, stream=None):
    """grad_logits = base + grad_loss[0] x the gradient of the loss that sums give,
    the picks held fixed.  grad_loss: one float32, or None for 1.  base: like
    grad_logits, or None for 0; base is grad_logits adds in place (to
    route_experts_grad's, say)."""
    what = "balance_loss_grad"
    T, E = _two(logits, what, "logits")
    k = _two(ids, what, "ids")[1]
    ld = _matrix(logits, T, E, logits.dtype, what, "logits")
    dt = _values(logits, what)
    _packed(ids, (T, k), torch.int32, what, "ids")
    _packed(sums, (2 * E + 1,), torch.float32, what, "sums")
    if grad_loss is not None:
        _packed(grad_loss, (1,), torch.float32, what, "grad_loss")
    ldb = _matrix(base, T, E, logits.dtype, what, "base") if base is not None else 0
    ldg = _matrix(grad_logits, T, E, logits.dtype, what, "grad_logits")
    _call(P.purlin_balance_loss_grad, what, handle, stream, logits, ld, dt, ids, T, k, E, int(scores), scale, sums,
          grad_loss, base, ldb, grad_logits, ldg)


def _teacher(logits, ids, teacher, what, first, vocabulary, temperature, scale):
    """Checks what the distillation's calls share: (tokens, width, stride, dtype, the C struct)."""
    T, R = _two(logits, what, "logits")
    k = _two(ids, what, "ids")[1]
    ld = _matrix(logits, T, R, logits.dtype, what, "logits")
    dt = _values(logits, what)
    if ids.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"{what}: ids must be int32 or int64")
    _packed(ids, (T, k), ids.dtype, what, "ids")
    dq = _values(teacher, what)
    _packed(teacher, (T, k), teacher.dtype, what, "teacher")
    return T, R, ld, dt, P.make_distillation(R, first, first + R if vocabulary is None else vocabulary, k,
                                             8 if ids.dtype is torch.int64 else 4, dq, temperature, scale)


def distil_loss(logits, ids, teacher, loss, stats, handle: Handle, temperature=1.0, scale=1.0, stream=None):
    """loss[t] = scale x the Kullback-Leibler divergence of the softmax of
    logits[t] / temperature from that of teacher[t] / temperature over the words
    ids[t]; ids outside the vocabulary are no picks, and a token without picks has
    loss 0.  logits: tokens x vocabulary; ids (int32 or int64) and teacher
    (float32 or bfloat16): tokens x picks; loss: float32, one for each token;
    stats: float32, tokens x 2, for the gradient."""
    what = "distil_loss"
    T, _, ld, dt, d = _teacher(logits, ids, teacher, what, 0, None, temperature, scale)
    _packed(loss, (T,), torch.float32, what, "loss")
    _packed(stats, (T, 2), torch.float32, what, "stats")
    _call(P.purlin_distil_loss, what, handle, stream, logits, ld, dt, T, d, ids, teacher, loss, stats)


def distil_parts(logits, ids, teacher, parts, handle: Handle, first=0, vocabulary=None, temperature=1.0, stream=None):
    """parts (float32, tokens x 4) = what distil_join needs of one range of the
    vocabulary.  logits: tokens x words, those of the words first .. first +
    words; vocabulary: the words of all ranges (None: this is the last)."""
    what = "distil_parts"
    T, _, ld, dt, d = _teacher(logits, ids, teacher, what, first, vocabulary, temperature, 1.0)
    _packed(parts, (T, 4), torch.float32, what, "parts")
    _call(P.purlin_distil_parts, what, handle, stream, logits, ld, dt, T, d, ids, teacher, parts)


def distil_join(parts, loss, stats, handle: Handle, temperature=1.0, scale=1.0, stream=None):
    """loss and stats as distil_loss gives them, from the parts of all ranges:
    ranges x tokens x 4, or (ranges x tokens) x 4, as all_gather leaves them."""
    what = "distil_join"
    T = loss.numel()
    ranges = parts.numel() // (4 * T) if T else 1
    if parts.shape[-1:] != (4,) or ranges == 0 or parts.numel() != 4 * T * ranges:
        raise ValueError(f"{what}: parts must be ranges x {T} x 4, got {tuple(parts.shape)}")
    _packed(parts, parts.shape, torch.float32, what, "parts")
    _packed(loss, (T,), torch.float32, what, "loss")
    _packed(stats, (T, 2), torch.float32, what, "stats")
    _call(P.purlin_distil_join, what, handle, stream, parts, ranges, T, temperature, scale, loss, stats)


def distil_loss_grad(logits, ids, teacher, stats, grad_loss, grad_logits, handle: Handle, first=0, vocabulary=None,
                     temperature=1.0, scale=1.0, stream=None):
    """grad_logits (like logits, or logits itself) = grad_loss[t] x the gradient of
    loss[t], for a range's logits too, given the whole vocabulary's stats."""
    what = "distil_loss_grad"
    T, R, ld, dt, d = _teacher(logits, ids, teacher, what, first, vocabulary, temperature, scale)
    _packed(stats, (T, 2), torch.float32, what, "stats")
    _packed(grad_loss, (T,), torch.float32, what, "grad_loss")
    ldg = _matrix(grad_logits, T, R, logits.dtype, what, "grad_logits")
    _call(P.purlin_distil_loss_grad, what, handle, stream, logits, ld, dt, T, d, ids, teacher, stats, grad_loss, grad_logits,
          ldg)


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
