"""The index-driven operators around the collectives, as cases to measure.

Expert routing decides what an all-to-all-v carries; plan, dispatch and combine
pack token rows by expert and sum them back; the embedding looks rows up in one
rank's range of the vocabulary, whose parts an all-reduce sums; the clip takes
the global norm of the gradients that a reduce-scatter or all-reduce left.

Every operator has a plain form here (elementary torch operations in 32 bits,
rounded once) and is called through the framework's torch front end where
`own` is true.
"""

import math

import numpy as np
import torch

own = False

_DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}
_DEVICE = torch.device("cuda" if torch.cuda.is_available() else "cpu")
_handles = []


def listed():
    return [
        # One token of a decoding request picks 6 of 64 experts: latency only.
        _route("route, one token", "forward", 1, 64, 6, "softmax", "float32"),
        # A long prefill batch: sigmoid scores, balance bias, 4 of 8 groups kept by their two best, renormalised.
        _route("route, grouped prefill", "forward", 16384, 256, 8, "sigmoid", "float32",
               bias=True, groups=8, kept_groups=4, group_best=2, scale=2.5),
        # The router's gradient in a training step with a ragged batch, whose padding tokens have no expert left.
        _route("route, training gradient", "backward", 8191, 60, 4, "softmax", "bfloat16", empty=0.03),
        # A decoding batch of 17 requests is packed for the exchange: plan and copy, both small.
        _exchange("dispatch, decode batch", "dispatch", 17, 2048, 128, 8, "bfloat16"),
        # A training micro-batch is packed for the exchange: one read of each token, eight copies.
        _exchange("dispatch, training", "dispatch", 8192, 4096, 256, 8, "bfloat16"),
        # Expert outputs in 32 bits come back to an odd number of tokens at an odd width.
        _exchange("combine, ragged 32-bit", "combine", 3001, 1537, 32, 6, "float32", empty=0.05),
        # The gradient of the weighted sum: rows' gradients, and a product of two rows for each weight.
        _exchange("combine, training gradient", "combine_grad", 8192, 2048, 64, 6, "bfloat16"),
        # Next tokens of 8 requests, scaled by the root of the width.
        _embed("embed, decode batch", "forward", 8, 4096, 32000, 32000, 0, 64.0, "bfloat16", "bfloat16", False),
        # A prefill looks up one rank's quarter of the vocabulary; the other ranks' tokens give zero rows.
        _embed("embed, vocabulary range", "forward", 32768, 5120, 131072, 32768, 32768, 1.0, "bfloat16", "bfloat16", False),
        # A training step's dense table gradient from tokens as frequent as words are.
        _embed("embed, dense gradient", "backward", 16384, 4096, 65536, 65536, 0, 64.0, "bfloat16", "bfloat16", False),
        # A small model's gradients: few tensors, odd lengths.
        _clip("clip, small model", 14, 4001, "bfloat16"),
        # A large rank's shard of gradients, mean over 8 ranks taken on the way.
        _clip("clip, large shard", 180, 3000007, "float32", scale=0.125),
    ]


def _route(name, direction, tokens, experts, top_k, scores, dtype, bias=False, groups=1, kept_groups=1, group_best=1,
           renormalise=True, scale=1.0, empty=0.0):
    return {"name": name, "op": "route", "direction": direction, "tokens": tokens, "experts": experts, "top_k": top_k,
            "scores": scores, "dtype": dtype, "bias": bias, "groups": groups, "kept_groups": kept_groups,
            "group_best": group_best, "renormalise": renormalise, "scale": scale, "empty": empty}


def _exchange(name, direction, tokens, width, experts, top_k, dtype, empty=0.0):
    return {"name": name, "op": "exchange", "direction": direction, "tokens": tokens, "width": width,
            "experts": experts, "top_k": top_k, "dtype": dtype, "empty": empty}


def _embed(name, direction, tokens, width, vocabulary, rows, first, scale, dtype, table_dtype, accumulate):
    return {"name": name, "op": "embed", "direction": direction, "tokens": tokens, "width": width,
            "vocabulary": vocabulary, "rows": rows, "first": first, "scale": scale, "dtype": dtype,
            "table_dtype": table_dtype, "accumulate": accumulate}


def _clip(name, tensors, longest, dtype, scale=1.0, max_norm=1.0):
    return {"name": name, "op": "clip", "tensors": tensors, "longest": longest, "dtype": dtype, "scale": scale,
            "max_norm": max_norm}


def _log_int(rng, low, high):
    """A whole number spread over the logarithm of [low, high]."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A row width: a multiple of 64 mostly, of 8 or an odd one sometimes."""
    w = _log_int(rng, low, high)
    step = rng.choice((64, 64, 64, 8, 1))
    return max(step, w // step * step) if step > 1 else w | 1


def draw(rng):
    kind = rng.choice(("route", "route", "exchange", "exchange", "exchange", "embed", "embed", "embed", "clip", "clip"))
    dtype = rng.choice(("float32", "bfloat16"))
    if kind == "route":
        groups = rng.choice((1, 1, 4, 8))
        experts = groups * _log_int(rng, max(2, 8 // groups), 512 // groups)
        kept = rng.randint(max(1, groups // 2), groups)
        top_k = min(rng.randint(1, 10), kept * (experts // groups))
        sigmoid = rng.random() < 0.5
        c = _route("", rng.choice(("forward", "backward")), _log_int(rng, 1, 16384), experts, top_k,
                   "sigmoid" if sigmoid else "softmax", dtype, sigmoid and rng.random() < 0.7, groups, kept,
                   rng.choice((1, 2)), top_k > 1 and rng.random() < 0.7, rng.choice((1.0, 2.5)), rng.choice((0.0, 0.05)))
    elif kind == "exchange":
        width, top_k = _width(rng, 256, 6144), rng.randint(1, 8)
        most = 8192 * 4096 * 9 // (width * (2 * top_k + 1) * (2 if dtype == "float32" else 1))
        c = _exchange("", rng.choice(("dispatch", "combine", "combine_grad")), _log_int(rng, 1, max(1, min(16384, most))),
                      width, _log_int(rng, 8, 512), top_k, dtype, rng.choice((0.0, 0.05)))
    elif kind == "embed":
        direction, width, vocabulary = rng.choice(("forward", "backward")), _width(rng, 256, 6144), _log_int(rng, 8000, 131072)
        parts = rng.choice((1, 1, 4, 8))
        rows = -(-vocabulary // parts)
        first = rows * rng.randrange(parts)
        rows = min(rows, vocabulary - first)
        table = rng.choice(("float32", dtype))
        rows = max(1, min(rows, (65536 * 4096 // width) // (2 if table == "float32" else 1)))
        c = _embed("", direction, _log_int(rng, 1, max(1, min(32768, 16384 * 4096 // width))), width, vocabulary, rows, first,
                   rng.choice((1.0, round(math.sqrt(width), 3))), dtype if direction == "backward" else table, table,
                   direction == "backward" and rng.random() < 0.5)
    else:
        tensors = _log_int(rng, 1, 180)
        c = _clip("", tensors, _log_int(rng, 100, 3000007), dtype, rng.choice((1.0, 0.125)), rng.choice((0.5, 1.0, 1e9)))
    del c["name"]
    return c


def _sizes(case):
    """Lengths of the clip's tensors: matrices of several sizes and short vectors, odd ones among them."""
    n, m = case["tensors"], case["longest"]
    return [max(1, (m, m // 4 + i, m // 97 + 1, m // 2 - i)[i % 4]) for i in range(n)]


def _starts(sizes):
    """Places of the tensors in one flat buffer, each on a 64-element boundary."""
    ends = np.cumsum([-(-s // 64) * 64 for s in sizes])
    return [0] + [int(e) for e in ends[:-1]], int(ends[-1])


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=_DEVICE)
    g.manual_seed(seed)
    return {"route": _prepare_route, "exchange": _prepare_exchange, "embed": _prepare_embed,
            "clip": _prepare_clip}[case["op"]](case, g)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=_DEVICE, dtype=torch.float32).to(dtype)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=_DEVICE)


def _empty(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device=_DEVICE)


def _prepare_route(case, g):
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    dtype = _DTYPES[case["dtype"]]
    # logits of a trained router: a spread of about two, and experts that are liked more than others
    logits = _randn(g, T, E) * 1.5 + _randn(g, E)
    # padding tokens: no expert may take them
    logits = logits.masked_fill((_rand(g, T) < case["empty"])[:, None], -math.inf).to(dtype)
    s = {"case": case, "logits": logits, "bias": _randn(g, E) * 0.1 if case["bias"] else None,
         "ids": _empty(torch.int32, T, k), "weights": _empty(torch.float32, T, k)}
    if case["direction"] == "backward":
        s["ids"], _ = _route_plain(s)
        s["grad_weights"] = _randn(g, T, k)
        s["grad_logits"] = _empty(dtype, T, E)
    return s


def _prepare_exchange(case, g):
    T, D, E, k = case["tokens"], case["width"], case["experts"], case["top_k"]
    dtype = _DTYPES[case["dtype"]]
    # k different experts for each token, some experts liked more than others
    ids = (_rand(g, T, E).log().neg().log().neg() + _randn(g, E)).topk(k, 1).indices.to(torch.int32)
    ids = ids.masked_fill((_rand(g, T) < case["empty"])[:, None], -1)
    s = {"case": case, "ids": ids, "offsets": _empty(torch.int32, E + 1), "places": _empty(torch.int32, T, k)}
    if case["direction"] == "dispatch":
        s["x"] = _randn(g, T, D, dtype=dtype)
        s["rows"] = _empty(dtype, T * k, D)
        return s
    s["places"] = _plan_plain(ids, E)[1]
    s["rows"] = _randn(g, T * k, D, dtype=dtype)
    s["weights"] = _rand(g, T, k) / k * 2
    s["y"] = _empty(dtype, T, D)
    if case["direction"] == "combine_grad":
        s["grad_y"] = _randn(g, T, D, dtype=dtype)
        s["grad_rows"] = _empty(dtype, T * k, D)
        s["grad_weights"] = _empty(torch.float32, T, k)
    return s


def _prepare_embed(case, g):
    T, D, R = case["tokens"], case["width"], case["rows"]
    table = _DTYPES[case["table_dtype"]]
    # token frequencies fall as one over their rank
    tokens = (torch.exp(_rand(g, T) * math.log(case["vocabulary"] + 1)) - 1).to(torch.int64).clamp_(0, case["vocabulary"] - 1)
    s = {"case": case, "tokens": tokens}
    if case["direction"] == "forward":
        s["table"] = _randn(g, R, D, dtype=table) * 0.02
        s["out"] = _empty(table, T, D)
    else:
        s["grad_out"] = _randn(g, T, D, dtype=_DTYPES[case["dtype"]]) * 0.01
        s["grad_table"] = _empty(table, R, D)
        s["before"] = _randn(g, R, D, dtype=table) * 0.01 if case["accumulate"] else None
    return s


def _prepare_clip(case, g):
    dtype, sizes = _DTYPES[case["dtype"]], _sizes(case)
    starts, total = _starts(sizes)
    flat = torch.zeros(total, dtype=dtype, device=_DEVICE)
    return {"case": case, "grads": [_randn(g, n, dtype=dtype) * 0.02 for n in sizes], "flat": flat,
            "outs": [flat[a:a + n] for a, n in zip(starts, sizes)], "norm": _empty(torch.float32, 1)}


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "route":
        return _route_grad_plain(state) if case["direction"] == "backward" else _route_plain(state)
    if case["op"] == "exchange":
        return {"dispatch": _dispatch_plain, "combine": _combine_plain, "combine_grad": _combine_grad_plain}[case["direction"]](state)
    if case["op"] == "embed":
        return _embed_grad_plain(state) if case["direction"] == "backward" else _embed_plain(state)
    return _clip_plain(state)


def _run_own(s, case):
    from collective_datapath_reduce_gb300 import torch_api as purlin

    if not _handles:
        _handles.append(purlin.initialize(8))
    h = _handles[0]
    if case["op"] == "route":
        scores = purlin.Scores.SIGMOID if case["scores"] == "sigmoid" else purlin.Scores.SOFTMAX
        if case["direction"] == "backward":
            purlin.route_experts_grad(s["logits"], s["ids"], s["grad_weights"], s["grad_logits"], h, scores=scores,
                                      renormalise=case["renormalise"], scale=case["scale"])
            return s["grad_logits"]
        purlin.route_experts(s["logits"], s["ids"], s["weights"], h, bias=s["bias"], scores=scores, groups=case["groups"],
                             kept_groups=case["kept_groups"], group_best=case["group_best"],
                             renormalise=case["renormalise"], scale=case["scale"])
        return s["ids"], s["weights"]
    if case["op"] == "exchange":
        if case["direction"] == "dispatch":
            purlin.expert_plan(s["ids"], s["offsets"], s["places"], h)
            purlin.dispatch_rows(s["x"], s["places"], s["rows"], h)
            return s["offsets"], s["places"], s["rows"]
        if case["direction"] == "combine":
            purlin.combine_rows(s["rows"], s["places"], s["weights"], s["y"], h)
            return s["y"]
        purlin.combine_rows_grad(s["rows"], s["places"], s["weights"], s["grad_y"], s["grad_rows"], s["grad_weights"], h)
        return s["grad_rows"], s["grad_weights"]
    if case["op"] == "embed":
        if case["direction"] == "forward":
            purlin.embed(s["table"], s["tokens"], s["out"], h, first=case["first"], scale=case["scale"])
            return s["out"]
        purlin.embed_grad(s["grad_out"], s["tokens"], s["grad_table"], h, first=case["first"], scale=case["scale"],
                          base=s["before"])
        return s["grad_table"]
    purlin.clip_grad_norm(s["grads"], s["outs"], case["max_norm"], s["norm"], h, scale=case["scale"])
    return s["flat"], s["norm"]


# ---------------------------------------------------------------- plain forms

def _scores_plain(x, scores):
    if scores == "sigmoid":
        return 1 / (1 + torch.exp(-x)), None
    best = x.max(1, keepdim=True).values
    e = torch.exp(x - torch.where(best == -math.inf, torch.zeros_like(best), best))
    return e / e.sum(1, keepdim=True), e


def _route_plain(s):
    case, x = s["case"], s["logits"].float()
    k, G = case["top_k"], case["groups"]
    score, e = _scores_plain(x, case["scores"])
    off = x == -math.inf
    # without a bias the logits are in the scores' order
    key = (score + s["bias"] if case["bias"] else x).masked_fill(off, -math.inf)
    if G > 1:
        if case["group_best"] == 2:
            two = (key if case["bias"] else score if e is None else e).masked_fill(off, -math.inf)
            two = two.view(-1, G, x.shape[1] // G).sort(2, descending=True).values[:, :, :2]
            of_group = two[:, :, 0] + two[:, :, 1:].masked_fill(two[:, :, 1:] == -math.inf, 0).sum(2)
        else:
            of_group = key.view(-1, G, x.shape[1] // G).max(2).values
        kept = of_group.sort(dim=1, descending=True, stable=True).indices[:, :case["kept_groups"]]
        keep = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, kept, True)
        key = key.masked_fill(~keep.repeat_interleave(x.shape[1] // G, 1), -math.inf)
    key, ids = (t[:, :k] for t in key.sort(dim=1, descending=True, stable=True))
    none = key == -math.inf
    w = score.gather(1, ids).masked_fill(none, 0)
    if case["renormalise"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return ids.masked_fill(none, -1).to(torch.int32), w * case["scale"]


def _route_grad_plain(s):
    case, x = s["case"], s["logits"].float()
    score, _ = _scores_plain(x, case["scores"])
    none = s["ids"] < 0
    at = s["ids"].clamp(min=0).long()
    w, dw = score.gather(1, at).masked_fill(none, 0), s["grad_weights"].masked_fill(none, 0) * case["scale"]
    if case["renormalise"]:
        total = w.sum(1, keepdim=True) + 1e-20
        dw = ((dw - (dw * w).sum(1, keepdim=True) / total) / total).masked_fill(none, 0)
    if case["scores"] == "sigmoid":
        picked = torch.zeros_like(x).scatter_add_(1, at, dw * w * (1 - w))
        return picked.to(s["logits"].dtype)
    dx = torch.zeros_like(x).scatter_add_(1, at, dw) - (dw * w).sum(1, keepdim=True)
    dx = (dx * score).masked_fill(none.all(1, keepdim=True), 0)
    return dx.to(s["logits"].dtype)


def _plan_plain(ids, experts):
    none = (ids < 0).flatten()
    key = ids.flatten().long().masked_fill(none, experts)
    order = key.sort(stable=True).indices
    places = torch.empty_like(order)
    places[order] = torch.arange(order.numel(), device=order.device)
    counts = (key[:, None] == torch.arange(experts, device=key.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return offsets.to(torch.int32), torch.where(none, ~places, places).view(ids.shape).to(torch.int32), order


def _dispatch_plain(s):
    offsets, places, order = _plan_plain(s["ids"], s["case"]["experts"])
    rows = s["x"][order // places.shape[1]]
    live = torch.arange(order.numel(), device=order.device) < offsets[-1]
    return offsets, places, rows * live[:, None]


def _combine_plain(s):
    none = s["places"] < 0
    rows = s["rows"][s["places"].clamp(min=0).long()].float()
    return (rows * s["weights"].masked_fill(none, 0)[:, :, None]).sum(1).to(s["rows"].dtype)


def _combine_grad_plain(s):
    none = s["places"] < 0
    at = torch.where(none, ~s["places"], s["places"]).long()
    dy = s["grad_y"].float()[:, None, :]
    dw = (s["rows"][at].float() * dy).sum(2).masked_fill(none, 0)
    rows = torch.empty_like(s["rows"])
    rows[at] = (dy * s["weights"].masked_fill(none, 0)[:, :, None]).to(rows.dtype)
    return rows, dw


def _embed_plain(s):
    at = s["tokens"] - s["case"]["first"]
    inside = (at >= 0) & (at < s["case"]["rows"])
    out = s["table"][at.clamp(0, s["case"]["rows"] - 1)].float() * s["case"]["scale"]
    return (out * inside[:, None]).to(s["table"].dtype)


def _embed_grad_plain(s):
    at = s["tokens"] - s["case"]["first"]
    inside = (at >= 0) & (at < s["case"]["rows"])
    # the sum of each row's tokens in 32 bits, sorted so that it is the same each time
    key, order = at.masked_fill(~inside, s["case"]["rows"]).sort(stable=True)
    total = torch.zeros((s["case"]["rows"] + 1, s["case"]["width"]), device=at.device)
    total.index_put_((key,), s["grad_out"][order].float(), accumulate=True)
    total = total[:-1] * s["case"]["scale"]
    if s["before"] is not None:
        total = total + s["before"].float()
    return total.to(s["grad_table"].dtype)


def _clip_plain(s):
    case = s["case"]
    squares = torch.stack([g.float().square().sum() for g in s["grads"]])
    norm = squares.sum().sqrt() * case["scale"]
    factor = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0) * case["scale"]
    [o.copy_(g.float() * factor) for o, g in zip(s["outs"], s["grads"])]
    return s["flat"], norm.view(1)


# ---------------------------------------------------------------- what a pass cannot do without

def _distinct(case):
    """How many rows of the range the tokens are expected to name, and how many tokens fall into it."""
    v = np.arange(case["first"], case["first"] + case["rows"], dtype=np.float64)
    p = np.log1p(1 / (v + 1)) / math.log(case["vocabulary"] + 1)
    return float((1 - np.exp(case["tokens"] * np.log1p(-p))).sum()), float(case["tokens"] * p.sum())


def work(case):
    es = 4 if case["dtype"] == "float32" else 2
    T = case.get("tokens", 0)
    if case["op"] == "route":
        E, k = case["experts"], case["top_k"]
        if case["direction"] == "backward":
            read = T * E if case["scores"] == "softmax" else T * k
            return {"bytes": es * (read + T * E) + 8 * T * k, "flops": 6 * read + 8 * T * k}
        return {"bytes": es * T * E + 4 * E * case["bias"] + 8 * T * k, "flops": 5 * T * E}
    if case["op"] == "exchange":
        D, k = case["width"], case["top_k"]
        if case["direction"] == "dispatch":
            return {"bytes": es * T * D * (k + 1) + 8 * T * k + 4 * (case["experts"] + 1), "flops": 0}
        if case["direction"] == "combine":
            return {"bytes": es * T * D * (k + 1) + 8 * T * k, "flops": 2 * T * k * D}
        return {"bytes": es * T * D * (2 * k + 1) + 12 * T * k, "flops": 3 * T * k * D}
    if case["op"] == "embed":
        D, ts = case["width"], 4 if case["table_dtype"] == "float32" else 2
        distinct, inside = _distinct(case)
        if case["direction"] == "forward":
            return {"bytes": ts * D * (distinct + T) + 8 * T, "flops": inside * D}
        table = 2 * case["rows"] if case["accumulate"] else case["rows"]
        return {"bytes": es * inside * D + ts * table * D + 8 * T, "flops": inside * D}
    n = sum(_sizes(case))
    return {"bytes": 2 * es * n + 4, "flops": 3 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        x = s["logits"].double()
        p = torch.sigmoid(x) if case["scores"] == "sigmoid" else torch.softmax(x, 1).nan_to_num(0.0)
        if case["direction"] == "backward":
            return _exact_route_grad(case, s, x)
        key = torch.where(torch.isinf(x), x, p + s["bias"].double()) if case["bias"] else x
        key = _exact_groups(case, key, p)
        order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :case["top_k"]]
        w = torch.take_along_dim(p, order, 1) * torch.isfinite(torch.take_along_dim(key, order, 1))
        w = w / (w.sum(1, keepdim=True) + 1e-20) if case["renormalise"] else w
        return None, w * case["scale"]
    if case["op"] == "exchange":
        T, k = case["tokens"], case["top_k"]
        if case["direction"] == "dispatch":
            none = s["ids"].flatten() < 0
            order = torch.argsort(torch.where(none, case["experts"], s["ids"].flatten()), stable=True)
            rows = torch.index_select(s["x"].double(), 0, torch.div(order, k, rounding_mode="floor"))
            rows[none[order]] = 0
            return None, None, rows
        live = (s["places"] >= 0).double()
        row = torch.where(s["places"] >= 0, s["places"], -1 - s["places"]).long().flatten()
        if case["direction"] == "combine":
            return torch.einsum("tkd,tk->td", s["rows"].double()[row].view(T, k, -1), live * s["weights"].double())
        dy = s["grad_y"].double()
        dw = torch.einsum("tkd,td->tk", s["rows"].double()[row].view(T, k, -1), dy) * live
        out = torch.empty(T * k, case["width"], dtype=torch.float64, device=dy.device)
        out[row] = torch.einsum("tk,td->tkd", live * s["weights"].double(), dy).reshape(T * k, -1)
        return out, dw
    if case["op"] == "embed":
        at = s["tokens"] - case["first"]
        live = torch.nonzero((at >= 0) & (at < case["rows"])).flatten()
        if case["direction"] == "forward":
            out = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device=at.device)
            out[live] = s["table"].double()[at[live]] * case["scale"]
            return out
        out = torch.zeros(case["rows"], case["width"], dtype=torch.float64, device=at.device)
        out.index_add_(0, at[live], s["grad_out"][live].double() * case["scale"])
        return out + s["before"].double() if case["accumulate"] else out
    starts, total = _starts(_sizes(case))
    norm = case["scale"] * math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in s["grads"]))
    flat = torch.zeros(total, dtype=torch.float64, device=_DEVICE)
    for a, g in zip(starts, s["grads"]):
        flat[a:a + g.numel()] = g.double() * (case["scale"] * min(1.0, case["max_norm"] / (norm + 1e-6)))
    return flat, torch.tensor([norm], dtype=torch.float64)


def _exact_groups(case, key, p):
    """-inf in place of the keys of the groups that are not kept."""
    T, E, G = key.shape[0], key.shape[1], case["groups"]
    if G == 1:
        return key
    by = key.reshape(T, G, E // G)
    if case["group_best"] == 1 or E // G == 1:
        best = by.amax(2)
    else:
        by = by if case["bias"] else torch.where(torch.isinf(by), by, p.reshape(T, G, E // G))
        first, second = by.topk(2, 2).values.unbind(2)
        best = first + torch.where(torch.isinf(second), 0.0, second)
    rank = torch.argsort(torch.argsort(best, dim=1, descending=True, stable=True), dim=1)
    return torch.where((rank < case["kept_groups"]).repeat_interleave(E // G, 1), key, -math.inf)


def _exact_route_grad(case, s, x):
    """The gradient by the Jacobian's rows: d s / d x of all scores, applied to d L / d s."""
    live = s["ids"] >= 0
    at = torch.where(live, s["ids"], 0).long()
    p = torch.sigmoid(x) if case["scores"] == "sigmoid" else torch.softmax(x, 1).nan_to_num(0.0)
    picked = torch.take_along_dim(p, at, 1) * live
    dw = s["grad_weights"].double() * live * case["scale"]
    if case["renormalise"]:
        total = picked.sum(1) + 1e-20
        dw = dw / total[:, None] - ((dw * picked).sum(1) / total**2)[:, None]
    ds = torch.zeros_like(p)
    ds.scatter_add_(1, at, dw * live)
    if case["scores"] == "sigmoid":
        return ds * p * (1 - p)
    return p * ds - p * (p * ds).sum(1, keepdim=True)
