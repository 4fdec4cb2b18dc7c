"""The row-wise operators of an expert-parallel training step, as cases to measure.

A layer norm stands behind a residual stream that an all-reduce or a combine
left, before the router; the balance loss looks at what the router picked, its
sums joined over ranks by an all-reduce; the distillation loss compares a
vocabulary's logits, or one rank's range of them, with a teacher's top logits,
the ranges' parts joined after an all-gather.

Every operator has a plain form here (elementary torch operations in 32 bits,
rounded once) and is called through the framework's torch front end where
`own` is true.
"""

import math

import torch

own = False

_DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}
_DEVICE = torch.device("cuda" if torch.cuda.is_available() else "cpu")
_EPS = 1e-5
_handles = []


def listed():
    return [
        # One token of a decoding request, added to its residual: latency only.
        _norm("norm, one token", "forward", 1, 4096, "bfloat16", "bfloat16", residual=True, stats=False),
        # A training micro-batch behind an all-reduce: sum with the residual, norm and statistics in one pass.
        _norm("norm, training", "forward", 16384, 5120, "bfloat16", "float32", residual=True),
        # 32-bit rows of an odd width, so that hardly any row starts on a vector's boundary.
        _norm("norm, ragged 32-bit", "forward", 3001, 1537, "float32", "float32", bias=False),
        # The gradient of a pre-norm layer: into the residual stream's gradient, and both parameters'.
        _norm("norm gradient, training", "backward", 8192, 4096, "bfloat16", "bfloat16", residual=True),
        # A narrow layer with many tokens: the columns' sums weigh as much as the rows.
        _norm("norm gradient, narrow", "backward", 20011, 520, "float32", "float32"),
        # A small micro-batch's counts and loss, with padding tokens that have no expert.
        _balance("balance, small batch", "forward", 300, 64, 6, "softmax", "float32", empty=0.05),
        # A large batch of a model with many experts: sigmoid scores.
        _balance("balance, large batch", "forward", 65536, 256, 8, "sigmoid", "float32"),
        # The router's gradient: added to the one that the picks' weights gave.
        _balance("balance gradient, training", "backward", 16383, 160, 6, "softmax", "bfloat16", base=True, empty=0.03),
        # Five tokens in front of a vocabulary: few rows, each of them long.
        _distil("distil, few tokens", "loss", 5, 32000, 32000, 0, 16, "bfloat16"),
        # A micro-batch of a training step, the whole vocabulary on one rank.
        _distil("distil, training", "loss", 4096, 131072, 131072, 0, 64, "bfloat16", temperature=2.0),
        # One rank's quarter of the vocabulary, the second: parts that the ranks join.
        _distil("distil, vocabulary range", "parts", 8191, 32768, 131072, 32768, 64, "bfloat16", empty=0.05),
        # The logits' gradient, of a vocabulary that is no multiple of a vector.
        _distil("distil gradient, ragged", "backward", 2047, 65537, 65537, 0, 32, "float32", temperature=2.0, empty=0.05),
    ]


def _norm(name, direction, tokens, width, dtype, weights, residual=False, bias=True, stats=True):
    return {"name": name, "op": "norm", "direction": direction, "tokens": tokens, "width": width, "dtype": dtype,
            "weights": weights, "residual": residual, "bias": bias, "stats": stats}


def _balance(name, direction, tokens, experts, top_k, scores, dtype, base=False, empty=0.0, scale=0.01):
    return {"name": name, "op": "balance", "direction": direction, "tokens": tokens, "experts": experts, "top_k": top_k,
            "scores": scores, "dtype": dtype, "base": base, "empty": empty, "scale": scale}


def _distil(name, direction, tokens, width, vocabulary, first, picks, dtype, temperature=1.0, empty=0.0):
    return {"name": name, "op": "distil", "direction": direction, "tokens": tokens, "width": width,
            "vocabulary": vocabulary, "first": first, "picks": picks, "dtype": dtype, "temperature": temperature,
            "empty": empty}


def _log_int(rng, low, high):
    """A whole number spread over the logarithm of [low, high]."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A row width: a multiple of 64 mostly, of 8 or an odd one sometimes."""
    w = _log_int(rng, low, high)
    step = rng.choice((64, 64, 64, 8, 1))
    return max(step, w // step * step) if step > 1 else w | 1


def draw(rng):
    kind = rng.choice(("norm", "norm", "balance", "distil", "distil"))
    dtype = rng.choice(("float32", "bfloat16"))
    es = 4 if dtype == "float32" else 2
    if kind == "norm":
        width = _width(rng, 64, 8192)
        c = _norm("", rng.choice(("forward", "backward")), _log_int(rng, 1, max(1, min(32768, 16384 * 5120 * 2 // (width * es)))),
                  width, dtype, rng.choice(("float32", dtype)), rng.random() < 0.5, rng.random() < 0.7, rng.random() < 0.8)
    elif kind == "balance":
        experts = _log_int(rng, 8, 512)
        c = _balance("", rng.choice(("forward", "backward")), _log_int(rng, 1, min(65536, 65536 * 256 // experts)), experts,
                     rng.randint(1, 8), rng.choice(("softmax", "sigmoid")), dtype, rng.random() < 0.5, rng.choice((0.0, 0.05)))
    else:
        parts = rng.choice((1, 1, 4, 8))
        vocabulary = _log_int(rng, 8000, 131072)
        vocabulary = vocabulary // 64 * 64 if rng.random() < 0.6 else vocabulary | 1
        width = -(-vocabulary // parts)
        first = width * rng.randrange(parts)
        width = min(width, vocabulary - first)
        direction = rng.choice(("loss", "backward")) if parts == 1 else rng.choice(("parts", "backward"))
        most = 4096 * 131072 // (width * (2 if direction == "backward" else 1) * (2 if dtype == "float32" else 1))
        c = _distil("", direction, _log_int(rng, 1, min(8192, most)), width, vocabulary, first, _log_int(rng, 1, 128), dtype,
                    rng.choice((1.0, 2.0, 0.75)), rng.choice((0.0, 0.05)))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=_DEVICE)
    g.manual_seed(seed)
    return {"norm": _prepare_norm, "balance": _prepare_balance, "distil": _prepare_distil}[case["op"]](case, g)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=_DEVICE, dtype=torch.float32).to(dtype)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=_DEVICE)


def _empty(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device=_DEVICE)


def _prepare_norm(case, g):
    T, D, dtype, weights = case["tokens"], case["width"], _DTYPES[case["dtype"]], _DTYPES[case["weights"]]
    # activations: channels of unequal size, a few of them large, and a mean that is not zero
    size = torch.exp(0.5 * _randn(g, D)) * torch.where(_rand(g, D) < 0.005, 20.0, 1.0)
    x = (_randn(g, T, D) * size + 0.2 * _randn(g, T, 1)).to(dtype)
    s = {"case": case, "x": x, "weight": (1 + 0.1 * _randn(g, D)).to(weights),
         "bias": (0.1 * _randn(g, D)).to(weights) if case["bias"] else None}
    if case["direction"] == "forward":
        s["residual"] = _randn(g, T, D, dtype=dtype) if case["residual"] else None
        s["y"], s["total"] = _empty(dtype, T, D), _empty(dtype, T, D) if case["residual"] else None
        s["stats"] = _empty(torch.float32, T, 2) if case["stats"] else None
        return s
    wide = x.double()
    mean = wide.mean(1, keepdim=True)
    rstd = ((wide - mean).square().mean(1, keepdim=True) + _EPS).rsqrt()
    s["stats"] = torch.cat([mean, rstd], 1).float()
    s["grad_y"] = _randn(g, T, D, dtype=dtype) * 0.01
    s["grad_total"] = _randn(g, T, D, dtype=dtype) * 0.01 if case["residual"] else None
    s["grad_x"], s["grad_weight"] = _empty(dtype, T, D), _empty(weights, D)
    s["grad_bias"] = _empty(weights, D) if case["bias"] else None
    return s


def _prepare_balance(case, g):
    T, E, k, dtype = case["tokens"], case["experts"], case["top_k"], _DTYPES[case["dtype"]]
    # logits of a trained router: a spread of about two, and experts that are liked more than others
    logits = _randn(g, T, E) * 1.5 + _randn(g, E)
    pad = _rand(g, T) < case["empty"]
    logits = logits.masked_fill(pad[:, None], -math.inf).to(dtype)
    ids = logits.float().topk(k, 1).indices.to(torch.int32).masked_fill(pad[:, None], -1).contiguous()
    s = {"case": case, "logits": logits, "ids": ids, "counts": _empty(torch.int32, E),
         "sums": _empty(torch.float32, 2 * E + 1), "loss": _empty(torch.float32, 1)}
    if case["direction"] == "backward":
        s["sums"] = _balance_plain(s)[1]
        s["grad_loss"] = 1 + 0.1 * _randn(g, 1)
        s["base"] = _randn(g, T, E, dtype=dtype) * 1e-6 if case["base"] else None
        s["grad_logits"] = _empty(dtype, T, E)
    return s


def _prepare_distil(case, g):
    T, R, V, K, dtype = case["tokens"], case["width"], case["vocabulary"], case["picks"], _DTYPES[case["dtype"]]
    # the teacher's best words, all different, its logits falling from the first to the last
    step = V // K
    ids = (torch.randint(V, (T, 1), generator=g, device=_DEVICE) + step * torch.arange(K, device=_DEVICE)
           + torch.randint(step, (T, K), generator=g, device=_DEVICE)) % V
    teacher = 12 - 2.5 * torch.log1p(torch.arange(K, device=_DEVICE).float()) + 0.5 * _randn(g, T, K)
    # the student thinks alike, roughly
    logits = _randn(g, T, R, dtype=dtype)
    logits *= 2
    token, pick = ((ids >= case["first"]) & (ids < case["first"] + R)).nonzero(as_tuple=True)
    logits[token, ids[token, pick] - case["first"]] = (teacher - 4 + _randn(g, T, K))[token, pick].to(dtype)
    # padding tokens have no teacher
    ids = ids.masked_fill((_rand(g, T) < case["empty"])[:, None], -1)
    s = {"case": case, "logits": logits, "ids": ids, "teacher": teacher}
    if case["direction"] == "loss":
        s["loss"], s["stats"] = _empty(torch.float32, T), _empty(torch.float32, T, 2)
    elif case["direction"] == "parts":
        s["parts"] = _empty(torch.float32, T, 4)
    else:
        best = logits.amax(1, keepdim=True).float()
        total = torch.exp((logits.float() - best) / case["temperature"]).sum(1, keepdim=True, dtype=torch.float64)
        # the other ranks' ranges weigh as much as this one, each
        s["stats"] = torch.cat([best, (total * (V / R)).float()], 1)
        s["grad_loss"] = (1 + 0.1 * _randn(g, T)) / T
        s["grad_logits"] = _empty(dtype, T, R)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "norm":
        return _norm_plain(state) if case["direction"] == "forward" else _norm_grad_plain(state)
    if case["op"] == "balance":
        return _balance_plain(state) if case["direction"] == "forward" else _balance_grad_plain(state)
    return {"loss": _distil_loss_plain, "parts": _distil_parts_plain, "backward": _distil_grad_plain}[case["direction"]](state)


def _run_own(s, case):
    from collective_datapath_reduce_gb300 import torch_api as purlin

    if not _handles:
        _handles.append(purlin.initialize(8))
    h = _handles[0]
    if case["op"] == "norm":
        if case["direction"] == "forward":
            purlin.layer_norm(s["x"], s["weight"], s["bias"], s["y"], h, residual=s["residual"], total=s["total"],
                              stats=s["stats"], eps=_EPS)
            return s["y"], s["total"], s["stats"]
        purlin.layer_norm_grad(s["grad_y"], s["x"], s["stats"], s["weight"], s["grad_x"], s["grad_weight"],
                               s["grad_bias"], h, grad_total=s["grad_total"])
        return s["grad_x"], s["grad_weight"], s["grad_bias"]
    if case["op"] == "balance":
        scores = purlin.Scores.SIGMOID if case["scores"] == "sigmoid" else purlin.Scores.SOFTMAX
        if case["direction"] == "forward":
            purlin.balance_loss(s["logits"], s["ids"], s["counts"], s["sums"], s["loss"], h, scores=scores,
                                scale=case["scale"])
            return s["counts"], s["sums"], s["loss"]
        purlin.balance_loss_grad(s["logits"], s["ids"], s["sums"], s["grad_loss"], s["grad_logits"], h, scores=scores,
                                 scale=case["scale"], base=s["base"])
        return s["grad_logits"]
    tau = case["temperature"]
    if case["direction"] == "loss":
        purlin.distil_loss(s["logits"], s["ids"], s["teacher"], s["loss"], s["stats"], h, temperature=tau, scale=tau * tau)
        return s["loss"], s["stats"]
    if case["direction"] == "parts":
        purlin.distil_parts(s["logits"], s["ids"], s["teacher"], s["parts"], h, first=case["first"],
                            vocabulary=case["vocabulary"], temperature=tau)
        return s["parts"]
    purlin.distil_loss_grad(s["logits"], s["ids"], s["teacher"], s["stats"], s["grad_loss"], s["grad_logits"], h,
                            first=case["first"], vocabulary=case["vocabulary"], temperature=tau, scale=tau * tau)
    return s["grad_logits"]


# ---------------------------------------------------------------- plain forms

def _norm_plain(s):
    x, total = s["x"], None
    if s["residual"] is not None:
        x = total = (x.float() + s["residual"].float()).to(x.dtype)
    off = x.float()
    mean = off.mean(1, keepdim=True)
    off = off - mean
    rstd = 1 / torch.sqrt((off * off).mean(1, keepdim=True) + _EPS)
    y = off * rstd * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(x.dtype), total, torch.cat([mean, rstd], 1) if s["case"]["stats"] else None


def _norm_grad_plain(s):
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    dy, hat = s["grad_y"].float(), (s["x"].float() - mean) * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    if s["grad_total"] is not None:
        dx = dx + s["grad_total"].float()
    to = s["weight"].dtype
    return dx.to(s["x"].dtype), (dy * hat).sum(0).to(to), dy.sum(0).to(to) if s["bias"] is not None else None


def _shares_plain(s):
    """Each token's scores as shares of one, and the scores themselves."""
    x = s["logits"].float()
    if s["case"]["scores"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
        return score / (score.sum(1, keepdim=True) + 1e-20), score
    best = x.amax(1, keepdim=True)
    e = torch.exp(x - best.masked_fill(best == -math.inf, 0))
    total = e.sum(1, keepdim=True)
    return e / total.masked_fill(total == 0, 1), None


def _balance_plain(s):
    E, k, scale = s["case"]["experts"], s["case"]["top_k"], s["case"]["scale"]
    picked = s["ids"].flatten()[:, None] == torch.arange(E, device=s["ids"].device, dtype=torch.int32)
    counts = picked.sum(0)
    counted = (s["ids"] >= 0).any(1)
    sums = (_shares_plain(s)[0] * counted[:, None]).sum(0)
    of_picks, of_scores = counts / counts.sum().clamp(min=1), sums / counted.sum().clamp(min=1)
    loss = scale * E * (of_picks * of_scores).sum()
    return counts.to(torch.int32), torch.cat([counts.float(), sums, counted.sum().view(1).float()]), loss.view(1)


def _balance_grad_plain(s):
    E = s["case"]["experts"]
    picks, tokens = s["sums"][:E], s["sums"][2 * E]
    c = s["grad_loss"] * s["case"]["scale"] * E * picks / (picks.sum() * tokens).clamp(min=1)
    share, score = _shares_plain(s)
    dx = share * (c - (share * c).sum(1, keepdim=True))
    if score is not None:
        dx = dx * (1 - score)
    dx = dx * (s["ids"] >= 0).any(1)[:, None]
    if s["base"] is not None:
        dx = dx + s["base"].float()
    return dx.to(s["logits"].dtype)


def _teacher_plain(s):
    """q and its logarithm, where in the range the picks stand, and which of them stand in it."""
    case = s["case"]
    live = (s["ids"] >= 0) & (s["ids"] < case["vocabulary"])
    t = s["teacher"].masked_fill(~live, -math.inf) / case["temperature"]
    best = t.amax(1, keepdim=True)
    t = t - best.masked_fill(best == -math.inf, 0)
    total = torch.exp(t).sum(1, keepdim=True)
    log_q = t - torch.log(total.masked_fill(total == 0, 1))
    at = s["ids"] - case["first"]
    return torch.exp(log_q), log_q, at.clamp(0, case["width"] - 1), live & (at >= 0) & (at < case["width"])


def _distil_parts_plain(s):
    tau, z = s["case"]["temperature"], s["logits"].float()
    best = z.amax(1, keepdim=True)
    total = torch.exp((z - best) / tau).sum(1, keepdim=True)
    q, log_q, at, inside = _teacher_plain(s)
    term = q * (log_q - (z.gather(1, at) - best) / tau)
    term = term.masked_fill(~(inside & (q > 0)), 0).sum(1, keepdim=True)
    return torch.cat([best, total, term, (q * inside).sum(1, keepdim=True)], 1)


def _distil_loss_plain(s):
    best, total, term, mass = _distil_parts_plain(s).unbind(1)
    tau = s["case"]["temperature"]
    return tau * tau * (term + mass * torch.log(total)), torch.stack([best, total], 1)


def _distil_grad_plain(s):
    tau = s["case"]["temperature"]
    q, _, at, inside = _teacher_plain(s)
    g = s["grad_loss"][:, None] * tau * tau / tau
    dz = torch.exp((s["logits"].float() - s["stats"][:, :1]) / tau) / s["stats"][:, 1:]
    dz *= q.sum(1, keepdim=True)
    dz.scatter_add_(1, at, -q * inside)
    return (dz * g).to(s["logits"].dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    es, T = 4 if case["dtype"] == "float32" else 2, case["tokens"]
    if case["op"] == "norm":
        D, ws, extra = case["width"], 4 if case["weights"] == "float32" else 2, case["residual"]
        vectors = ws * D * (2 if case["bias"] else 1)
        if case["direction"] == "forward":
            return {"bytes": es * T * D * (4 if extra else 2) + vectors + 8 * T * case["stats"], "flops": 8 * T * D}
        return {"bytes": es * T * D * (4 if extra else 3) + vectors + ws * D + 8 * T, "flops": 13 * T * D}
    if case["op"] == "balance":
        E, k = case["experts"], case["top_k"]
        if case["direction"] == "forward":
            return {"bytes": es * T * E + 4 * T * k + 4 * (3 * E + 2), "flops": 6 * T * E}
        return {"bytes": es * T * E * (3 if case["base"] else 2) + 4 * T * k + 4 * E, "flops": 10 * T * E}
    R, K = case["width"], case["picks"]
    picks = 12 * T * K
    if case["direction"] == "backward":
        return {"bytes": 2 * es * T * R + picks + 12 * T, "flops": 5 * T * R + 6 * T * K}
    return {"bytes": es * T * R + picks + (16 if case["direction"] == "parts" else 12) * T, "flops": 5 * T * R + 8 * T * K}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "balance": _exact_balance, "distil": _exact_distil}[case["op"]](case, s)


def _exact_norm(case, s):
    w = s["weight"].double()
    if case["direction"] == "forward":
        x, total = s["x"].double(), None
        if case["residual"]:
            total = x + s["residual"].double()
            x = total.to(s["x"].dtype).double()          # the norm is of what is stored
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        y = torch.addcmul(s["bias"].double() if case["bias"] else torch.zeros_like(w), (x - mean) / (var + _EPS) ** 0.5, w)
        return y, total, torch.hstack([mean, (var + _EPS) ** -0.5]) if case["stats"] else None
    mean, rstd = s["stats"].double().split(1, dim=1)
    dy, D = s["grad_y"].double(), case["width"]
    hat = torch.addcmul(-mean * rstd, s["x"].double(), rstd)
    # the Jacobian of a row is rstd (1 - (1 1' + hat hat') / D)
    g = dy * w
    dx = rstd * (g - (torch.einsum("td->t", g)[:, None] + hat * torch.einsum("td,td->t", g, hat)[:, None]) / D)
    if case["residual"]:
        dx = dx + s["grad_total"].double()
    return dx, torch.einsum("td,td->d", dy, hat), torch.einsum("td->d", dy) if case["bias"] else None


def _exact_shares(case, s):
    x = s["logits"].double()
    if case["scores"] == "sigmoid":
        p = torch.sigmoid(x)
        return p / (p.sum(1, keepdim=True) + 1e-20), p
    return torch.softmax(x, 1).nan_to_num(0.0), torch.zeros((), dtype=torch.float64, device=x.device)


def _exact_balance(case, s):
    E = case["experts"]
    live = (s["ids"] >= 0).any(1).double()
    if case["direction"] == "forward":
        counts = torch.bincount(s["ids"][s["ids"] >= 0].long(), minlength=E).double()
        scores = torch.mv(_exact_shares(case, s)[0].t(), live)
        loss = case["scale"] * E * torch.dot(counts, scores) / max(1.0, float(counts.sum() * live.sum()))
        return None, torch.cat([counts, scores, live.sum().view(1)]), loss.view(1)
    sums = s["sums"].double()
    c = sums[:E] * (float(s["grad_loss"]) * case["scale"] * E / max(1.0, float(sums[:E].sum() * sums[2 * E])))
    p, sigma = _exact_shares(case, s)
    dx = p * (1 - sigma) * (c - torch.mv(p, c)[:, None]) * live[:, None]
    return dx + s["base"].double() if case["base"] else dx


def _exact_distil(case, s):
    tau, V, R = case["temperature"], case["vocabulary"], case["width"]
    live = (s["ids"] >= 0) & (s["ids"] < V)
    q = torch.softmax(torch.where(live, s["teacher"].double(), -math.inf) / tau, 1).nan_to_num(0.0)
    at = s["ids"] - case["first"]
    q_here = q * (live & (at >= 0) & (at < R))
    at = at.clamp(0, R - 1)
    if case["direction"] == "backward":
        g = s["grad_loss"].double()[:, None] * tau
        # p = e^(z / tau) over the sum, the sum given by its largest term and the rest
        log_sum = s["stats"][:, :1].double() / tau + torch.log(s["stats"][:, 1:].double())
        dz = s["logits"].double().div_(tau).sub_(log_sum).exp_().mul_(q.sum(1, keepdim=True) * g)
        return dz.scatter_add_(1, at, -q_here * g)
    z = s["logits"].double()
    best = z.amax(1)
    log_sum = torch.logsumexp(z / tau, 1)
    entropy = torch.special.xlogy(q_here, q).sum(1)
    if case["direction"] == "loss":
        loss = entropy - (q_here * z.gather(1, at)).sum(1) / tau + q_here.sum(1) * log_sum
        return tau * tau * loss, torch.stack([best, torch.exp(log_sum - best / tau)], 1)
    here = entropy - (q_here * (z.gather(1, at) - best[:, None])).sum(1) / tau
    return torch.stack([best, torch.exp(log_sum - best / tau), here, q_here.sum(1)], 1)
