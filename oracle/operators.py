"""The operators around the collectives, stated plainly in 64 bits (numpy).

Values come in as float64 arrays and indices as integer arrays; every function
follows its definition one token, pick or row at a time.
"""

from __future__ import annotations

import math

import numpy as np


def scores_of(x, kind):
    """Expert scores of one token's logits."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        best = np.max(x) if np.max(x) > -np.inf or np.isnan(np.max(x)) else 0.0
        e = np.exp(x - best)
        return e / e.sum() if e.sum() != 0.0 else e


def _first_best(keys, count):
    """Numbers of the `count` best finite-or-+inf keys, best first, equal ones by number."""
    order = sorted((i for i in range(len(keys)) if keys[i] > -np.inf), key=lambda i: (-keys[i], i))
    return order[:count]


def group_score(keys, best):
    """A group's score from its experts' keys."""
    top = sorted((v for v in keys if v > -np.inf), reverse=True)
    return -np.inf if not top else sum(top[:best])


def route(logits, top_k, kind="softmax", bias=None, groups=1, kept_groups=1, group_best=1, renormalise=True, scale=1.0,
          margin=None):
    """(ids, weights) of every token.  `margin`: a list that receives the smallest
    gap between two different keys that a decision lay between."""
    T, E = logits.shape
    ids, weights = np.full((T, top_k), -1, dtype=np.int64), np.zeros((T, top_k))
    n = E // groups

    def note(values):
        v = np.sort(np.asarray([x for x in values if np.isfinite(x)]))
        gaps = np.diff(v)
        if margin is not None and (gaps > 0).any():
            margin.append(gaps[gaps > 0].min())

    for t in range(T):
        x = logits[t]
        s = scores_of(x, kind)
        key = x.copy() if bias is None else s + bias
        key[~(x > -np.inf)] = -np.inf
        key[np.isnan(key)] = -np.inf
        note(key)
        if groups > 1:
            of = s if bias is None and group_best == 2 else key
            if of is s and kind == "softmax":
                of = np.where(key == np.inf, key, np.where(np.max(key) == np.inf, 0.0, s))  # the limit, as s has none
            value = [group_score(np.where(key[g * n:(g + 1) * n] > -np.inf, of[g * n:(g + 1) * n], -np.inf), group_best)
                     for g in range(groups)]
            note(value)
            kept = _first_best(value, kept_groups)
            for g in range(groups):
                if g not in kept:
                    key[g * n:(g + 1) * n] = -np.inf
        picks = _first_best(key, top_k)
        w = s[picks]
        if renormalise:
            w = w / (w.sum() + 1e-20)
        ids[t, :len(picks)] = picks
        weights[t, :len(picks)] = w * scale
    return ids, weights


def weights_of(x, picks, kind, renormalise, scale):
    """The weights of fixed picks of one token (picks < 0 have weight 0)."""
    s = scores_of(x, kind)
    w = np.array([s[e] if e >= 0 else 0.0 for e in picks])
    if renormalise:
        w = w / (w.sum() + 1e-20)
    return w * scale


def route_grad(logits, ids, grad_weights, kind="softmax", renormalise=True, scale=1.0):
    """Gradient of the logits, through the Jacobian of weights by scores and of scores by logits."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        live = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if not live:
            continue
        s = scores_of(logits[t], kind)
        total = sum(s[ids[t, j]] for j in live) + 1e-20
        ds = np.zeros(E)
        for j in live:
            if renormalise:
                for i in live:
                    d = ((i == j) * total - s[ids[t, j]]) / total ** 2
                    ds[ids[t, i]] += scale * grad_weights[t, j] * d
            else:
                ds[ids[t, j]] += scale * grad_weights[t, j]
        if kind == "sigmoid":
            out[t] = ds * s * (1 - s)
        else:
            out[t] = s * (ds - np.dot(s, ds))
    return out


def plan(ids, experts):
    """(offsets, places) of picks sorted by expert, dropped picks last as ~row."""
    flat = np.asarray(ids).reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable")
    places = np.empty(flat.size, dtype=np.int64)
    places[order] = np.arange(flat.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=experts + 1)[:experts])])
    return offsets, np.where(key == experts, ~places, places).reshape(np.shape(ids))


def dispatch(x, places):
    T, k = places.shape
    rows = np.zeros((T * k, x.shape[1]), dtype=x.dtype)
    for t in range(T):
        for p in places[t]:
            if p >= 0:
                rows[p] = x[t]
    return rows


def combine(rows, places, weights=None):
    T, k = places.shape
    y = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if places[t, j] >= 0:
                y[t] += (1.0 if weights is None else weights[t, j]) * rows[places[t, j]]
    return y


def combine_grad(rows, places, weights, grad_y):
    T, k = places.shape
    grad_rows, grad_weights = np.zeros(rows.shape), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if places[t, j] >= 0:
                grad_rows[places[t, j]] = weights[t, j] * grad_y[t]
                grad_weights[t, j] = np.dot(rows[places[t, j]], grad_y[t])
    return grad_rows, grad_weights


def embed(table, tokens, first=0, scale=1.0):
    out = np.zeros((len(tokens), table.shape[1]))
    for i, v in enumerate(tokens):
        if first <= v < first + table.shape[0]:
            out[i] = scale * table[v - first]
    return out


def embed_grad(grad_out, tokens, rows, first=0, scale=1.0, base=None):
    total = np.zeros((rows, grad_out.shape[1]))
    for i, v in enumerate(tokens):
        if first <= v < first + rows:
            total[v - first] += grad_out[i]
    return scale * total + (0.0 if base is None else base)


def clip(grads, max_norm, scale=1.0):
    """(outputs, norm)."""
    norm = abs(scale) * math.sqrt(math.fsum(float(np.dot(g.ravel(), g.ravel())) for g in grads))
    factor = 1.0 if math.isinf(max_norm) else min(1.0, max_norm / (norm + 1e-6))
    return [g * (scale * factor) for g in grads], norm


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, stats) of rows x."""
    y, stats = np.zeros(x.shape), np.zeros((x.shape[0], 2))
    for t, row in enumerate(x):
        mean = math.fsum(row) / len(row)
        rstd = 1.0 / math.sqrt(math.fsum((row - mean) ** 2) / len(row) + eps)
        y[t] = (row - mean) * rstd * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
        stats[t] = mean, rstd
    return y, stats


def layer_norm_grad(grad_y, x, stats, weight=None, grad_total=None):
    """(grad_x, grad_weight, grad_bias), through each row's Jacobian."""
    grad_x, grad_weight, grad_bias = np.zeros(x.shape), np.zeros(x.shape[1]), np.zeros(x.shape[1])
    for t in range(x.shape[0]):
        hat = (x[t] - stats[t, 0]) * stats[t, 1]
        g = grad_y[t] * (1.0 if weight is None else weight)
        grad_x[t] = stats[t, 1] * (g - g.mean() - hat * (g * hat).mean())
        grad_weight += grad_y[t] * hat
        grad_bias += grad_y[t]
    return grad_x + (0.0 if grad_total is None else grad_total), grad_weight, grad_bias


def shares_of(x, kind):
    """A token's scores as shares of one."""
    s = scores_of(x, kind)
    return s / (s.sum() + 1e-20) if kind == "sigmoid" else s


def balance(logits, ids, kind="softmax", scale=1.0):
    """(counts, sums, loss)."""
    T, E = logits.shape
    counts, shares, tokens = np.zeros(E, dtype=np.int64), np.zeros(E), 0
    for t in range(T):
        live = [e for e in ids[t] if 0 <= e < E]
        if live:
            tokens += 1
            shares += shares_of(logits[t], kind)
            for e in live:
                counts[e] += 1
    sums = np.concatenate([counts, shares, [tokens]])
    return counts, sums, balance_of(sums, scale)


def balance_of(sums, scale=1.0):
    E = len(sums) // 2
    all_ = sums[:E].sum() * sums[2 * E]
    return scale * E * np.dot(sums[:E], sums[E:2 * E]) / all_ if all_ > 0 else 0.0


def balance_grad(logits, ids, sums, grad_loss=1.0, kind="softmax", scale=1.0):
    T, E = logits.shape
    out = np.zeros((T, E))
    all_ = sums[:E].sum() * sums[2 * E]
    for t in range(T):
        if all_ > 0 and any(0 <= e < E for e in ids[t]):
            c = grad_loss * scale * E * sums[:E] / all_
            s, p = scores_of(logits[t], kind), shares_of(logits[t], kind)
            jacobian = np.diag(p) - np.outer(p, p)          # of the shares by the scores' logarithms
            out[t] = (c @ jacobian) * ((1 - s) if kind == "sigmoid" else 1.0)
    return out


def teacher_of(ids, teacher, vocabulary, temperature):
    """q of one token's picks, 0 for those that are none."""
    t = np.where((ids >= 0) & (ids < vocabulary), teacher, -np.inf) / temperature
    return scores_of(t, "softmax") if np.isfinite(np.max(t)) or np.isnan(np.max(t)) else np.zeros(len(t))


def distil_parts(logits, ids, teacher, first=0, vocabulary=None, temperature=1.0):
    T, R = logits.shape
    vocabulary = first + R if vocabulary is None else vocabulary
    out = np.zeros((T, 4))
    for t in range(T):
        q = teacher_of(ids[t], teacher[t], vocabulary, temperature)
        m = np.max(logits[t]) if R else -np.inf
        ref = m if m > -np.inf else 0.0
        s = np.exp((logits[t] - ref) / temperature).sum()
        c = mass = 0.0
        for k, i in enumerate(ids[t]):
            if first <= i < first + R and q[k] > 0:
                c += q[k] * (math.log(q[k]) - (logits[t, i - first] - ref) / temperature)
                mass += q[k]
        out[t] = m, s, c, mass
    return out


def distil_join(parts, temperature=1.0, scale=1.0):
    """(loss, stats) from the parts of all ranges: ranges x tokens x 4."""
    T = parts.shape[1]
    loss, stats = np.zeros(T), np.zeros((T, 2))
    for t in range(T):
        M = parts[:, t, 0].max()
        ref = M if M > -np.inf else 0.0
        own = np.where(parts[:, t, 0] > -np.inf, parts[:, t, 0], 0.0)
        S = sum(p[1] * math.exp((o - ref) / temperature) for p, o in zip(parts[:, t], own) if p[1] != 0)
        mass = parts[:, t, 3].sum()
        stats[t] = M, S
        if S != 0 and mass != 0:
            loss[t] = scale * (sum(p[2] - p[3] * (o - ref) / temperature for p, o in zip(parts[:, t], own) if p[3] != 0)
                               + mass * math.log(S))
    return loss, stats


def distil_grad(logits, ids, teacher, stats, grad_loss, first=0, vocabulary=None, temperature=1.0, scale=1.0):
    T, R = logits.shape
    vocabulary = first + R if vocabulary is None else vocabulary
    out = np.zeros((T, R))
    for t in range(T):
        q = teacher_of(ids[t], teacher[t], vocabulary, temperature)
        if q.sum() == 0 or stats[t, 1] == 0:
            continue
        ref = stats[t, 0] if stats[t, 0] > -np.inf else 0.0
        out[t] = q.sum() * np.exp((logits[t] - ref) / temperature) / stats[t, 1]
        for k, i in enumerate(ids[t]):
            if first <= i < first + R:
                out[t, i - first] -= q[k]
        out[t] *= grad_loss[t] * scale / temperature
    return out
