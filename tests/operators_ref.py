"""64-bit definitions of the language-model operators, row by row in numpy (test oracles)."""
import numpy as np


def sample_row(l, u, t, k, p, m):
    """(token, logprob, margin): margin is the least distance, in units of the kept or the
    top-k mass, of a decision (the nucleus border, min-p, the draw) from its other side."""
    l = np.asarray(l, np.float64)
    if np.isnan(l).any():
        return -1, np.nan, np.inf
    live = np.flatnonzero(l > -np.inf)
    if live.size == 0:
        return -1, -np.inf, np.inf
    order = live[np.argsort(-l[live], kind="stable")]
    if not t > 0:
        return int(order[0]), 0.0, np.inf
    top = l[order[0]]
    if 0 < k < order.size:
        order = order[:k]
    with np.errstate(invalid="ignore"):
        d = np.where(l[order] == top, 0.0, (l[order] - top) / t)
    w = np.exp(d)
    c = np.cumsum(w)
    margin = np.inf
    n = order.size
    if p < 1:
        goal = p * c[-1]
        n = min(int(np.searchsorted(c, goal, side="left")) + 1, n)
        margin = np.min(np.abs(c - goal)) / c[-1]
    if m > 0:
        n = min(n, int(np.count_nonzero(w >= m)))
        near = np.abs(w - m)[w != m]
        if near.size:
            margin = min(margin, near.min() / m)
    n = max(n, 1)
    goal = min(max(u, 0.0), 1 - 2.0 ** -24) * c[n - 1] if u == u else 0.0
    j = min(int(np.searchsorted(c[:n], goal, side="right")), n - 1)
    margin = min(margin, np.min(np.abs(c[:n] - goal)) / c[n - 1])
    return int(order[j]), float(d[j] - np.log(c[n - 1])), margin


def softmax(x, mask=None):
    x = np.asarray(x, np.float64)
    live = (x > -np.inf).any(axis=1) | np.isnan(x).any(axis=1)
    if mask is not None:
        live &= mask
    p = np.zeros_like(x)
    for t in np.flatnonzero(live):
        e = np.exp(x[t] - x[t].max())
        p[t] = e / e.sum()
    return p, live


def balance(p, live, experts, k):
    """(loss, counts, rows, d loss / d logits)"""
    T, E = p.shape
    counts = np.zeros(E, np.int64)
    for t in np.flatnonzero(live):
        for e in experts[t]:
            if 0 <= e < E:
                counts[e] += 1
    n = int(live.sum())
    if n == 0:
        return 0.0, counts, 0, np.zeros_like(p)
    f = counts / (n * k)
    loss = E * float(f @ (p.sum(axis=0) / n))
    return loss, counts, n, E / n * p * (f[None, :] - (p @ f)[:, None])


def route(x, k, normalize, mask=None, d_weights=None, d_loss=0.0):
    """dict of weights, experts, counts, rows, loss, d_logits"""
    x = np.asarray(x, np.float64)
    p, live = softmax(x, mask)
    T, E = x.shape
    experts = np.full((T, k), -1, np.int64)
    weights = np.zeros((T, k))
    grad = np.zeros((T, E))
    for t in np.flatnonzero(live):
        order = np.argsort(-x[t], kind="stable")[:k]
        order = order[x[t][order] > -np.inf]
        j = order.size
        experts[t, :j] = order
        w = p[t][order]
        if normalize:
            w = w / w.sum()
        weights[t, :j] = w
        if d_weights is not None:
            d = np.asarray(d_weights[t, :j], np.float64)
            if normalize:
                grad[t][order] += w * (d - w @ d)
            else:
                g = np.zeros(E)
                g[order] = d
                grad[t] += p[t] * (g - p[t] @ g)
    loss, counts, n, lgrad = balance(p, live, experts, k)
    return dict(weights=weights, experts=experts, counts=counts, rows=n, loss=loss, d_logits=grad + d_loss * lgrad, p=p)


def scored(x, k, how, mask=None, d_weights=None, d_loss=0.0):
    """Routing by scores: dict as route's, with score, p, falling (of the score, for its own
    logit) and ok (rows whose choice no distance below 1e-14 decides, but for equal entries)."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    sigmoid, bias, groups = how["scores"] == "sigmoid", how.get("bias"), how.get("groups", 1)
    top, best, scale = how.get("top_groups") or groups, how.get("group_best", 2), how.get("scale", 1.0)
    normalize = how.get("normalize", True)
    p, live = softmax(x, mask)
    with np.errstate(over="ignore"):
        up, down = 1 / (1 + np.exp(-x)), 1 / (1 + np.exp(x))
    score = np.where(live[:, None], up, 0.0) if sigmoid else p
    falling = down if sigmoid else np.ones_like(x)
    if sigmoid:
        total = score.sum(axis=1, keepdims=True)
        p = np.divide(score, total, out=np.zeros_like(score), where=total != 0)
    experts, weights, grad = np.full((T, k), -1, np.int64), np.zeros((T, k)), np.zeros((T, E))
    ok = np.ones(T, bool)

    def rank(values):
        """Order by value, NaN first, then index; whether every step down is a clear one or none."""
        key = np.where(np.isnan(values), np.inf, values)
        order = np.argsort(-key, kind="stable")
        with np.errstate(invalid="ignore"):
            gaps = -np.diff(key[order])
            return order, ~((gaps > 0) & (gaps < 1e-14))

    for t in np.flatnonzero(live):
        c = score[t] + (bias if bias is not None else 0.0)
        c = np.where((x[t] == -np.inf) | (c == -np.inf), -np.inf, c)
        if top < groups:
            value = np.full(groups, -np.inf)
            for g in range(groups):
                m = c[g * (E // groups):(g + 1) * (E // groups)]
                m = m[rank(m)[0]][:best]
                m = m[~(m == -np.inf)]
                if m.size:
                    value[g] = m.sum()
            order, clear = rank(value)
            ok[t] &= clear[top - 1] or value[order[top]] == -np.inf
            for g in order[top:]:
                c[g * (E // groups):(g + 1) * (E // groups)] = -np.inf
        order, clear = rank(c)
        ok[t] &= bool(clear[:k].all())
        order = order[:k]
        order = order[~(c[order] == -np.inf)]
        experts[t, :order.size] = order
        w = score[t][order]
        if normalize:
            w = w / w.sum() if w.sum() != 0 else np.zeros_like(w)
        weights[t, :order.size] = scale * w
        if d_weights is not None:
            d = scale * np.asarray(d_weights[t, :order.size], np.float64)
            if normalize:
                grad[t][order] += w * (d - w @ d)
            elif sigmoid:
                grad[t][order] += w * d
            else:
                g = np.zeros(E)
                g[order] = d
                grad[t] += p[t] * (g - p[t] @ g)
    loss, counts, n, lgrad = balance(p, live, experts, k)
    return dict(weights=weights, experts=experts, counts=counts, rows=n, loss=loss, score=score, p=p, falling=falling,
                ok=ok, d_logits=(grad + d_loss * lgrad) * falling)
