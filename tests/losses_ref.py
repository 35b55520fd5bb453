"""64-bit definitions of the losses over given tokens, row by row in numpy (test oracles).

Every function also gives how far 32-bit steps may take its results, worked out from h = 2^-24
(half a step of fp32).  With d the distance of an entry from its row's top over the temperature:
an exponential is off by 2 h for itself and 3 h d for d and its scaling; a sum of V of them adds
at most 32 + 14 roundings (a thread's four chains of 32, the lanes, the wavefronts).  So sums
are off by u = (64 + 4 reach) h of themselves, reach the largest finite d of the batch: the
distance of the token's own term counts in it too.  A log-probability is off by u times the
weight of the other entries, 1 - p <= min(1, |lp|) (doubled for a token below the top, whose own
term is in the sum), and by its rounding.
"""
import numpy as np

H = 2.0 ** -24


def rows(x, tokens, tau, mask=None):
    """dict: lp (0 where not live), live, p, others = 1 - p of the token, err of lp, u"""
    x = np.asarray(x, np.float64)
    T, V = x.shape
    live = (tokens >= 0) & (tokens < V)
    if mask is not None:
        live &= mask
    lp, others, err = np.zeros(T), np.zeros(T), np.zeros(T)
    p = np.zeros((T, V))
    finite = np.where(np.isfinite(x), x, np.nan)
    ok = np.isfinite(x).any(axis=1)
    reach = float(np.nanmax(np.nanmax(finite[ok], axis=1)[:, None] - finite[ok]) / tau) if ok.any() else 0.0
    u = (64 + 4 * min(reach, 1e3)) * H  # beyond 150 an exponential is 0
    for t in np.flatnonzero(live):
        a = int(tokens[t])
        r = x[t]
        if np.isnan(r).any() or (r == np.inf).any():
            lp[t] = others[t] = np.nan
            p[t] = np.nan
            continue
        if r[a] == -np.inf:
            lp[t] = -np.inf
            continue
        top = r.max()
        e = np.exp((r - top) / tau)
        p[t] = e / e.sum()
        rest = np.delete(e, a).sum()
        others[t] = rest / e.sum()
        lp[t] = -np.log1p(rest) if r[a] == top else (r[a] - top) / tau - np.log(e.sum())
        err[t] = 2 * u * min(1.0, abs(lp[t])) + 4 * H * abs(lp[t])
    return dict(lp=lp, live=live, p=p, others=others, err=err, u=u, tau=tau, tokens=tokens)


def grad(r, c, c_err=None):
    """(gradient, how far it may be off before its rounding) for coefficients c (rows of c 0 and
    absent tokens: 0)"""
    T, V = r["p"].shape
    g = np.zeros((T, V))
    off = np.zeros((T, V))
    for t in np.flatnonzero(r["live"]):
        if c[t] == 0 or r["lp"][t] == -np.inf:
            continue
        d = -r["p"][t].copy()
        d[int(r["tokens"][t])] = r["others"][t]
        g[t] = c[t] / r["tau"] * d
        off[t] = np.abs(g[t]) * (2 * r["u"] + 8 * H) + 2.0 ** -126 * abs(c[t]) / r["tau"]
        if c_err is not None:
            off[t] += np.abs(d) * c_err[t] / r["tau"]
    return g, off


def policy(r, old, adv, ref=None, weights=None, low=0.2, high=0.2, kl_weight=0.0, d_loss=1.0):
    """dict of loss, kl, clipped, rows, c and *_err; no ratio may be within its error of a border"""
    T = r["lp"].size
    n = int(r["live"].sum())
    out = dict(loss=0.0, kl=0.0, clipped=0, rows=n, c=np.zeros(T), c_err=np.zeros(T), loss_err=0.0, kl_err=0.0, near=np.inf)
    for t in np.flatnonzero(r["live"]):
        lp = r["lp"][t]
        if lp == -np.inf:
            continue
        w = float(weights[t]) if weights is not None else 1.0 / n
        e = r["err"][t] + 8 * H + 2 * H * abs(lp - old[t])
        ratio = np.exp(lp - old[t])
        cut = min(max(ratio, 1 - low), 1 + high)
        clipped = cut * adv[t] < ratio * adv[t]
        if adv[t]:
            out["near"] = min(out["near"], abs(ratio - (1 + high if adv[t] > 0 else 1 - low)) / (ratio * (e + 4 * H)))
        value = -adv[t] * (cut if clipped else ratio)
        slope = 0.0 if clipped else -adv[t] * ratio
        value_err = slope_err = abs(adv[t]) * (4 * H if clipped else ratio * e)
        if clipped:
            slope_err = 0.0
        if ref is not None:
            q = ref[t] - lp
            k = np.expm1(q) - q
            k_err = abs(np.expm1(q)) * e + 16 * H * (abs(np.expm1(q)) + abs(q) if abs(q) > 0.5 else k)
            out["kl"] += w * k
            out["kl_err"] += abs(w) * k_err
            value, slope = value + kl_weight * k, slope - kl_weight * np.expm1(q)
            value_err += kl_weight * k_err
            slope_err += kl_weight * np.exp(q) * e + 4 * H * kl_weight * abs(np.expm1(q))
        out["loss"] += w * value
        out["loss_err"] += abs(w) * value_err
        out["clipped"] += int(clipped)
        out["c"][t] = w * slope * d_loss
        out["c_err"][t] = abs(w * d_loss) * (slope_err + 4 * H * abs(slope))
    out["loss_err"] += 2 * H * abs(out["loss"])
    out["kl_err"] += 2 * H * abs(out["kl"])
    return out


def preference(r, offsets, pairs, ref=None, beta=0.1, smoothing=0.0, margin=0.0, average=False):
    T = r["lp"].size
    bounds = np.minimum(np.maximum.accumulate(np.maximum(np.asarray(offsets, np.int64), 0)), T)
    sums, ratio, share, err = np.zeros(2 * pairs), np.zeros(2 * pairs), np.ones(2 * pairs), np.zeros(2 * pairs)
    spans, n = [], 0
    for s in range(2 * pairs):
        span = [t for t in range(bounds[s], bounds[s + 1]) if r["live"][t]]
        spans.append(span)
        n += len(span)
        if average and span:
            share[s] = 1 / len(span)
        there = [t for t in span if r["lp"][t] != -np.inf]
        sums[s] = share[s] * sum(r["lp"][t] for t in there)
        ratio[s] = share[s] * sum(r["lp"][t] - (ref[t] if ref is not None else 0.0) for t in there)
        err[s] = share[s] * sum(r["err"][t] for t in there)
    z = beta * (ratio[:pairs] - ratio[pairs:]) - margin
    z_err = abs(beta) * (err[:pairs] + err[pairs:]) + 2 * H * np.abs(z)
    sig = 1 / (1 + np.exp(-z))
    loss = (1 - smoothing) * np.logaddexp(0, -z) + smoothing * np.logaddexp(0, z)
    slope = beta / pairs * (smoothing * sig - (1 - smoothing) / (1 + np.exp(z)))
    c, c_err = np.zeros(T), np.zeros(T)
    for s, span in enumerate(spans):
        i = s % pairs
        c[span] = (slope[i] if s < pairs else -slope[i]) * share[s]
        # the slope's slope is at most 1/4
        c_err[span] = (abs(beta) / pairs * 0.25 * z_err[i] + 2 * H * abs(slope[i])) * share[s]
    return dict(loss=loss.mean(), margins=z, sequence_logprobs=sums, rows=n, c=c, c_err=c_err, z_err=z_err,
                sums_err=err + 2 * H * np.abs(sums), loss_err=z_err.mean() + 2 * H * loss.mean())
