"""Routing by scores where the scores are far below 1, or no numbers at all.

Tolerances, in units of h = 2^-24.  Shares are of exponentials of distances from the largest of
those that share; a distance d is rounded by d h at most, and the shares with an exponential below
2^-126 count as 0, so d is below 88 where it counts.  With an exponential's 4 h, a sum of 1024's 22,
a division's and the scale's that is (64 + 8 + 4 * 88) h, for a share that is both above and below
the line; where no share is below 2^-96 of the largest, the rest is exact zeros.
"""
import numpy as np
import pytest

import sampling_threshold_filtering_amd as stf
from tests.operators_ref import scored as scored_ref
from tests.test_gpu_scored import TYPES, H, host, logits, say, values

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
TOL = (64 + 8 + 4 * 88) * H
NOTHING = 2.0 ** -95


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_switched_off_experts_of_rows_that_are_no_numbers(dtype, scores):
    """An expert of bias -inf is never chosen, whatever its row holds: NaN and +inf too."""
    import torch
    rng = np.random.default_rng(31)
    T, E, k = 90, 24, 5
    x = logits(rng, T, E, dtype)
    rows = torch.arange(T, device="cuda")
    at = torch.from_numpy(rng.integers(0, E, T)).cuda()
    x[rows[::3], at[::3]] = NAN
    x[rows[1::3], at[1::3]] = INF
    x[0], x[1] = NAN, INF
    off = [0, 1, 2, 5, 6, 7, 12, 13, 14, 15, 20]  # of groups of four, the fourth whole
    bias = values(rng.standard_normal(E) * 0.1)
    bias[off] = -INF
    on = np.setdiff1d(np.arange(E), off)
    b = host(bias).astype(np.float64)
    for groups, top, best in ((1, 1, 2), (6, 2, 2), (6, 2, 1), (6, 5, 2), (6, 6, 1)):
        say("switched off", dtype, scores, groups, top, best)
        r = stf.route_tokens(x, k, scores=scores, bias=bias, groups=groups, top_groups=top, group_best=best, balance=True)
        got = host(r.experts)
        assert not np.isin(got, off).any() and not r.counts[off].any()
        assert int(r.counts.sum()) == int((r.experts >= 0).sum()) and int(r.rows) == T
        n = host(x).astype(np.float64)
        for t in range(T):
            if scores == "softmax" and not (n[t] < INF).all():
                c = np.where(b > -INF, NAN, -INF)  # no score of such a row is a number
            elif scores == "softmax":
                c = np.exp(n[t] - n[t].max()) / np.exp(n[t] - n[t].max()).sum() + b
            else:
                c = np.where(b > -INF, 1 / (1 + np.exp(-n[t])) + b, -INF)
            key = np.where(np.isnan(c), INF, c)  # NaN first
            if top < groups:
                size = E // groups
                value = []
                for q in range(groups):
                    m = np.sort(key[q * size:(q + 1) * size])[::-1][:best]
                    m = m[m > -INF]
                    value.append(m.sum() if m.size else -INF)
                for q in np.argsort(-np.array(value), kind="stable")[top:]:
                    key[q * size:(q + 1) * size] = -INF
            order = np.argsort(-key, kind="stable")[:k]
            order = order[key[order] > -INF]
            assert got[t].tolist() == order.tolist() + [-1] * (k - order.size), t
            assert np.isin(order, on).all()


def check_far(x, k, how, mask=None, d_weights=None, d_loss=1.0):
    import torch
    r = stf.route_tokens(x, k, mask=mask, balance=True, **how)
    m = mask.cpu().numpy() if mask is not None else None
    dw = host(d_weights).astype(np.float64)
    exact = dict(how)
    if how.get("bias") is not None:
        exact["bias"] = host(how["bias"]).astype(np.float64)
    want = scored_ref(host(x), k, exact, m, dw, d_loss)
    scale, normalize = how.get("scale", 1.0), how.get("normalize", True)
    assert np.array_equal(host(r.experts), want["experts"])
    assert np.array_equal(host(r.counts), want["counts"]) and int(r.rows) == want["rows"]
    assert np.all(np.abs(host(r.weights) - want["weights"]) <= TOL * want["weights"] + NOTHING * scale)
    assert abs(float(r.loss) - want["loss"]) <= TOL * want["loss"] + NOTHING
    g = stf.route_tokens_grad(x, r, d_weights, d_loss, normalize=normalize, mask=mask, scores=how["scores"], scale=scale)
    eps = torch.finfo(g.dtype).eps / 2
    p = want["p"]
    w = np.zeros_like(p)
    for t in range(p.shape[0]):
        for j in range(k):
            if want["experts"][t, j] >= 0:
                w[t, want["experts"][t, j]] = want["weights"][t, j]
    big = np.abs(dw).max(axis=1)[:, None]
    size = 2 * big * np.maximum(w, scale * p if how["scores"] == "softmax" and not normalize else 0)
    f = want["counts"] / max(want["rows"] * k, 1)
    size = size + abs(d_loss) * p.shape[1] / max(want["rows"], 1) * p * (f[None, :] + (p @ f)[:, None])
    least = 2.0 ** -25 if g.dtype == torch.float16 else 1e-38
    off = 2 * TOL * size + NOTHING * scale * big
    bound = off + eps * (np.abs(want["d_logits"]) + off) + least
    assert np.all(np.abs(host(g) - want["d_logits"]) <= bound), np.abs(host(g) - want["d_logits"]).max()
    one = stf.route_tokens_grad(x, r, d_weights, None, normalize=normalize, mask=mask, scores=how["scores"], scale=scale)
    assert bool(torch.isfinite(one).all())
    return r, want
