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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,k,groups,top", [(8, 1, 1, 1), (24, 5, 8, 3), (60, 20, 6, 5), (160, 6, 8, 3), (700, 20, 7, 3),
                                            (1024, 64, 64, 33)])
def test_sigmoid_scores_far_below_one(E, k, groups, top, dtype):
    """Rows whose every score is next to nothing share as others do, down to where 64 bits hold no
    score (e^-745)."""
    import torch
    rng = np.random.default_rng(E)
    T = 90
    x = rng.standard_normal((T, E)) * rng.choice([0.5, 3.0, 20.0], (T, 1))
    x += np.resize([-18.0, -24.0, -60.0, -87.0, -88.5, -100.0, -150.0, -300.0, -500.0, 0.0], T)[:, None]
    x = np.maximum(x, -690.0)  # scores that 64 bits hold to the full
    x[5] = -60000.0            # and none
    x[6, 1:] = -60000.0
    x[7, ::2] = -INF
    x[8, 2:] = -800.0
    x = torch.from_numpy(x).to("cuda", dtype=getattr(torch, dtype))
    mask = torch.from_numpy(rng.random(T) < 0.9).cuda()
    mask[5:9] = True
    dw = values(rng.standard_normal((T, k)))
    # steps of 1/16, beside which a far score does not count: the lower index decides among equal ones
    steps = values(rng.integers(-8, 9, E) / 16.0)
    off = values(np.where(rng.random(E) < 0.3, -INF, 0.0))
    for bias in (None, off) if dtype != "float32" else (None, off, steps):
        for normalize, scale in ((True, 2.5), (False, 1.0)):
            if bias is steps:
                rows = (host(x) < -45).all(axis=1)
                y, m, d = x[torch.from_numpy(rows).cuda()], None, dw[torch.from_numpy(rows).cuda()]
            else:
                y, m, d = x, mask, dw
            say("far sigmoid", E, k, dtype, normalize, bias is None)
            r, want = check_far(y, k, dict(scores="sigmoid", bias=bias, groups=groups, top_groups=top, group_best=1,
                                           normalize=normalize, scale=scale), m, d)
            if normalize and k == 1:
                held = host(y).astype(np.float64)[np.arange(len(want["experts"])), want["experts"][:, 0]] > -745
                held &= want["experts"][:, 0] >= 0
                assert np.all(host(r.weights)[held] == scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,k,groups", [(8, 1, 4), (24, 5, 4), (60, 20, 6), (256, 8, 8), (700, 20, 7)])
def test_a_softmax_whose_top_is_not_chosen(E, k, groups, dtype):
    """With the row's top switched off, or its group left out, the others share what is left, however
    far below they are."""
    import torch
    rng = np.random.default_rng(E + 1)
    T = 60
    x = rng.standard_normal((T, E)) * rng.choice([1.0, 5.0], (T, 1))
    x[:, 1] = np.resize([18.0, 25.0, 90.0, 130.0, 400.0, 600.0, 2.0, 60000.0], T)
    x = torch.from_numpy(x).to("cuda", dtype=getattr(torch, dtype))
    dw = values(rng.standard_normal((T, k)))
    off = np.zeros(E)
    off[1] = -INF
    left_out = np.zeros(E)
    left_out[:E // groups] = -4.0
    for bias, top in ((off, groups), (left_out, groups - 1)):
        for normalize in (True, False):
            say("far softmax", E, k, dtype, normalize, top)
            r, want = check_far(x, k, dict(scores="softmax", bias=values(bias), groups=groups, top_groups=top, group_best=1,
                                           normalize=normalize, scale=1.5), None, dw)
            if normalize:
                sums = host(r.weights).astype(np.float64).sum(axis=1)
                far = np.resize([1, 1, 1, 1, 1, 1, 1, 0], T)  # beyond e^-745 there is no score
                assert np.all(np.abs(sums - 1.5 * far) <= 64 * H)


def test_gradients_of_far_scores_against_differences():
    """Through backward(), against differences of the 64-bit definition."""
    import torch
    rng = np.random.default_rng(8)
    T, E, k = 4, 12, 3
    base = np.stack([rng.permutation(E) for _ in range(T)]).astype(np.float32) * 0.25
    dw = values(rng.standard_normal((T, k)))
    d = host(dw).astype(np.float64)
    bias = np.zeros(E)
    bias[4] = -INF
    for scores, far in (("sigmoid", -100.0), ("sigmoid", -300.0), ("softmax", 150.0)):
        n = base.copy()
        if scores == "sigmoid":
            n += np.float32(far)
        else:
            n[:, 4] = far
        leaf = torch.from_numpy(n).cuda().requires_grad_()
        r = stf.route_tokens(leaf, k, scores=scores, bias=values(bias), balance=True, scale=2.0)
        ((r.weights * dw).sum() + 3.0 * r.loss).backward()
        how = dict(scores=scores, bias=bias, scale=2.0)

        def value(v):
            w = scored_ref(v, k, how)
            assert np.array_equal(w["experts"], host(r.experts))
            return float((w["weights"] * d).sum()) + 3.0 * w["loss"]

        n = n.astype(np.float64)
        say("differences", scores, far)
        for t in range(T):
            for e in range(E):
                up, down = n.copy(), n.copy()
                up[t, e] += 1e-5
                down[t, e] -= 1e-5
                slope = (value(up) - value(down)) / 2e-5
                assert abs(slope - float(leaf.grad[t, e])) <= 2 * TOL * (4 * np.abs(d).max() + 3.0 * E) + 1e-8


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(24, 5, 4), (60, 20, 6), (256, 8, 8)])
def test_far_rows_among_others_in_long_batches(E, k, groups, scores):
    """A group of lanes takes far and ordinary rows in turn: each is what it is in a batch of its own.
    Up to 64 experts a long batch has 8 lanes a row and a short one 16, so shares are summed in another
    order: each of the two sums is off by 22 h at most, as are the gradient's sums, and the products by
    4 h; from 65 experts on the bits are the same."""
    import torch
    rng = np.random.default_rng(E + 2)
    T, few = 70001, 257
    gen = torch.Generator(device="cuda")
    gen.manual_seed(E)
    x = torch.randn((T, E), generator=gen, device="cuda") * 2
    far = torch.rand(T, generator=gen, device="cuda") < 0.3
    if scores == "sigmoid":
        x[far] -= 120.0
    else:
        x[far, 1] = 150.0
    bias = np.zeros(E)
    bias[1] = -INF
    dw = torch.randn((T, k), generator=gen, device="cuda")
    how = dict(scores=scores, bias=values(bias), groups=groups, top_groups=groups - 1, group_best=1, scale=2.0)
    say("long far", scores, E, k)
    r = stf.route_tokens(x, k, **how)
    g = stf.route_tokens_grad(x, r, dw, scores=scores, scale=2.0)
    assert np.all(np.abs(r.weights.double().sum(dim=1).cpu().numpy() - 2.0) <= 64 * H)
    for s in (slice(0, few), slice(T // 2, T // 2 + few), slice(T - few, T)):
        q = stf.route_tokens(x[s], k, **how)
        h = stf.route_tokens_grad(x[s], q, dw[s], scores=scores, scale=2.0)
        assert torch.equal(q.experts, r.experts[s])
        if E > 64:
            assert torch.equal(q.weights, r.weights[s]) and torch.equal(h, g[s])
        else:
            assert bool(((q.weights - r.weights[s]).abs() <= 52 * H * q.weights).all())
            size = 2.0 * dw[s].abs().amax(dim=1, keepdim=True)
            assert bool(((h - g[s]).abs() <= 4 * 52 * H * size).all())
    at = torch.from_numpy(np.sort(rng.choice(T, 200, replace=False))).cuda()
    check_far(x[at], k, how, None, dw[at], 0.5)
