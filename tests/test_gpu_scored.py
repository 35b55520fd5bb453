"""Routing by scores against its definition in 64 bits.

Tolerances, in units of h = 2^-24 (half a step of fp32).  A softmax's probability is off by (32 +
2 |d|) h of itself (test_gpu_route.py).  A sigmoid: the exponential of -|x| is off by 4 h, the sum
with 1, the reciprocal and the product by h each, its complement as much: 8 h of itself.  The sum of
up to 1024 of them adds 22 h, a division, the scale and the rounding h each.  Twice that covers a
weight over the chosen ones' sum.  Gradients are sums of products of such numbers: that, times the
sum of the absolute terms, plus half a step of their type.
"""
import numpy as np
import pytest

import sampling_threshold_filtering_amd as stf
from tests.operators_ref import scored as scored_ref

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
TYPES = ["float32", "float16", "bfloat16"]
# experts, k, groups, groups kept, best of a group
SHAPES = [(1, 1, 1, 1, 1), (2, 1, 2, 1, 1), (7, 3, 1, 1, 2), (8, 2, 4, 2, 2), (16, 16, 4, 4, 2), (24, 5, 8, 3, 2),
          (33, 4, 11, 2, 1), (60, 4, 6, 3, 2), (64, 6, 64, 9, 2), (64, 8, 8, 4, 1), (100, 10, 5, 2, 2), (130, 20, 2, 1, 2),
          (160, 6, 8, 3, 1), (256, 8, 8, 4, 2), (256, 9, 64, 7, 2), (260, 3, 13, 5, 2), (384, 8, 1, 1, 2),
          (500, 64, 10, 4, 2), (512, 8, 16, 5, 2), (700, 20, 7, 3, 2), (1024, 64, 64, 33, 2)]


def say(*a):
    print("[case]", *a, flush=True)


def host(t):
    return t.detach().float().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


def logits(rng, T, E, dtype, spread=1.5):
    import torch
    x = rng.standard_normal((T, E)) * spread + rng.standard_normal(E) * 0.7
    return torch.from_numpy(x).to("cuda", dtype=getattr(torch, dtype))


def values(v):
    import torch
    return torch.from_numpy(np.asarray(v, np.float32)).cuda()


def reach(x):
    a = host(x).astype(np.float64)
    a = np.where(np.isfinite(a), a, np.nan)
    a = a[np.isfinite(a).any(axis=1)]
    return float(np.nanmax(np.nanmax(a, axis=1)[:, None] - a)) if a.size else 0.0


def check(x, k, how, mask=None, d_weights=None, d_loss=None, rows_ok=None):
    """A call against the definition; (Routing, the definition's results)."""
    import torch
    r = stf.route_tokens(x, k, mask=mask, balance=True, **how)
    plain = stf.route_tokens(x, k, mask=mask, **how)
    assert plain.loss is None and torch.equal(plain.experts, r.experts) and torch.equal(plain.counts, r.counts)
    assert torch.equal(plain.weights, r.weights) and torch.equal(plain.rows, r.rows)
    m = mask.cpu().numpy() if mask is not None else None
    dw = host(d_weights).astype(np.float64) if d_weights is not None else None
    exact = dict(how)
    if how.get("bias") is not None:
        exact["bias"] = host(how["bias"]).astype(np.float64)
    exact["scale"] = float(np.float32(how.get("scale", 1.0)))
    want = scored_ref(host(x), k, exact, m, dw, float(np.float32(d_loss)) if d_loss is not None else 0.0)
    assert want["ok"].all()
    tol = (64 + (8 if how["scores"] == "sigmoid" else 4 * reach(x))) * H
    assert np.array_equal(host(r.experts), want["experts"])
    assert np.array_equal(host(r.counts), want["counts"]) and int(r.rows) == want["rows"]
    assert np.all(np.abs(host(r.weights) - want["weights"]) <= tol * np.abs(want["weights"]) + 2.0 ** -120)
    assert abs(float(r.loss) - want["loss"]) <= tol * want["loss"]
    if d_weights is None and d_loss is None:
        return r, want
    kw = dict(normalize=how.get("normalize", True), mask=mask, scores=how["scores"], scale=how.get("scale", 1.0))
    g = stf.route_tokens_grad(x, r, d_weights, d_loss, **kw)
    assert g.dtype == x.dtype and g.shape == x.shape
    eps = torch.finfo(g.dtype).eps / 2
    p = want["p"]
    size = np.zeros_like(p)  # the sum of the absolute terms
    if dw is not None and dw.size:
        big = np.abs(dw).max(axis=1, initial=0.0)[:, None] * exact["scale"]
        w = np.zeros_like(p)
        for t in range(p.shape[0]):
            for j in range(k):
                if want["experts"][t, j] >= 0:
                    w[t, want["experts"][t, j]] = want["weights"][t, j] / exact["scale"]
        size += 2 * big * np.maximum(w, p if how["scores"] == "softmax" else 0)
    if d_loss is not None and want["rows"]:
        f = want["counts"] / (want["rows"] * k)
        size += abs(d_loss) * p.shape[1] / want["rows"] * p * (f[None, :] + (p @ f)[:, None])
    size *= want["falling"]
    least = float(torch.finfo(g.dtype).tiny) * 2 * eps if g.dtype == torch.float16 else 1e-38
    bound = 2 * tol * size + eps * (np.abs(want["d_logits"]) + 2 * tol * size) + least
    assert np.all(np.abs(host(g) - want["d_logits"]) <= bound), np.abs(host(g) - want["d_logits"]).max()
    return r, want


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top,best", SHAPES)
def test_shapes(E, k, groups, top, best, scores, dtype):
    rng = np.random.default_rng(E * 100 + k)
    for T in (1, 2, 17, 70):
        say("scored", T, E, k, groups, top, best, scores, dtype)
        x = logits(rng, T, E, dtype)
        dw = values(rng.standard_normal((T, k)))
        for normalize, biased, scale in ((True, True, 2.5), (False, False, 1.0), (True, False, 1.0), (False, True, 16.0)):
            # without a bias equal logits tie exactly; with one every score is its own
            bias = values(rng.standard_normal(E) * 0.1) if biased else None
            check(x, k, dict(scores=scores, bias=bias, groups=groups, top_groups=top, group_best=best,
                             normalize=normalize, scale=scale), d_weights=dw, d_loss=0.7)


@pytest.mark.parametrize("T", [0, 777, 20011])
def test_token_counts(T):
    rng = np.random.default_rng(T)
    x = logits(rng, T, 24, "bfloat16")
    say("tokens", T)
    how = dict(scores="sigmoid", bias=values(rng.standard_normal(24) * 0.1), groups=4, top_groups=2, scale=2.0)
    r, _ = check(x, 3, how, d_weights=values(rng.standard_normal((T, 3))), d_loss=0.01)
    if T == 0:
        assert float(r.loss) == 0.0 and int(r.rows) == 0 and r.counts.sum().item() == 0


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_many_rows_choose_as_64_bits_do(scores):
    """Rows enough that some choices fall within 32-bit rounding, against torch in 64 bits."""
    import torch
    rng = np.random.default_rng(12)
    T, E, k, groups, top = 60000, 256, 8, 8, 4
    for dtype, step in (("float32", 0.05), ("bfloat16", 0.05), ("float32", 0.0)):
        x = logits(rng, T, E, dtype)
        bias = values(rng.standard_normal(E) * step)  # step 0: as training starts
        say("many rows", scores, dtype, step)
        r = stf.route_tokens(x, k, scores=scores, bias=bias, groups=groups, top_groups=top)
        xd = x.double()
        s = torch.sigmoid(xd) if scores == "sigmoid" else torch.softmax(xd, dim=1)
        c = s + bias.double()
        value = c.view(T, groups, -1).topk(2, dim=2)[0].sum(2)
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, value.sort(dim=1, descending=True, stable=True)[1][:, :top], True)
        c = c.masked_fill(~keep.repeat_interleave(E // groups, 1), float("-inf"))
        assert torch.equal(r.experts, c.sort(dim=1, descending=True, stable=True)[1][:, :k])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_expert(dtype, scores):
    import torch
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.integers(-2, 3, (300, 48)).astype(np.float64)).to("cuda", dtype=getattr(torch, dtype))
    x[:20] = 0.0
    x[20:40] = -0.0
    x[30:40, ::2] = 0.0
    dw = values(rng.standard_normal((300, 9)))
    # s(1) + s(-1) = 2 s(0) for a sigmoid: groups that tie in the mathematics, and which last bits of
    # 64 tell apart; so there the best alone
    best = 1 if scores == "sigmoid" else 2
    for bias in (None, values(np.zeros(48)), values(rng.integers(-1, 2, 48) * 0.5), values(np.full(48, 1e6))):
        for top in (1, 3, 6):
            check(x, 9, dict(scores=scores, bias=bias, groups=6, top_groups=top, group_best=best), d_weights=dw, d_loss=1.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_biases_of_every_size(dtype, scores):
    """The choice is that of 64 bits however far the biases reach."""
    rng = np.random.default_rng(16)
    x = logits(rng, 200, 60, dtype)
    for size in (1e-6, 1.0, 1e3, 1e8, 3e38):
        bias = rng.standard_normal(60)
        bias = values(bias / np.abs(bias).max() * size)
        say("biases", scores, dtype, size)
        check(x, 6, dict(scores=scores, bias=bias, groups=5, top_groups=2, normalize=False), d_loss=1.0)
    for odd in (float("inf"), float("nan"), float("-inf")):
        b = bias.clone() * 0
        b[[3, 17]] = odd
        r, _ = check(x, 6, dict(scores=scores, bias=b, groups=1))
        if odd == float("-inf"):
            assert not r.counts[[3, 17]].any()
        else:
            assert r.experts[:, :2].tolist() == [[3, 17]] * 200


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(12, 3), (60, 6), (200, 50)])
def test_masked_tokens_and_switched_off_experts(dtype, scores, E, groups):
    import torch
    rng = np.random.default_rng(7 + E)
    T, k, size = 203, 5, E // groups
    x = logits(rng, T, E, dtype)
    x[:, [1, E - 1]] = float("-inf")
    x[3] = float("-inf")                       # nothing left
    x[4] = float("-inf")
    x[4, 7] = 1.0                              # fewer than k left, and a group of one
    x[5, size:] = float("-inf")                # one group left
    x[6, 2:] = -30.0                           # all but two scores next to nothing
    mask = torch.from_numpy(rng.random(T) < 0.7).cuda()
    mask[[3, 4, 5, 6]] = True
    mask[[8, 9]] = False
    x[8] = float("nan")                        # masked places may hold anything
    x[9] = float("inf")
    dw = values(rng.standard_normal((T, k)))
    dw[8] = float("nan")
    clean, d0 = x.clone(), dw.clone()
    clean[8:10] = 0.0
    d0[8] = 0.0
    for normalize in (True, False):
        for bias in (None, values(rng.standard_normal(E) * 0.3)):
            say("masked", dtype, scores, E, normalize)
            how = dict(scores=scores, bias=bias, groups=groups, top_groups=2, normalize=normalize, scale=1.5)
            r = stf.route_tokens(x, k, mask=mask, balance=True, **how)
            g = stf.route_tokens_grad(x, r, dw, 0.3, normalize=normalize, mask=mask, scores=scores, scale=1.5)
            assert torch.isfinite(r.weights).all() and torch.isfinite(g).all() and torch.isfinite(r.loss)
            assert (g[8:10] == 0).all() and (g[3] == 0).all() and (r.experts[8] == -1).all()
            assert r.experts[4].tolist() == [7, -1, -1, -1, -1]
            if normalize:
                assert r.weights[4, 0].item() == 1.5
                only = stf.route_tokens_grad(x, r, dw, None, normalize=True, mask=mask, scores=scores, scale=1.5)
                assert not only[4].any()  # a row's only weight is 1, whatever its logit
            check(clean, k, how, mask, d0, 0.3)
    none = torch.zeros(T, dtype=torch.bool, device="cuda")
    r = stf.route_tokens(x, k, mask=none, balance=True, scores=scores, groups=groups, top_groups=1)
    assert float(r.loss) == 0.0 and int(r.rows) == 0 and (r.experts == -1).all() and (r.weights == 0).all()
    assert (stf.route_tokens_grad(x, r, dw, 0.3, mask=none, scores=scores) == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_lowest_values_and_infinities(dtype):
    import torch
    low = torch.finfo(getattr(torch, dtype)).min
    x = torch.zeros((4, 20), device="cuda").to(getattr(torch, dtype))
    x[0, 2:] = low
    x[1] = low
    x[2, 5] = float("inf")
    x[3, 11] = float("nan")
    for normalize in (True, False):
        r = stf.route_tokens(x, 4, normalize=normalize, scores="sigmoid")
        assert r.experts[:3, 0].tolist() == [0, 0, 5] and r.experts[3, 0].item() == 11
        assert torch.isfinite(r.weights[:3]).all() and torch.isnan(r.weights[3]).any()
        assert not r.weights[1].any()  # scores of 0 have no shares
        g = stf.route_tokens_grad(x, r, torch.ones((4, 4), device="cuda"), None, normalize=normalize, scores="sigmoid")
        assert torch.isfinite(g[:3]).all()
    r = stf.route_tokens(x[:2], 4, scores="softmax", scale=2.0)
    assert r.experts.tolist() == [[0, 1, 2, 3]] * 2 and r.weights[1].tolist() == [0.5] * 4
    r = stf.route_tokens(x[3:], 2, scores="softmax", scale=2.0, balance=True)
    assert torch.isnan(r.weights).all() and torch.isnan(r.loss)


def test_softmax_alone_is_the_plain_routing():
    """Without bias, groups and scale nothing changes; with all groups kept neither does the choice."""
    import torch
    rng = np.random.default_rng(4)
    for dtype in TYPES:
        x = logits(rng, 500, 60, dtype)
        a = stf.route_tokens(x, 4, balance=True)
        b = stf.route_tokens(x, 4, balance=True, scores="softmax", bias=None, groups=1, top_groups=1, scale=1.0)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        c = stf.route_tokens(x, 4, balance=True, groups=6, top_groups=6)
        assert torch.equal(a.experts, c.experts) and torch.equal(a.counts, c.counts)
        assert torch.allclose(a.weights, c.weights, rtol=64 * H, atol=0)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradients_against_differences(normalize, scores):
    """Through backward(), against differences of the 64-bit definition of the same choice."""
    import torch
    rng = np.random.default_rng(21)
    T, E, k = 6, 12, 3
    # entries 1/4 apart, so that no step changes the choice
    x = torch.from_numpy(np.stack([rng.permutation(E) for _ in range(T)]).astype(np.float32) * 0.25 - 1.5).cuda()
    dw = values(rng.standard_normal((T, k)))
    bias = values(rng.standard_normal(E) * 0.01)
    how = dict(scores=scores, bias=bias, groups=4, top_groups=2, normalize=normalize, scale=2.5)
    leaf = x.clone().requires_grad_()
    r = stf.route_tokens(leaf, k, balance=True, **how)
    ((r.weights * dw).sum() + 3.0 * r.loss).backward()
    exact = dict(how, bias=host(bias).astype(np.float64))
    d = host(dw).astype(np.float64)
    n = host(x).astype(np.float64)

    def value(v):
        w = scored_ref(v, k, exact)
        assert np.array_equal(w["experts"], host(r.experts))
        return float((w["weights"] * d).sum()) + 3.0 * w["loss"]

    step = 1e-5
    for t in range(T):
        for e in range(E):
            up, down = n.copy(), n.copy()
            up[t, e] += step
            down[t, e] -= step
            slope = (value(up) - value(down)) / (2 * step)
            # 64-bit differences are good to 1e-9; the kernel to (128 + 8 * 3) h of its absolute terms
            assert abs(slope - float(leaf.grad[t, e])) <= 152 * H * (2.5 * np.abs(d).max() * 2 + 3.0 * E) + 1e-8


def test_rows_strided_offset_and_broadcast():
    import torch
    rng = np.random.default_rng(14)
    for dtype in TYPES:
        wide = logits(rng, 40, 132, dtype)
        for x, groups in ((wide[:, 1:], 1), (wide[:, 4:68], 8), (wide[::3, 6:], 6), (wide.t()[:36].t(), 4),
                          (wide[:, ::2], 11), (wide[:1].expand(9, -1), 3), (wide[:, :1], 1)):
            say("strides", dtype, tuple(x.shape), x.stride())
            k = min(4, x.shape[1])
            dw = values(rng.standard_normal((x.shape[0], 2 * k)))[:, ::2]
            mask = torch.from_numpy(rng.random(2 * x.shape[0]) < 0.8).cuda()[::2]
            bias = values(rng.standard_normal(2 * x.shape[1]) * 0.1)[::2]
            check(x, k, dict(scores="sigmoid", bias=bias, groups=groups, top_groups=(groups + 1) // 2, scale=1.25), mask,
                  dw, 0.2)


def test_other_stream_and_graph():
    import torch
    rng = np.random.default_rng(41)
    x = logits(rng, 3000, 64, "bfloat16")
    dw, bias = values(rng.standard_normal((3000, 4))), values(rng.standard_normal(64) * 0.1)
    how = dict(scores="sigmoid", bias=bias, groups=8, top_groups=3, scale=2.0)

    def step():
        r = stf.route_tokens(x, 4, balance=True, **how)
        return tuple(r) + (stf.route_tokens_grad(x, r, dw, 0.1, scores="sigmoid", scale=2.0),)

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        x.copy_(logits(rng, 3000, 64, "bfloat16"))
        want = step()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_refusals():
    import torch
    x = torch.zeros((4, 12), device="cuda")
    bias = torch.zeros(12, device="cuda")
    for kw in (dict(scores="tanh"), dict(scores=None), dict(scores=1), dict(groups=5, top_groups=2), dict(groups=0),
               dict(groups=-3), dict(groups=4, top_groups=0), dict(groups=4, top_groups=5), dict(groups=1, top_groups=2),
               dict(groups=4, top_groups=2, group_best=3), dict(group_best=0), dict(groups=2.0, top_groups=1),
               dict(bias=bias[:5]), dict(bias=bias.double()), dict(bias=bias.cpu()), dict(bias=0.5),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(scale="a")):
        with pytest.raises(ValueError):
            stf.route_tokens(x, 2, **kw)
    with pytest.raises(stf.ProfkError) as err:
        stf.route_tokens(torch.zeros((4, 130), device="cuda"), 2, groups=65, top_groups=3)
    assert err.value.code == stf.PROFK_EUNSUPPORTED
    r = stf.route_tokens(x, 2, scores="sigmoid", balance=True)
    for kw in (dict(scores="tanh"), dict(scale=float("nan"))):
        with pytest.raises(ValueError):
            stf.route_tokens_grad(x, r, torch.zeros((4, 2), device="cuda"), None, **kw)
