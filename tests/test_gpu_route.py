"""Routing and the balance loss against their definitions in 64 bits.

Tolerances, in units of h = 2^-24 (half a step of fp32).  A weight p = e / s: the
difference from the row's top is off by h |d|, the exponential by 4 h, the sum of up to
1024 terms in 16 steps per lane and 6 exchanges by 22 h beside its terms' errors, the
reciprocal and the product by h each: (32 + 2 |d|) h of p, and once more for a sum and a
division by it where the weights are normalised.  Gradients are sums of two products of
such numbers: that, times the sum of the absolute terms, plus half a step of their type.
"""
import numpy as np
import pytest

import sampling_threshold_filtering_amd as stf
from tests.operators_ref import balance as balance_ref
from tests.operators_ref import route as route_ref
from tests.operators_ref import softmax as softmax_ref

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
TYPES = ["float32", "float16", "bfloat16"]


def say(*a):
    print("[case]", *a, flush=True)


def host(t):
    return t.detach().float().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


def logits(rng, T, E, dtype, spread=1.5):
    import torch
    x = rng.standard_normal((T, E)) * spread + rng.standard_normal(E) * 0.7
    return torch.from_numpy(x).to("cuda", dtype=getattr(torch, dtype))


def reach(x):
    """The largest distance of a finite entry from its row's top."""
    a = host(x).astype(np.float64)
    a = np.where(np.isfinite(a), a, np.nan)
    a = a[np.isfinite(a).any(axis=1)]
    return float(np.nanmax(np.nanmax(a, axis=1)[:, None] - a)) if a.size else 0.0


def check_route(x, k, normalize, mask=None, d_weights=None, d_loss=None):
    import torch
    r = stf.route_tokens(x, k, normalize=normalize, mask=mask, balance=True)
    plain = stf.route_tokens(x, k, normalize=normalize, mask=mask)
    assert plain.loss is None and torch.equal(plain.experts, r.experts) and torch.equal(plain.counts, r.counts)
    assert torch.equal(plain.weights, r.weights) and torch.equal(plain.rows, r.rows)
    m = mask.cpu().numpy() if mask is not None else None
    dw = d_weights.cpu().numpy() if d_weights is not None else None
    want = route_ref(host(x), k, normalize, m, dw, float(np.float32(d_loss)) if d_loss is not None else 0.0)
    tol = (64 + 4 * reach(x)) * H
    assert np.array_equal(host(r.experts), want["experts"])
    assert np.array_equal(host(r.counts), want["counts"]) and int(r.rows) == want["rows"]
    assert np.all(np.abs(host(r.weights) - want["weights"]) <= tol * want["weights"])
    assert abs(float(r.loss) - want["loss"]) <= tol * want["loss"]
    if d_weights is None and d_loss is None:
        return r, None
    g = stf.route_tokens_grad(x, r, d_weights, d_loss, normalize=normalize, mask=mask)
    assert g.dtype == x.dtype and g.shape == x.shape
    check_grad(g, want, x, tol, dw, d_loss, k)
    return r, g


def check_grad(g, want, x, tol, dw, d_loss, k):
    import torch
    eps = torch.finfo(g.dtype).eps / 2
    p = want["p"]
    size = np.zeros_like(p)  # the sum of the absolute terms
    if dw is not None and dw.size:
        big = np.abs(dw).max(axis=1, initial=0.0)[:, None]
        w = np.zeros_like(p)
        for t in range(p.shape[0]):
            for j in range(k):
                if want["experts"][t, j] >= 0:
                    w[t, want["experts"][t, j]] = want["weights"][t, j]
        size += 2 * big * np.maximum(w, p)
    if d_loss is not None and want["rows"]:
        f = want["counts"] / (want["rows"] * k)
        size += abs(d_loss) * p.shape[1] / want["rows"] * p * (f[None, :] + (p @ f)[:, None])
    least = float(torch.finfo(g.dtype).tiny) * 2 * eps if g.dtype == torch.float16 else 1e-38
    bound = 2 * tol * size + eps * (np.abs(want["d_logits"]) + 2 * tol * size) + least
    assert np.all(np.abs(host(g) - want["d_logits"]) <= bound), np.abs(host(g) - want["d_logits"]).max()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 3), (8, 2), (16, 16), (17, 1), (33, 5), (60, 4), (64, 6), (65, 8),
                                 (100, 10), (128, 8), (160, 6), (256, 8), (257, 2), (300, 64), (512, 4), (1000, 9),
                                 (1024, 64)])
def test_shapes(E, k, dtype):
    import torch
    rng = np.random.default_rng(E * 100 + k)
    for T in (1, 2, 5, 17, 130):
        say("shapes", T, E, k, dtype)
        x = logits(rng, T, E, dtype)
        dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
        for normalize in (True, False):
            check_route(x, k, normalize, d_weights=dw, d_loss=0.7)


@pytest.mark.parametrize("T", [0, 777, 10007])
def test_token_counts(T):
    import torch
    rng = np.random.default_rng(T)
    x = logits(rng, T, 24, "bfloat16")
    dw = torch.from_numpy(rng.standard_normal((T, 3)).astype(np.float32)).cuda()
    say("tokens", T)
    r, _ = check_route(x, 3, True, d_weights=dw, d_loss=0.01)
    if T == 0:
        assert float(r.loss) == 0.0 and int(r.rows) == 0 and r.counts.sum().item() == 0


def test_many_tokens_sum_exactly_enough():
    """100,000 rows against a vectorised 64-bit sum of the same probabilities."""
    import torch
    rng = np.random.default_rng(2)
    x = logits(rng, 100000, 32, "float32")
    r = stf.route_tokens(x, 2, balance=True)
    p = torch.softmax(x.double(), dim=1)
    f = r.counts.double() / (100000 * 2)
    loss = float((32 * f * p.mean(dim=0)).sum())
    assert r.counts.sum().item() == 200000
    # besides the weights' own error: lane sums of at most 100000 / (512 blocks * 16 rows) + 1 = 14 terms, 2 exchanges
    assert abs(float(r.loss) - loss) <= (64 + 4 * reach(x) + 16) * H * loss
    again = stf.route_tokens(x, 2, balance=True)
    assert torch.equal(again.loss, r.loss)  # the same bits


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("normalize", [True, False])
def test_ties_go_to_the_lower_expert(dtype, normalize):
    import torch
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.integers(-2, 3, (300, 50)).astype(np.float64)).to("cuda", dtype=getattr(torch, dtype))
    x[:20] = 0.0
    x[20:40] = -0.0
    x[30:40, ::2] = 0.0
    dw = torch.from_numpy(rng.standard_normal((300, 9)).astype(np.float32)).cuda()
    check_route(x, 9, normalize, d_weights=dw, d_loss=1.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [12, 60, 200])
def test_masked_tokens_and_switched_off_experts(dtype, E):
    import torch
    rng = np.random.default_rng(7 + E)
    T, k = 203, 5
    x = logits(rng, T, E, dtype)
    x[:, [1, E - 1]] = float("-inf")
    x[3] = float("-inf")                       # nothing left
    x[4] = float("-inf")
    x[4, 7] = 1.0                              # fewer than k left
    x[5, :] = torch.finfo(x.dtype).min         # the type's lowest value is a value
    x[6, 2:] = torch.finfo(x.dtype).min
    mask = torch.from_numpy(rng.random(T) < 0.7).cuda()
    mask[[3, 4, 5, 6]] = True
    mask[[8, 9]] = False
    x[8] = float("nan")                        # masked places may hold anything
    x[9] = float("inf")
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    dw[8] = float("nan")
    xx = x.clone()
    for normalize in (True, False):
        say("masked", dtype, E, normalize)
        r = stf.route_tokens(x, k, normalize=normalize, mask=mask, balance=True)
        g = stf.route_tokens_grad(x, r, dw, 0.3, normalize=normalize, mask=mask)
        assert torch.isfinite(r.weights).all() and torch.isfinite(g).all() and torch.isfinite(r.loss)
        assert (g[8:10] == 0).all() and (g[3] == 0).all() and (r.experts[8] == -1).all()
        assert r.experts[4].tolist() == [7, -1, -1, -1, -1] and r.weights[4, 0].item() == 1.0
        xx[8:10] = 0.0
        d0 = dw.clone()
        d0[8] = 0.0
        # rows 5 and 6 reach as far as the type: their entries there are 0 or equal, whatever the distance
        rows = [t for t in range(T) if t not in (5, 6)]
        m2 = mask[rows].contiguous()
        check_route(xx[rows].contiguous(), k, normalize, m2, d0[rows].contiguous(), 0.3)
        assert r.experts[5].tolist() == list(range(k))  # all of row 5 was set, the switched-off columns too
        if normalize:
            assert torch.allclose(r.weights[5], torch.full((k,), 1.0 / k, device="cuda"), rtol=8 * H, atol=0)
        assert (r.weights[6, 1:] == 0).all()
    none = torch.zeros(T, dtype=torch.bool, device="cuda")
    r = stf.route_tokens(x, k, mask=none, balance=True)
    assert float(r.loss) == 0.0 and int(r.rows) == 0 and (r.experts == -1).all() and (r.weights == 0).all()
    assert (stf.route_tokens_grad(x, r, dw, 0.3, mask=none) == 0).all()


def test_nan_in_a_live_row_shows():
    import torch
    x = torch.zeros((3, 20), device="cuda")
    x[1, 11] = float("nan")
    r = stf.route_tokens(x, 2, balance=True)
    assert torch.isnan(r.weights[1]).all() and r.experts[1, 0].item() == 11 and torch.isnan(r.loss)
    assert torch.isfinite(r.weights[[0, 2]]).all()


def test_rows_strided_offset_and_broadcast():
    import torch
    rng = np.random.default_rng(14)
    for dtype in TYPES:
        wide = logits(rng, 40, 131, dtype)
        for x in (wide[:, 1:], wide[:, 3:67], wide[::3, 5:], wide.t()[:37].t(), wide[:, ::2], wide[:1].expand(9, -1),
                  wide[:, :1]):
            say("strides", dtype, tuple(x.shape), x.stride())
            k = min(4, x.shape[1])
            dw = torch.from_numpy(rng.standard_normal((x.shape[0], 2 * k)).astype(np.float32)).cuda()[:, ::2]
            mask = torch.from_numpy(rng.random(2 * x.shape[0]) < 0.8).cuda()[::2]
            check_route(x, k, False, mask, dw, 0.2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (500, 10, 1), (333, 64, 2), (200, 160, 6), (64, 700, 20),
                                   (0, 5, 2)])
def test_balance_loss_of_a_given_choice(T, E, k, dtype):
    import torch
    rng = np.random.default_rng(T + E)
    x = logits(rng, T, E, dtype)
    experts = rng.integers(-1, E + 1, (T, k))  # dropped slots on both sides of the range, repeats
    if T > 3:
        x[2] = float("-inf")
        experts[3, 0] = 1 << 40
    mask = torch.from_numpy(rng.random(T) < 0.8).cuda()
    say("balance", T, E, k, dtype)
    for m in (None, mask):
        b = stf.balance_loss(x, torch.from_numpy(experts).cuda(), mask=m)
        p, live = softmax_ref(host(x), None if m is None else m.cpu().numpy())
        loss, counts, rows, grad = balance_ref(p, live, experts, k)
        tol = (64 + 4 * reach(x)) * H
        assert np.array_equal(host(b.counts), counts) and int(b.rows) == rows
        assert abs(float(b.loss) - loss) <= tol * loss
        one = torch.tensor(2.0, device="cuda")
        g = stf.balance_loss_grad(x, b, one, mask=m)
        assert torch.equal(g, stf.balance_loss_grad(x, b, 2.0, mask=m))
        want = dict(p=p, counts=counts, rows=rows, d_logits=2.0 * grad)
        check_grad(g, want, x, tol, None, 2.0, k)


@pytest.mark.parametrize("normalize", [True, False])
def test_gradients_against_differences(normalize):
    """Central differences of the kernel's own forward pass, whose value is off by its
    tolerance and whose third derivative is at most 6 times the absolute terms."""
    import torch
    rng = np.random.default_rng(21)
    T, E, k, h = 6, 12, 3, 2.0 ** -6
    # entries 1/4 apart, so that no step changes the choice
    x = torch.from_numpy(np.stack([rng.permutation(E) for _ in range(T)]).astype(np.float32) * 0.25).cuda()
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    r = stf.route_tokens(x, k, normalize=normalize, balance=True)
    g = stf.route_tokens_grad(x, r, dw, 3.0, normalize=normalize)

    def value(y):
        q = stf.route_tokens(y, k, normalize=normalize)
        assert torch.equal(q.experts, r.experts)
        b = stf.balance_loss(y, r.experts)
        return float((q.weights.double() * dw.double()).sum()) + 3.0 * float(b.loss)

    size = float(dw.abs().sum()) + 3.0 * float(r.loss)
    for t in range(T):
        for e in range(E):
            up, dn = x.clone(), x.clone()
            up[t, e] += h
            dn[t, e] -= h
            diff = (value(up) - value(dn)) / float(up[t, e] - dn[t, e])
            assert abs(diff - float(g[t, e])) <= 6 * size * h * h / 6 + 96 * H * size / h


def test_autograd_and_accumulation():
    import torch
    rng = np.random.default_rng(31)
    x = logits(rng, 50, 20, "float32").requires_grad_()
    dw = torch.from_numpy(rng.standard_normal((50, 4)).astype(np.float32)).cuda()
    mask = torch.from_numpy(rng.random(50) < 0.8).cuda()
    r = stf.route_tokens(x, 4, mask=mask, balance=True)
    assert not r.experts.requires_grad and not r.counts.requires_grad
    ((r.weights * dw).sum() + 0.5 * r.loss).backward()
    want = stf.route_tokens_grad(x.detach(), r, dw, 0.5, mask=mask)
    assert torch.equal(x.grad, want)
    b = stf.balance_loss(x, r.experts, mask=mask)
    assert torch.equal(b.loss.detach(), r.loss.detach()) and torch.equal(b.counts, r.counts)
    b.loss.backward()
    assert torch.equal(x.grad, want + stf.balance_loss_grad(x.detach(), b, 1.0, mask=mask))
    x.grad = None
    r = stf.route_tokens(x, 4, mask=mask)       # no loss asked for
    (r.weights * dw).sum().backward()
    assert torch.equal(x.grad, stf.route_tokens_grad(x.detach(), r, dw, None, mask=mask))
    with torch.no_grad():
        assert not stf.route_tokens(x, 4).weights.requires_grad
    assert (stf.route_tokens_grad(x.detach(), r) == 0).all()


def test_other_stream_and_graph():
    import torch
    rng = np.random.default_rng(41)
    x = logits(rng, 3000, 64, "bfloat16")
    dw = torch.from_numpy(rng.standard_normal((3000, 4)).astype(np.float32)).cuda()

    def step():
        r = stf.route_tokens(x, 4, balance=True)
        return (r.weights, r.experts, r.counts, r.rows, r.loss, stf.route_tokens_grad(x, r, dw, 0.1))

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
    x = torch.zeros((4, 10), device="cuda")
    e = torch.zeros((4, 2), dtype=torch.int64, device="cuda")
    mask = torch.ones(4, dtype=torch.bool, device="cuda")
    for xx, k, m in ((x, 0, None), (x, 11, None), (x.double(), 2, None), (x[0], 2, None), (x, 2, mask[:3]),
                     (x, 2, mask.cpu()), (x, 2, mask.int()), (x.cpu(), 2, None)):
        with pytest.raises(ValueError):
            stf.route_tokens(xx, k, mask=m)
    with pytest.raises(stf.ProfkError) as err:
        stf.route_tokens(torch.zeros((4, 100), device="cuda"), 65)
    assert err.value.code == stf.PROFK_EUNSUPPORTED
    with pytest.raises(stf.ProfkError) as err:
        stf.route_tokens(torch.zeros((4, 1025), device="cuda"), 2)
    for ee in (e[:3], e.int(), e[:, 0], e.cpu(), e[:, :0]):
        with pytest.raises(ValueError):
            stf.balance_loss(x, ee)
    r = stf.route_tokens(x, 2, balance=True)
    for dw, dl in ((torch.zeros((4, 3), device="cuda"), None), (torch.zeros((4, 2)), None),
                   (torch.zeros((4, 2), dtype=torch.float64, device="cuda"), None),
                   (None, torch.zeros(2, device="cuda")), (None, torch.zeros(1))):
        with pytest.raises(ValueError):
            stf.route_tokens_grad(x, r, dw, dl)
