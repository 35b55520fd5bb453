"""The token losses and routing by scores at the edges of what their inputs and outputs may be."""
import numpy as np
import pytest

import sampling_threshold_filtering_amd as stf
from tests import losses_ref as ref
from tests.test_gpu_scored import logits as router
from tests.test_gpu_token_losses import TYPES, H, batch, check_grad, check_logprobs, close, host, say, some_tokens, values

pytestmark = pytest.mark.gpu


def policy_inputs(T, V, dtype, seed=0, weighted=False):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = (torch.randn((T, V), generator=gen, device="cuda") * 2).to(getattr(torch, dtype))
    tokens = torch.randint(0, V, (T,), generator=gen, device="cuda")
    old = torch.full((T,), -float(np.log(V)), device="cuda") - torch.rand(T, generator=gen, device="cuda")
    adv = torch.randn(T, generator=gen, device="cuda")
    w = torch.rand(T, generator=gen, device="cuda") / T if weighted else None
    mask = torch.rand(T, generator=gen, device="cuda") < 0.8
    return x, tokens, old, adv, w, mask


def test_logits_beyond_32_bits_of_entries():
    """More than 2^32 entries, in and out: rows at both ends are those of a batch of their own."""
    import torch
    T, V, few = 33000, 131072, 600
    assert T * V > 1 << 32
    x = torch.empty((T, V), dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 3000):
        x[i:i + 3000].normal_()
    tokens = torch.randint(0, V, (T,), device="cuda")
    old, adv, w = (torch.randn(T, device="cuda") for _ in range(3))
    old -= 10
    say("beyond 32 bits", T, V)
    r, g = stf.policy_loss_and_grad(x, tokens, old, adv, weights=w)
    for s in (slice(0, few), slice(T - few, T)):
        q, h = stf.policy_loss_and_grad(x[s], tokens[s], old[s], adv[s], weights=w[s])
        assert torch.equal(r.logprobs[s], q.logprobs) and torch.equal(g[s], h)
    want = torch.log_softmax(x[-100:].double(), dim=1).gather(1, tokens[-100:, None])[:, 0]
    assert (r.logprobs[-100:].double() - want).abs().max() < 4e-6


def test_more_rows_than_one_grid_holds():
    """Rows of few entries take a wavefront each: 2^26 rows and more are several launches."""
    import torch
    T, V = (1 << 26) + 1000, 2
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn((T, V), generator=gen, device="cuda").bfloat16()
    tokens = torch.randint(0, 2, (T,), generator=gen, device="cuda")
    say("rows", T)
    lp = stf.token_logprobs(x, tokens)
    picked = x.gather(1, tokens[:, None])[:, 0].float()
    other = x.gather(1, 1 - tokens[:, None])[:, 0].float()
    want = -torch.nn.functional.softplus(other - picked)
    assert ((lp - want).abs() <= 64 * H * want.abs() + 1e-30).all()
    r = stf.policy_loss(x, tokens, want, torch.ones(T, device="cuda"))
    assert int(r.rows) == T and int(r.clipped) == 0
    assert abs(float(r.loss) + 1) < 1e-6  # every ratio is 1


@pytest.mark.parametrize("T,V", [(40, 40000), (700, 3000), (700, 60000)])
def test_other_streams_graphs_and_two_at_once(T, V):
    import torch
    x, tokens, old, adv, w, mask = policy_inputs(T, V, "bfloat16", T, True)
    d = torch.randn(T, device="cuda")
    offsets = torch.tensor([0, T // 4, T // 3, T // 2, T], device="cuda")
    scale = torch.tensor(3.0, device="cuda")

    def step():
        p, g = stf.policy_loss_and_grad(x, tokens, old, adv, ref_logprobs=old, kl_weight=0.1, mask=mask, d_loss=scale)
        q, h = stf.policy_loss_and_grad(x, tokens, old, adv, weights=w)
        f = stf.policy_loss(x, tokens, old, adv, mask=mask)
        z = stf.preference_loss(x, tokens, offsets, old, mask)
        return (*p, g, *q, h, *f, *z, stf.preference_loss_grad(x, tokens, z, scale, mask), stf.token_logprobs(x, tokens),
                stf.token_logprobs_grad(x, tokens, d, mask))

    def same(a, b):
        return all(torch.equal(p, q) for p, q in zip(a, b))

    want = step()
    assert same(step(), want)  # the same bits on every run
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:  # side by side
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(step())
    torch.cuda.synchronize()
    assert all(same(g, want) for g in got)
    del got
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.normal_()
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want), i
        del want


def test_two_graphs_side_by_side():
    """Each has scratch of its own; replayed in turn and together with eager calls."""
    import torch
    x, tokens, old, adv, w, mask = policy_inputs(600, 9000, "float32", 3)
    y, *_ = policy_inputs(600, 9000, "float32", 4)
    graphs, outs = [], []
    for v in (x, y):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(stf.policy_loss_and_grad(v, tokens, old, adv, mask=mask))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        eager = [stf.policy_loss_and_grad(v, tokens, old, adv, mask=mask) for v in (x, y)]
        torch.cuda.synchronize()
        for (p, g), (q, h) in zip(outs, eager):
            assert torch.equal(p.loss, q.loss) and torch.equal(g, h)
        del eager


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_offset_and_broadcast_inputs(dtype):
    import torch
    rng = np.random.default_rng(4)
    wide = batch(rng, 30, 1031, dtype)
    for x in (wide[:, 1:], wide[::3, 5:900], wide.t()[:600].t(), wide[:, ::2], wide[:1].expand(9, -1), wide[:, :1],
              wide.flip(0)[:, 3:]):
        T = x.shape[0]
        say("strides", dtype, tuple(x.shape), x.stride())
        tokens = torch.stack([some_tokens(rng, x)] * 2, dim=1)[:, 1]
        mask = torch.from_numpy(rng.random(2 * T) < 0.7).cuda()[::2]
        d = values(rng.standard_normal(3 * T))[::3]
        r = check_logprobs(x, tokens, 0.9, mask, d)
        old, adv = values(np.full(2 * T, -2.0))[::2], values(rng.standard_normal(2 * T))[1::2]
        got, _ = stf.policy_loss_and_grad(x, tokens, old, adv, weights=old, mask=mask, temperature=0.9)
        want = ref.policy(r, host(old), host(adv), None, host(old))
        if want["near"] > 2:
            close(host(got.loss), want["loss"], want["loss_err"], "loss")
        offsets = torch.tensor([0, 0, 1, 9, T // 3, 9, T // 2, 9, T, 9], device="cuda")[::2]
        got = stf.preference_loss(x, tokens, offsets, mask=mask, temperature=0.9)
        want = ref.preference(r, host(offsets), 2)
        close(host(got.margins), want["margins"], want["z_err"], "margins")


def test_settings_at_their_limits():
    import torch
    rng = np.random.default_rng(9)
    for dtype in TYPES:
        x = batch(rng, 7, 500, dtype)
        tokens = some_tokens(rng, x)
        for tau in (2.0 ** -20, 2.0 ** -8, 2.0 ** 20):
            say("temperature", tau, dtype)
            r = ref.rows(host(x), tokens.cpu().numpy(), tau)
            got = host(stf.token_logprobs(x, tokens, temperature=tau))
            # distances of up to 2^25 are rounded once, to 2^-24 of themselves; the outputs and each of the
            # 500 exponentials are fp32, whose least normal number is 2^-126 (by arithmetic: the oracle's
            # -2.6e-297 and -2.5e-238 lie under all that fp32 can hold)
            close(got, r["lp"], r["err"] + 2 * H * np.abs(r["lp"]) + 501 * 2.0 ** -126, "logprobs")
            g = stf.token_logprobs_grad(x, tokens, values(np.ones(7)), temperature=tau)
            # up to 1 / temperature: 2^20 is beyond fp16's greatest number, 65504, and rounds to infinity there
            want = -torch.softmax(x.double() / tau, dim=1)
            want.scatter_add_(1, tokens[:, None], torch.ones((7, 1), dtype=torch.float64, device="cuda"))
            assert bool((torch.isfinite(g) | ((want.abs() / tau > 60000) & (g * want > 0) & (dtype == "float16"))).all())
    x, tokens, old, adv, w, mask = policy_inputs(300, 700, "float32", 5)
    inf = float("inf")
    a = stf.policy_loss(x, tokens, old, adv, clip_low=inf, clip_high=inf)
    assert int(a.clipped) == 0
    b = stf.policy_loss(x, tokens, old, adv, clip_low=0, clip_high=0)  # any ratio but 1 is clipped on its side
    ratio = torch.exp(b.logprobs - old)
    assert int(b.clipped) == int((((ratio > 1) & (adv > 0)) | ((ratio < 1) & (adv < 0))).sum())
    for beta, smoothing, margin in ((0.0, 0.0, 0.0), (1e30, 1.0, 0.0), (-1.0, 0.5, 1e30), (1e4, 0.0, 0.0)):
        p = stf.preference_loss(x, tokens, torch.tensor([0, 100, 300], device="cuda"), beta=beta, smoothing=smoothing,
                                margin=margin)
        assert bool(torch.isfinite(p.coefficients).all()) and not bool(torch.isnan(p.loss))


def test_refusals():
    import torch
    x, tokens, old, adv, w, mask = policy_inputs(6, 50, "float32", 1, True)
    offsets = torch.tensor([0, 3, 6], device="cuda")
    for xx, tt, mm, tau in ((x.double(), tokens, None, 1.0), (x[0], tokens, None, 1.0), (x, tokens[:5], None, 1.0),
                            (x, tokens.int(), None, 1.0), (x, tokens.cpu(), None, 1.0), (x, None, None, 1.0),
                            (x, tokens, mask[:4], 1.0), (x, tokens, mask.float(), 1.0), (x, tokens, mask.cpu(), 1.0),
                            (x, tokens, None, 0.0), (x, tokens, None, -1.0), (x, tokens, None, float("nan")),
                            (x, tokens, None, 2.0 ** 21), (x, tokens, None, "1"), (x[:, :0], tokens, None, 1.0),
                            (x.cpu(), tokens, None, 1.0), (3, tokens, None, 1.0)):
        for call in (lambda: stf.token_logprobs(xx, tt, mm, tau), lambda: stf.token_logprobs_grad(xx, tt, old, mm, tau),
                     lambda: stf.policy_loss(xx, tt, old, adv, mask=mm, temperature=tau),
                     lambda: stf.preference_loss(xx, tt, offsets, mask=mm, temperature=tau)):
            with pytest.raises((ValueError, AttributeError)):
                call()
    for kw in (dict(old_logprobs=None), dict(old_logprobs=old[:4]), dict(old_logprobs=old.double()), dict(advantages=None),
               dict(advantages=adv.cpu()), dict(ref_logprobs=old[:2]), dict(weights=w.half()), dict(clip_low=-0.1),
               dict(clip_high=float("nan")), dict(kl_weight=-1.0), dict(kl_weight=0.1), dict(kl_weight=float("inf"), ref_logprobs=old)):
        with pytest.raises(ValueError):
            stf.policy_loss(x, tokens, **{**dict(old_logprobs=old, advantages=adv), **kw})
    for d in (torch.zeros(2, device="cuda"), torch.zeros(1), torch.zeros(1, device="cuda").double(), "x", None):
        with pytest.raises(ValueError):
            stf.policy_loss_and_grad(x, tokens, old, adv, d_loss=d)
    for kw in (dict(offsets=offsets[:2]), dict(offsets=offsets[:1]), dict(offsets=offsets.int()), dict(offsets=offsets.cpu()),
               dict(offsets=[0, 3, 6]), dict(offsets=torch.zeros((3, 1), dtype=torch.int64, device="cuda")), dict(beta=float("inf")),
               dict(smoothing=1.5), dict(margin=float("nan")), dict(average=torch.zeros(2)), dict(ref_logprobs=old[:3])):
        with pytest.raises(ValueError):
            stf.preference_loss(x, tokens, **{**dict(offsets=offsets), **kw})
    with pytest.raises(stf.ProfkError) as err:
        stf.token_logprobs(torch.zeros((1, (1 << 24) + 1), dtype=torch.float16, device="cuda"), tokens[:1])
    assert err.value.code == stf.PROFK_EUNSUPPORTED


def test_autograd():
    import torch
    x, tokens, old, adv, w, mask = policy_inputs(200, 300, "float32", 6, True)
    offsets = torch.tensor([0, 50, 100, 130, 200], device="cuda")
    leaf = x.clone().requires_grad_()
    lp = stf.token_logprobs(leaf, tokens, mask, 0.7)
    (lp * adv).sum().backward()
    assert torch.equal(leaf.grad, stf.token_logprobs_grad(x, tokens, adv, mask, 0.7))
    leaf.grad = None
    r = stf.policy_loss(leaf, tokens, old, adv, old, w, mask, kl_weight=0.2)
    assert r.loss.requires_grad and not any(t.requires_grad for t in r[1:])
    (1024.0 * r.loss).backward()
    want, g = stf.policy_loss_and_grad(x, tokens, old, adv, old, w, mask, kl_weight=0.2, d_loss=1024.0)
    assert torch.equal(leaf.grad, g)
    plain = stf.policy_loss(x, tokens, old, adv, old, w, mask, kl_weight=0.2)
    assert all(torch.equal(a.detach(), b) for a, b in zip(r, plain)) and not plain.loss.requires_grad
    leaf.grad = None
    p = stf.preference_loss(leaf, tokens, offsets, old, mask, beta=0.5)
    assert p.loss.requires_grad and not any(t.requires_grad for t in p[1:])
    (p.loss * 3).backward()
    q = stf.preference_loss(x, tokens, offsets, old, mask, beta=0.5)
    assert torch.equal(leaf.grad, stf.preference_loss_grad(x, tokens, q, torch.tensor(3.0, device="cuda"), mask))
    with torch.no_grad():
        assert not stf.policy_loss(leaf, tokens, old, adv).loss.requires_grad
    with torch.inference_mode():
        assert stf.token_logprobs(x, tokens).is_inference()
    # through a projection, in halves that add up: what a step by parts does
    head = torch.randn((16, 300), device="cuda", requires_grad=True)
    h = torch.randn((200, 16), device="cuda")
    stf.policy_loss(h @ head, tokens, old, adv, weights=w).loss.backward()
    whole = head.grad.clone()
    head.grad = None
    for s in (slice(0, 77), slice(77, 200)):
        stf.policy_loss(h[s] @ head, tokens[s], old[s], adv[s], weights=w[s]).loss.backward()
    assert torch.allclose(head.grad, whole, rtol=1e-4, atol=1e-6)


def test_forward_mode_tangents_are_refused():
    import torch
    import torch.autograd.forward_ad as forward
    x, tokens, old, adv, w, mask = policy_inputs(6, 50, "float32", 1)
    offsets = torch.tensor([0, 3, 6], device="cuda")
    with forward.dual_level():
        y = forward.make_dual(x, torch.ones_like(x))
        o = forward.make_dual(old, torch.ones_like(old))
        for call in (lambda: stf.token_logprobs(y, tokens), lambda: stf.token_logprobs_grad(x, tokens, o),
                     lambda: stf.policy_loss(y, tokens, old, adv), lambda: stf.policy_loss(x, tokens, o, adv),
                     lambda: stf.policy_loss(x, tokens, old, o), lambda: stf.preference_loss(y, tokens, offsets),
                     lambda: stf.preference_loss(x, tokens, offsets, o),
                     lambda: stf.route_tokens(y, 2, scores="sigmoid")):
            with pytest.raises(ValueError, match="tangent"):
                call()


def test_outputs_have_storages_of_their_own():
    import torch
    x, tokens, old, adv, w, mask = policy_inputs(600, 900, "float32", 1)
    p, g = stf.policy_loss_and_grad(x, tokens, old, adv)
    q = stf.preference_loss(x, tokens, torch.tensor([0, 100, 600], device="cuda"))
    out = [*p, g, *q, stf.token_logprobs(x, tokens), *stf.route_tokens(x, 4, scores="sigmoid", balance=True)]
    assert all(t.untyped_storage().nbytes() == t.numel() * t.element_size() and t.storage_offset() == 0 for t in out)
    assert len({t.untyped_storage().data_ptr() for t in out}) == len(out)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top", [(150001, 16, 4, 4, 2), (100001, 30, 9, 5, 3), (70001, 60, 20, 6, 5),
                                              (70003, 160, 6, 8, 3), (65537, 300, 40, 10, 4), (40001, 700, 64, 7, 3),
                                              (40003, 1024, 3, 64, 11)])
def test_several_rows_a_group(T, E, k, groups, top, scores):
    """Batches of which every group of lanes takes several rows: what one row left in registers and
    shared memory must not reach the next.  The formulas in 64 bits; tolerances as in
    test_gpu_scored."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(E + k)
    x = torch.randn((T, E), generator=gen, device="cuda") * 1.5 + torch.randn(E, generator=gen, device="cuda") * 0.7
    x[::7, 1::3] = float("-inf")
    x[5::1000, 1:] = float("-inf")
    x[6::1000] = float("-inf")
    mask = torch.rand(T, generator=gen, device="cuda") < 0.9
    bias = torch.randn(E, generator=gen, device="cuda") * 0.05
    dw = torch.randn((T, k), generator=gen, device="cuda")
    d_loss = 0.01 * T
    say("several rows", T, E, k, groups, top, scores)
    how = dict(scores=scores, bias=bias, groups=groups, top_groups=top, scale=1.5)
    r = stf.route_tokens(x, k, mask=mask, balance=True, **how)
    g = stf.route_tokens_grad(x, r, dw, d_loss, mask=mask, scores=scores, scale=1.5).double()
    xd = x.double()
    live = mask & (x > float("-inf")).any(dim=1)
    dead = ~live.unsqueeze(1)
    s = (torch.sigmoid(xd) if scores == "sigmoid" else torch.softmax(xd, dim=1)).masked_fill(dead, 0.0)
    c = (s + bias.double()).masked_fill(x == float("-inf"), float("-inf"))
    best = c.view(T, groups, -1).topk(2, dim=2)[0]
    value = best.masked_fill(best == float("-inf"), 0.0).sum(2).masked_fill(best[:, :, 0] == float("-inf"), float("-inf"))
    keep = torch.zeros_like(value, dtype=torch.bool)
    keep.scatter_(1, value.sort(dim=1, descending=True, stable=True)[1][:, :top], True)
    c = c.masked_fill(~keep.repeat_interleave(E // groups, 1), float("-inf"))
    val, at = c.sort(dim=1, descending=True, stable=True)
    at = at[:, :k]
    taken = (val[:, :k] > float("-inf")) & live.unsqueeze(1)
    assert torch.equal(r.experts, at.masked_fill(~taken, -1)) and int(r.rows) == int(live.sum())
    assert torch.equal(r.counts, torch.bincount(at[taken], minlength=E))
    w = s.gather(1, at) * taken
    w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    tol = (64 + 4 * 25) * H
    assert ((r.weights.double() - 1.5 * w).abs() <= tol * 1.5 * w).all()
    total = s.sum(dim=1, keepdim=True)
    p = s / torch.where(total > 0, total, 1.0)
    n = int(live.sum())
    f = r.counts.double() / (n * k)
    loss = float((E * f * p.sum(dim=0) / n).sum())
    assert abs(float(r.loss) - loss) <= (tol + 10 * H) * loss
    d = 1.5 * dw.double() * taken
    falling = torch.sigmoid(-xd) if scores == "sigmoid" else torch.ones_like(xd)
    pf = (p * f).sum(1, keepdim=True)
    want = torch.zeros_like(p).scatter_add_(1, at, w * (d - (w * d).sum(1, keepdim=True)))
    want = (want + d_loss * E / n * p * (f - pf)) * falling
    weight = torch.zeros_like(p).scatter_add_(1, at, w)
    size = (2 * d.abs().amax(1, keepdim=True) * weight + d_loss * E / n * p * (f + pf)) * falling
    assert ((g - want).abs() <= 2 * tol * size + H * (want.abs() + 2 * tol * size) + 1e-38).all()


@pytest.mark.parametrize("k", [1, 3, 20])
@pytest.mark.parametrize("E", [13, 60, 300])
def test_the_only_weight_of_a_row_has_no_gradient(E, k):
    import torch
    rng = np.random.default_rng(E)
    x = router(rng, 300, E, "float32")
    k = min(k, E)
    if k > 1:  # more slots, one expert that may be chosen
        at = torch.from_numpy(rng.integers(0, E, 300)).cuda()
        y = torch.full_like(x, float("-inf"))
        y[torch.arange(300, device="cuda"), at] = x[:, 0]
        x = y
    dw = values(rng.standard_normal((300, k)))
    r = stf.route_tokens(x, k, scores="sigmoid", scale=2.5)
    assert (r.weights[:, 0] == 2.5).all() and not r.weights[:, 1:].any()
    assert not stf.route_tokens_grad(x, r, dw, None, scores="sigmoid", scale=2.5).any()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [66, 130, 300, 1024])
@pytest.mark.parametrize("k", [1, 5, 63, 64])
def test_more_near_ties_than_lanes(E, k, scores):
    """Rows of one value, but for a few entries, behind the first 64, that are larger by a step of
    fp32: nearer than 32-bit scores tell, first in 64 bits."""
    import torch
    rng = np.random.default_rng(E + k)
    T = 500
    x = np.repeat(rng.standard_normal((T, 1)).astype(np.float32), E, axis=1)
    want = np.empty((T, k), dtype=np.int64)
    for t in range(T):
        up = np.sort(rng.choice(np.arange(64, E), size=min(t % 4, E - 64), replace=False))
        x[t, up] = np.nextafter(x[t, up], np.float32(np.inf))
        want[t] = np.concatenate([up, np.delete(np.arange(E), up)])[:k]
    say("more than lanes", E, k, scores)
    r = stf.route_tokens(torch.from_numpy(x).cuda(), k, scores=scores, bias=torch.zeros(E, device="cuda"))
    assert np.array_equal(host(r.experts), want)


@pytest.mark.parametrize("V,dtype,counts", [
    (4095, "float32", (512, 513)), (4097, "float32", (512, 513)), (8193, "bfloat16", (511, 513)),
    (16384, "float16", (255, 256, 257)), (16390, "float32", (64, 65, 127, 128)), (32769, "bfloat16", (64, 65, 129)),
    (32768, "bfloat16", (64, 65, 256)), (32768, "float32", (64, 65, 129)), (65535, "float16", (64, 65, 129, 513)),
    (65600, "float32", (64, 65, 512, 513)), (131072, "float16", (64, 65, 512, 513)), (131080, "bfloat16", (5, 512, 513))])
def test_few_rows_and_one_more(V, dtype, counts):
    """Around the numbers of rows and lengths up to which a row goes in slices: some rows of each
    against the formulas."""
    import torch
    rng = np.random.default_rng(V)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(V)
    T = max(counts)
    wide = (2 * torch.randn((T, V + 3), generator=gen, device="cuda")).to(getattr(torch, dtype))
    x = wide[:, 1:V + 1]
    at = np.unique(np.concatenate([[0, counts[0] - 1], rng.integers(0, counts[0], 4)]))
    tokens = torch.randint(0, V, (T,), generator=gen, device="cuda")
    tokens[at[0]] = x[at[0]].argmax()
    r = ref.rows(host(x[at.tolist()]), tokens.cpu().numpy()[at], 0.8)
    d = values(rng.standard_normal(T))
    old = torch.full((T,), 0.1 - float(np.log(V)) - 3.0, device="cuda")
    old[at.tolist()] = values(r["lp"] + 0.1)
    adv, w = values(rng.standard_normal(T)), values(rng.random(T))
    want = ref.policy(r, host(old)[at], host(adv)[at], None, host(w)[at], d_loss=64.0)
    assert want["near"] > 2
    for n in counts:
        say("rows and lengths", V, dtype, n)
        rows = at[at < n]
        assert rows.size == at.size
        y, t = x[:n], tokens[:n]
        err = r["err"] + H * np.abs(r["lp"])
        close(host(stf.token_logprobs(y, t, temperature=0.8))[at], r["lp"], err, "logprobs")
        check_grad(stf.token_logprobs_grad(y, t, d[:n], temperature=0.8)[at.tolist()], x[at.tolist()], r, host(d)[at])
        got, g = stf.policy_loss_and_grad(y, t, old[:n], adv[:n], weights=w[:n], temperature=0.8, d_loss=64.0)
        close(host(got.logprobs)[at], r["lp"], err, "policy's logprobs")
        check_grad(g[at.tolist()], x[at.tolist()], r, want["c"], want["c_err"])
        alone = stf.policy_loss(y, t, old[:n], adv[:n], weights=w[:n], temperature=0.8)
        close(host(alone.logprobs)[at], r["lp"], err, "logprobs without gradient")
        pref = stf.preference_loss(y, t, torch.tensor([0, n // 2, n], device="cuda"), temperature=0.8)
        close(host(pref.logprobs)[at], r["lp"], err, "preference's logprobs")
        # sums over all rows, of the rows' own values (rounded once: H of each)
        lp = got.logprobs.double()
        ratio = torch.exp(lp - old[:n].double())
        a, ww = adv[:n].double(), w[:n].double()
        terms = -ww * torch.minimum(ratio * a, ratio.clamp(0.8, 1.2) * a)
        off = (ww * ratio * a.abs() * (H * lp.abs() + 4 * H)).sum()
        for z in (got, alone):
            assert abs(float(z.loss) - float(terms.sum())) <= float(2 * off + 2 * H * terms.sum().abs())
        gap = float(pref.logprobs[:n // 2].double().sum() - pref.logprobs[n // 2:].double().sum())
        assert abs(float(pref.margins) - 0.1 * gap) <= 0.1 * float((lp.abs() * H).sum()) + 2 * H * abs(0.1 * gap)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_longest_rows(dtype):
    import torch
    V = 1 << 24
    x = torch.randn((3, V), device="cuda").to(getattr(torch, dtype))
    tokens = torch.tensor([V - 1, 0, V // 2], device="cuda")
    say("longest", dtype)
    lp = stf.token_logprobs(x, tokens)
    z = torch.logsumexp(x.double(), dim=1, keepdim=True)
    want = x.gather(1, tokens[:, None]).double() - z
    # 2^24 exponentials, each off by 4 h at most, of a sum that dominates: 8 h of it with the rest
    assert ((lp.double() - want[:, 0]).abs() <= 8 * H + H * want[:, 0].abs()).all()
    d = torch.full((3,), 65536.0, device="cuda")
    g = stf.token_logprobs_grad(x, tokens, d).double()
    formula = -65536.0 * torch.exp(x.double() - z)
    formula.scatter_add_(1, tokens[:, None], d.double()[:, None])
    assert ((g - formula).abs() <= (16 * H + torch.finfo(x.dtype).eps / 2) * formula.abs() + 1e-30).all()


def test_scratch_covers_every_number_of_rows():
    """More rows need more scratch, also where fewer go in slices."""
    L = stf.load_library()
    need = [L.profk_token_loss_scratch(t, 1 << 20) for t in (1, 511, 512, 513, 1024)]
    assert all(a < b for a, b in zip(need, need[1:]))


@pytest.mark.parametrize("size", [1e6, 3e7, 1e9, 1e10, 1.1e10, 7e11, 1e15, 1e20, 1e30, 3e38])
@pytest.mark.parametrize("T,V", [(9, 60), (5, 20000), (700, 17000)])
def test_rows_far_from_zero(T, V, size):
    """Rows whose largest entries are as large as fp32 holds, of either sign: all of one value (what
    a mask of -1e10 leaves), and with neighbouring values among them, whose distances are exact."""
    import torch
    rng = np.random.default_rng(V)
    say("far from zero", T, V, size)
    for sign in (1.0, -1.0):
        top = np.float32(sign * size)
        steps = [top]
        for _ in range(3):
            steps.append(np.nextafter(steps[-1], np.float32(-np.inf)))
        x = np.full((T, V), top, dtype=np.float32)
        x[1] = rng.choice(np.array(steps), size=V)
        x[2] = rng.choice(np.array(steps + [-np.inf, np.float32(-3.4e38), np.float32(min(top, -2e9))], dtype=np.float32), size=V)
        x[2, 5] = top
        x[3] = steps[1]
        x[3, 7] = top
        tokens = rng.integers(0, V, T)
        tokens[2:4] = (5, 7)
        for tau in (1.0, 0.3, 50.0):
            r = ref.rows(x, tokens, tau)
            y, t = torch.from_numpy(x).cuda(), torch.from_numpy(tokens).cuda()
            got = host(stf.token_logprobs(y, t, temperature=tau))
            # one entry of weight 2^-64 or less may count as none
            close(got, r["lp"], r["err"] + H * np.abs(r["lp"]) + V * 2.0 ** -64, "logprobs")
            c = rng.standard_normal(T)
            g = host(stf.token_logprobs_grad(y, t, values(c), temperature=tau))
            c = c.astype(np.float32).astype(np.float64)
            want, off = ref.grad(r, c)
            close(g, want, off + H * (np.abs(want) + off) + np.abs(c)[:, None] / tau * V * 2.0 ** -64, "d_logits")


@pytest.mark.parametrize("pairs,T,V", [(1023, 5000, 7), (1025, 3000, 7), (3000, 20000, 5), (5000, 600, 9000), (2500, 0, 5)])
def test_many_pairs(pairs, T, V):
    """More pairs than workgroups; offsets that rise and fall, below 0 and beyond T."""
    import torch
    rng = np.random.default_rng(pairs)
    say("many pairs", pairs, T, V)
    x = batch(rng, T, V, "float32")
    tokens = some_tokens(rng, x)
    mask = torch.from_numpy(rng.random(T) < 0.8).cuda()
    r = ref.rows(host(x), tokens.cpu().numpy(), 1.0, mask.cpu().numpy())
    rises = np.sort(rng.integers(-5, T + 6, 2 * pairs + 1))
    jumps = np.where(rng.random(2 * pairs + 1) < 0.2, rng.integers(-5, T // 2 + 1, 2 * pairs + 1), rises)
    for offsets in (rises, jumps):
        got = stf.preference_loss(x, tokens, torch.from_numpy(offsets).cuda(), mask=mask)
        want = ref.preference(r, offsets, pairs)
        close(host(got.margins), want["margins"], want["z_err"], "margins")
        close(host(got.loss), want["loss"], want["loss_err"], "loss")
        assert int(got.rows) == want["rows"]
        again = stf.preference_loss(x, tokens, torch.from_numpy(offsets).cuda(), mask=mask)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
