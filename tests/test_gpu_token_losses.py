"""Token log-probabilities, the policy loss and the preference loss against their definitions
in 64 bits; the tolerances are derived in losses_ref.py, with half a step of the gradient's type
for its one rounding (and half of the least step of fp16 where it is subnormal)."""
import numpy as np
import pytest

import sampling_threshold_filtering_amd as stf
from tests import losses_ref as ref

pytestmark = pytest.mark.gpu

H = ref.H
TYPES = ["float32", "float16", "bfloat16"]
# one entry, less than a vector, every size of team and its borders, segments of long rows
WIDTHS = [1, 2, 7, 9, 64, 1000, 2048, 2051, 8191, 8200, 16390, 32768, 32777, 65537, 131072]


def say(*a):
    print("[case]", *a, flush=True)


def host(t):
    return t.detach().double().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


def batch(rng, T, V, dtype, pad=0, offset=0, spread=2.0):
    """Logits with a few favoured entries per row, rows `pad` apart, the first `offset` entries
    from an aligned place."""
    import torch
    x = rng.standard_normal((T, V)) * spread
    for t in range(T):
        x[t, rng.integers(0, V, 4)] += 4 * spread
    store = torch.full((T * (V + pad) + offset + 8,), float("nan"), dtype=getattr(torch, dtype), device="cuda")
    view = store[offset:offset + T * (V + pad)].view(T, V + pad)[:, :V] if T else store[:0].view(0, V)
    view.copy_(torch.from_numpy(x))
    return view


def some_tokens(rng, x):
    """Mostly likely ones."""
    import torch
    T, V = x.shape
    a = host(x).argmax(axis=1) if T else np.zeros(0, np.int64)
    a = np.where(rng.random(T) < 0.4, rng.integers(0, V, T), a)
    return torch.from_numpy(a.astype(np.int64)).cuda()


def values(v):
    import torch
    return torch.from_numpy(np.asarray(v, np.float32)).cuda()


def close(got, want, off, what):
    got, want, off = np.asarray(got, np.float64), np.asarray(want, np.float64), np.asarray(off, np.float64)
    assert got.shape == want.shape, what
    same = (np.isnan(got) & np.isnan(want)) | (got == want)
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - want) <= off))
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4],
                           np.broadcast_to(off, got.shape)[bad][:4])


def check_grad(g, x, r, c, c_err=None):
    import torch
    assert g.dtype == x.dtype and g.shape == x.shape and g.is_contiguous()
    want, off = ref.grad(r, c, c_err)
    half = torch.finfo(x.dtype).eps / 2
    least = 2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -134 if x.dtype == torch.bfloat16 else 2.0 ** -150
    with np.errstate(invalid="ignore"):
        close(host(g), want, off + half * (np.abs(want) + off) + least, "d_logits")


def check_logprobs(x, tokens, tau=1.0, mask=None, d=None):
    m = mask.cpu().numpy() if mask is not None else None
    r = ref.rows(host(x), tokens.cpu().numpy(), tau, m)
    got = stf.token_logprobs(x, tokens, mask=mask, temperature=tau)
    close(host(got), r["lp"], r["err"] + H * np.abs(r["lp"]), "logprobs")
    if d is not None:
        check_grad(stf.token_logprobs_grad(x, tokens, d, mask=mask, temperature=tau), x, r, host(d))
    return r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", WIDTHS)
def test_logprobs_widths(V, dtype):
    rng = np.random.default_rng(V)
    for T, pad, offset, tau in ((5, 0, 0, 1.0), (3, 3, 1, 0.7)):
        say("logprobs", V, dtype, T, pad, offset)
        x = batch(rng, T, V, dtype, pad, offset)
        check_logprobs(x, some_tokens(rng, x), tau, d=values(rng.standard_normal(T)))


@pytest.mark.parametrize("dtype,V", [("float32", 200003), ("bfloat16", 400009), ("float16", 262144)])
def test_logprobs_long_rows(V, dtype):
    rng = np.random.default_rng(V)
    say("logprobs", V, dtype)
    x = batch(rng, 3, V, dtype, pad=1, offset=3)
    import torch
    # a token in each part of the row
    check_logprobs(x, torch.tensor([0, V // 2, V - 1], device="cuda"), 1.3, d=values([1.0, -2.0, 0.5]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(0, 100), (1, 100), (700, 33), (3001, 517), (300, 9000), (40, 33001)])
def test_policy(T, V, dtype):
    import torch
    rng = np.random.default_rng(T + V)
    x = batch(rng, T, V, dtype, pad=int(rng.integers(0, 5)))
    tokens = some_tokens(rng, x)
    for kl, weighted, masked, tau in ((0.05, False, False, 1.0), (0.0, True, True, 0.8)):
        say("policy", T, V, dtype, kl, weighted, masked)
        mask = torch.from_numpy(rng.random(T) < 0.7).cuda() if masked else None
        m = mask.cpu().numpy() if masked else None
        r = ref.rows(host(x), tokens.cpu().numpy(), tau, m)
        moved = 0.25 * rng.standard_normal(T)
        for border in (np.log(0.8), np.log(1.3)):
            moved = np.where(np.abs(moved - border) < 1e-3, moved + 3e-3, moved)
        old, adv = values(np.where(np.isfinite(r["lp"]), r["lp"], 0) - moved), values(rng.standard_normal(T))
        rf = values(r["lp"] + 0.3 * rng.standard_normal(T)) if kl else None
        w = values(rng.random(T) / max(T, 1)) if weighted else None
        d_loss = 8.0 * max(T, 1)  # keeps fp16 gradients normal
        kw = dict(ref_logprobs=rf, weights=w, mask=mask, clip_low=0.2, clip_high=0.3, kl_weight=kl, temperature=tau)
        got, g = stf.policy_loss_and_grad(x, tokens, old, adv, d_loss=d_loss, **kw)
        want = ref.policy(r, host(old), host(adv), host(rf) if kl else None, host(w) if weighted else None,
                          0.2, 0.3, kl, d_loss)
        assert want["near"] > 2
        assert int(got.rows) == want["rows"] and int(got.clipped) == want["clipped"]
        close(host(got.logprobs), r["lp"], r["err"] + H * np.abs(r["lp"]), "logprobs")
        close(host(got.loss), want["loss"], want["loss_err"], "loss")
        close(host(got.kl), want["kl"], want["kl_err"], "kl")
        check_grad(g, x, r, want["c"], want["c_err"])
        alone = stf.policy_loss(x, tokens, old, adv, **kw)
        # the pass without a gradient may add a row up in another order: within the same bounds
        assert int(alone.rows) == want["rows"] and int(alone.clipped) == want["clipped"]
        close(host(alone.logprobs), r["lp"], r["err"] + H * np.abs(r["lp"]), "logprobs without gradient")
        close(host(alone.loss), want["loss"], want["loss_err"], "loss without gradient")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairs,T,V", [(1, 2, 50), (1, 0, 50), (3, 100, 1000), (700, 3000, 64), (2, 37, 20001)])
def test_preference(pairs, T, V, dtype):
    import torch
    rng = np.random.default_rng(pairs + T + V)
    x = batch(rng, T, V, dtype, pad=2)
    tokens = some_tokens(rng, x)
    cut = np.sort(rng.integers(0, T + 1, 2 * pairs + 1))  # rows before the first and behind the last among them
    offsets = torch.from_numpy(cut).cuda()
    for average, smoothing, margin, masked in ((False, 0.0, 0.0, False), (True, 0.1, 0.5, True)):
        say("preference", pairs, T, V, dtype, average)
        mask = torch.from_numpy(rng.random(T) < 0.6).cuda() if masked else None
        r = ref.rows(host(x), tokens.cpu().numpy(), 1.0, mask.cpu().numpy() if masked else None)
        rf = values(r["lp"] + 0.3 * rng.standard_normal(T)) if not average else None
        got = stf.preference_loss(x, tokens, offsets, rf, mask, beta=0.3, smoothing=smoothing, margin=margin,
                                  average=average)
        want = ref.preference(r, cut, pairs, host(rf) if rf is not None else None, 0.3, smoothing, margin,
                              average)
        close(host(got.logprobs), r["lp"], r["err"] + H * np.abs(r["lp"]), "logprobs")
        close(host(got.margins), want["margins"], want["z_err"], "margins")
        close(host(got.sequence_logprobs), want["sequence_logprobs"], want["sums_err"], "sums")
        close(host(got.loss), want["loss"], want["loss_err"], "loss")
        close(host(got.coefficients), want["c"], want["c_err"] + H * np.abs(want["c"]), "coefficients")
        assert int(got.rows) == want["rows"]
        d_loss = 16.0 * max(T, 1)
        g = stf.preference_loss_grad(x, tokens, got, d_loss=d_loss, mask=mask)
        check_grad(g, x, r, want["c"] * d_loss, (want["c_err"] + 2 * H * np.abs(want["c"])) * d_loss)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_without_part(dtype):
    """Masked rows hold anything; tokens outside; blocked tokens; rows of -inf; lowest values."""
    import torch
    rng = np.random.default_rng(5)
    T, V = 12, 777
    x = batch(rng, T, V, dtype)
    low = torch.finfo(x.dtype).min
    tokens = some_tokens(rng, x)
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    x[0] = float("nan"); mask[0] = False
    x[1] = float("inf"); mask[1] = False
    tokens[2] = -1
    tokens[3] = V
    tokens[4] = -(1 << 62)
    x[5] = float("-inf")
    x[6, int(tokens[6])] = float("-inf")
    x[7] = low
    x[8, :700] = low; tokens[8] = 3
    x[9, :] = float("-inf"); x[9, 11] = -3.0; tokens[9] = 11
    x[10, 5] = float("nan")
    x[11, 6] = float("inf")
    say("rows without part", dtype)
    check_logprobs(x, tokens, 1.0, mask, values(np.ones(T)))
    r = stf.token_logprobs(x, tokens, mask=mask)
    assert r[:5].tolist() == [0.0] * 5 and r[5] == float("-inf") and r[6] == float("-inf") and r[9] == 0
    assert torch.isnan(r[10:]).all() and bool(torch.isfinite(r[7])) and bool(r[8] < -1e4)
    g = stf.token_logprobs_grad(x, tokens, values(np.ones(T)), mask=mask)
    assert not g[:7].any() and not g[9].any() and torch.isnan(g[10:]).any(dim=1).all()
    keep = slice(0, 10)
    old, adv = values(np.full(T, -3.0)), values(np.ones(T))
    got, g = stf.policy_loss_and_grad(x[keep], tokens[keep], old[keep], adv[keep], ref_logprobs=old[keep], kl_weight=0.0,
                                      mask=mask[keep])
    assert int(got.rows) == 5 and bool(torch.isfinite(got.loss)) and not g[:7].any() and bool(torch.isfinite(g).all())
    got, g = stf.policy_loss_and_grad(x, tokens, old, adv, mask=mask)
    assert torch.isnan(got.loss) and torch.isnan(g[10:]).any(dim=1).all() and not g[:7].any()
    none = torch.zeros(T, dtype=torch.bool, device="cuda")
    got, g = stf.policy_loss_and_grad(x, tokens, old, adv, mask=none)
    assert [float(got.loss), float(got.kl), int(got.clipped), int(got.rows)] == [0, 0, 0, 0] and not g.any()
    p = stf.preference_loss(x, tokens, torch.tensor([0, 7, 10], device="cuda"), mask=mask, beta=0.01)
    assert bool(torch.isfinite(p.loss)) and int(p.rows) == 5 and not p.coefficients[:5].any()
    p = stf.preference_loss(x, tokens, torch.tensor([0, 3, 7], device="cuda"), mask=none, margin=0.25)
    assert abs(float(p.loss) - np.log1p(np.exp(0.25))) < 1e-6 and int(p.rows) == 0 and not p.coefficients.any()


def test_offsets_that_do_not_rise():
    import torch
    rng = np.random.default_rng(8)
    x = batch(rng, 20, 90, "float32")
    tokens = some_tokens(rng, x)
    r = ref.rows(host(x), tokens.cpu().numpy(), 1.0)
    for cut in ([0, 9, 4, 12, 15], [-7, 3, 3, 99, 5], [30, 2, 2, 2, 2], [5, 4, 3, 2, 1]):
        say("offsets", cut)
        got = stf.preference_loss(x, tokens, torch.tensor(cut, device="cuda"), beta=1.0)
        want = ref.preference(r, cut, 2, beta=1.0)
        close(host(got.margins), want["margins"], want["z_err"], "margins")
        close(host(got.coefficients), want["c"], want["c_err"] + H * np.abs(want["c"]), "coefficients")
        assert int(got.rows) == want["rows"]


def test_likely_tokens_keep_their_digits():
    """A token of nearly all the weight: lp and 1 - p are far below fp32's step at 1."""
    import torch
    for V in (64, 5000, 40000, 140000):
        x = torch.full((2, V), -30.0, device="cuda")
        x[:, V // 2] = 0
        tokens = torch.tensor([V // 2, V // 2], device="cuda")
        r = check_logprobs(x, tokens, 1.0, d=values([1.0, 1.0]))
        assert 0 < -r["lp"][0] < 1e-7


@pytest.mark.parametrize("dtype", TYPES)
def test_against_differences(dtype):
    """Gradients through backward(), against differences of the 64-bit definitions."""
    import torch
    rng = np.random.default_rng(11)
    T, V = 9, 23
    x = batch(rng, T, V, dtype).detach().clone().requires_grad_()
    tokens = some_tokens(rng, x)
    n = host(x)
    old, adv = values(ref.rows(n, tokens.cpu().numpy(), 1.0)["lp"] + 0.05), values(rng.standard_normal(T))
    rf = values(host(old) + 0.2 * rng.standard_normal(T))
    offsets = torch.tensor([0, 2, 5, 6, 9], device="cuda")
    a = tokens.cpu().numpy()

    def of(kind, v):
        r = ref.rows(v, a, 1.0)
        if kind == "logprobs":
            return float(r["lp"] @ host(adv))
        if kind == "policy":
            return ref.policy(r, host(old), host(adv), host(rf), None, 0.2, 0.2, 0.5)["loss"]
        return ref.preference(r, [0, 2, 5, 6, 9], 2, host(rf), 0.4)["loss"]

    for kind in ("logprobs", "policy", "preference"):
        x.grad = None
        if kind == "logprobs":
            (stf.token_logprobs(x, tokens) * adv).sum().backward()
        elif kind == "policy":
            stf.policy_loss(x, tokens, old, adv, rf, kl_weight=0.5).loss.backward()
        else:
            stf.preference_loss(x, tokens, offsets, rf, beta=0.4).loss.backward()
        step = 1e-5
        want = np.zeros((T, V))
        for t in range(T):
            for j in range(V):
                up, down = n.copy(), n.copy()
                up[t, j] += step
                down[t, j] -= step
                want[t, j] = (of(kind, up) - of(kind, down)) / (2 * step)
        half = torch.finfo(x.dtype).eps / 2
        # differences of 64 bits: 2^-53 of the value over the step, and the step's square
        close(host(x.grad), want, (half + 1e-4) * np.abs(want) + 1e-7, kind)


def test_one_step_together():
    """Tokens drawn, scored by the old and a reference model, and learned from."""
    import torch
    rng = np.random.default_rng(3)
    T, V = 64, 3000
    x = batch(rng, T, V, "bfloat16")
    u = values(rng.random(T))
    tokens, drawn = stf.sample_tokens(x, u)
    old = stf.token_logprobs(x, tokens)
    assert bool((old - drawn).abs().max() < 1e-5)
    reference = stf.token_logprobs(batch(rng, T, V, "bfloat16"), tokens)
    leaf = x.detach().clone().requires_grad_()
    r = stf.policy_loss(leaf, tokens, old, values(rng.standard_normal(T)), ref_logprobs=reference, kl_weight=0.01)
    r.loss.backward()
    assert int(r.clipped) == 0 and torch.equal(r.logprobs, old) and bool(torch.isfinite(leaf.grad).all())
