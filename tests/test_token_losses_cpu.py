"""The token losses' argument checks, without a GPU: the C entry points return before anything
is enqueued, and the binding refuses what is no device tensor."""
import ctypes

import numpy as np
import pytest

import sampling_threshold_filtering_amd as stf
from sampling_threshold_filtering_amd.operators import PolicySettings, PreferenceSettings

FAKE = 1 << 20  # never dereferenced: every call below is refused before a launch


def lib():
    return stf.load_library()


def common(x=FAKE, dtype=0, T=4, V=10, ld=10, tokens=FAKE, mask=None, t=1.0):
    return [x, dtype, T, V, ld, tokens, mask, t]


BAD_ROWS = (dict(x=None), dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(V=0), dict(ld=9), dict(tokens=None), dict(t=0.0),
            dict(t=-1.0), dict(t=float("nan")), dict(t=float("inf")), dict(t=2.0 ** 21), dict(t=2.0 ** -21))


def each_call(**kw):
    """The status of every entry point with these common arguments."""
    policy = PolicySettings(FAKE, FAKE, None, None, 0.2, 0.2, 0.0)
    pairs = PreferenceSettings(FAKE, None, 1, 0.1, 0.0, 0.0, 0, 0)
    scratch = [kw.pop("scratch", FAKE), kw.pop("size", 1 << 40), None]
    c = common(**kw)
    return [lib().profk_token_logprobs(*c, FAKE, *scratch),
            lib().profk_token_logprobs_grad(*c, FAKE, None, 1.0, FAKE, *scratch),
            lib().profk_policy_loss(*c, ctypes.byref(policy), FAKE, FAKE, FAKE, FAKE, FAKE, None, 1.0, FAKE, *scratch),
            lib().profk_preference_loss(*c, ctypes.byref(pairs), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, *scratch)]


def test_scratch_query():
    for T, V in ((0, 1), (1, 1), (1 << 20, 1 << 24)):
        assert lib().profk_token_loss_scratch(T, V) > 0
    for T, V in ((-1, 5), (1, 0), (1, (1 << 24) + 1), (1 << 31, 5)):
        assert lib().profk_token_loss_scratch(T, V) == stf.PROFK_EINVAL


def test_common_refusals():
    for kw in BAD_ROWS + (dict(scratch=None), dict(scratch=FAKE + 8)):
        assert each_call(**kw) == [stf.PROFK_EINVAL] * 4, kw
    for kw in (dict(V=(1 << 24) + 1, ld=1 << 25), dict(T=1 << 31)):
        assert each_call(**kw) == [stf.PROFK_EUNSUPPORTED] * 4, kw
    assert each_call(size=lib().profk_token_loss_scratch(4, 10) - 1) == [stf.PROFK_ESCRATCH] * 4
    assert each_call(T=0, x=None, tokens=None)[:2] == [stf.PROFK_OK] * 2  # nothing to do, nothing enqueued


def test_own_refusals():
    s = [FAKE, 1 << 40, None]
    c = common()
    assert lib().profk_token_logprobs(*c, None, *s) == stf.PROFK_EINVAL
    assert lib().profk_token_logprobs_grad(*c, None, None, 1.0, FAKE, *s) == stf.PROFK_EINVAL
    assert lib().profk_token_logprobs_grad(*c, FAKE, None, 1.0, None, *s) == stf.PROFK_EINVAL

    def policy(outs=(FAKE,) * 5, none=False, **kw):
        base = dict(old_logprobs=FAKE, advantages=FAKE, clip_low=0.2, clip_high=0.2, kl_weight=0.0)
        how = PolicySettings(**{**base, **kw})
        return lib().profk_policy_loss(*c, None if none else ctypes.byref(how), *outs, None, 1.0, None, *s)

    nan, inf = float("nan"), float("inf")
    for kw in (dict(none=True), dict(old_logprobs=None), dict(advantages=None), dict(clip_low=-0.1), dict(clip_low=nan),
               dict(clip_high=-0.1), dict(clip_high=nan), dict(kl_weight=-1.0), dict(kl_weight=nan), dict(kl_weight=inf)):
        assert policy(**kw) == stf.PROFK_EINVAL, kw
    for i in range(5):
        assert policy(outs=tuple(None if j == i else FAKE for j in range(5))) == stf.PROFK_EINVAL

    def preference(outs=(FAKE,) * 6, none=False, **kw):
        how = PreferenceSettings(**{**dict(offsets=FAKE, pairs=1, beta=0.1, smoothing=0.0, margin=0.0), **kw})
        return lib().profk_preference_loss(*c, None if none else ctypes.byref(how), *outs, *s)

    for kw in (dict(none=True), dict(offsets=None), dict(pairs=0), dict(pairs=-1), dict(beta=nan), dict(beta=inf),
               dict(margin=nan), dict(smoothing=-0.1), dict(smoothing=1.1), dict(smoothing=nan)):
        assert preference(**kw) == stf.PROFK_EINVAL, kw
    assert preference(pairs=1 << 30) == stf.PROFK_EUNSUPPORTED
    for i in range(6):
        assert preference(outs=tuple(None if j == i else FAKE for j in range(6))) == stf.PROFK_EINVAL


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x, a = torch.zeros(2, 5), torch.zeros(2, dtype=torch.int64)
    f = torch.zeros(2)
    for call in (lambda v: stf.token_logprobs(v, a), lambda v: stf.token_logprobs_grad(v, a, f),
                 lambda v: stf.policy_loss(v, a, f, f), lambda v: stf.policy_loss_and_grad(v, a, f, f),
                 lambda v: stf.preference_loss(v, a, torch.tensor([0, 1, 2]))):
        with pytest.raises(ValueError):
            call(x)
        with pytest.raises(ValueError):
            call(x.requires_grad_())
    with pytest.raises(ValueError):
        stf.policy_loss_and_grad(x, a, f, f, d_loss=None)


def test_definitions_against_differences():
    """The oracle's gradients are those of its losses."""
    from tests import losses_ref as ref
    rng = np.random.default_rng(0)
    T, V = 6, 7
    x = rng.standard_normal((T, V)) * 2
    a = rng.integers(0, V, T)
    a[2] = -1
    lp = ref.rows(x, a, 0.8)["lp"]
    old, adv, rf = lp + 0.1 * rng.standard_normal(T), rng.standard_normal(T), lp + 0.3 * rng.standard_normal(T)
    cut = [0, 2, 3, 4, 6]

    def policy(v):
        return ref.policy(ref.rows(v, a, 0.8), old, adv, rf, None, 0.05, 0.05, 0.3)

    def preference(v):
        return ref.preference(ref.rows(v, a, 0.8), cut, 2, rf, 0.7, 0.1, 0.2, True)

    for f in (policy, preference):
        g, _ = ref.grad(ref.rows(x, a, 0.8), f(x)["c"])
        for t in range(T):
            for j in range(V):
                d = np.zeros_like(x)
                d[t, j] = 1e-5
                slope = (f(x + d)["loss"] - f(x - d)["loss"]) / 2e-5
                assert abs(slope - g[t, j]) < 1e-8, (f.__name__, t, j)
