"""Routing by scores: the C entries' argument checks, which return before anything is enqueued,
and the oracle's gradients against differences of its values; no GPU."""
import ctypes

import numpy as np
import pytest

import sampling_threshold_filtering_amd as stf
from sampling_threshold_filtering_amd.operators import ScoringSettings
from tests.operators_ref import scored

FAKE = 1 << 20  # never dereferenced: every call below is refused before a launch


def lib():
    return stf.load_library()


def test_refusals():
    def call(x=FAKE, dtype=0, T=4, E=12, ld=12, k=2, w=FAKE, e=FAKE, c=FAKE, r=FAKE, s=FAKE, size=1 << 40, none=False, **kw):
        how = ScoringSettings(**{**dict(scores=1, groups=4, top_groups=2, group_best=2, scale=1.0), **kw})
        return lib().profk_route_scored(x, dtype, T, E, ld, None, k, None if none else ctypes.byref(how), w, e, c, r, None,
                                        s, size, None)

    nan, inf = float("nan"), float("inf")
    for kw in (dict(x=None), dict(dtype=7), dict(T=-1), dict(E=0), dict(ld=11), dict(k=0), dict(k=13), dict(w=None),
               dict(e=None), dict(c=None), dict(r=None), dict(s=None), dict(s=FAKE + 8), dict(none=True), dict(scores=2),
               dict(scores=-1), dict(groups=0), dict(groups=5), dict(top_groups=0), dict(top_groups=5),
               dict(group_best=0), dict(group_best=3), dict(scale=nan), dict(scale=inf)):
        assert call(**kw) == stf.PROFK_EINVAL, kw
    assert call(E=1025, ld=2000, groups=5) == stf.PROFK_EUNSUPPORTED
    assert call(E=130, ld=130, groups=65) == stf.PROFK_EUNSUPPORTED
    assert call(T=1 << 31) == stf.PROFK_EUNSUPPORTED
    assert call(size=lib().profk_route_scratch(4, 12) - 1) == stf.PROFK_ESCRATCH


def test_gradient_refusals():
    def call(T=4, k=2, scores=1, scale=1.0, e=FAKE, dw=FAKE, c=FAKE, r=FAKE, out=FAKE):
        return lib().profk_route_scored_grad(FAKE, 0, T, 10, 10, None, k, 1, scores, scale, e, dw, c, r, None, 1.0, out, None)

    for kw in (dict(out=None), dict(e=None), dict(r=None), dict(dw=None, c=None), dict(k=0), dict(T=-1), dict(scores=2),
               dict(scale=float("nan"))):
        assert call(**kw) == stf.PROFK_EINVAL, kw
    assert call(T=0, out=None) == stf.PROFK_OK


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_oracle_against_differences(scores, normalize):
    rng = np.random.default_rng(1)
    T, E, k = 4, 12, 3
    x = np.stack([rng.permutation(E) for _ in range(T)]) * 0.25 - 1.5
    how = dict(scores=scores, bias=rng.standard_normal(E) * 0.01, groups=4, top_groups=2, normalize=normalize, scale=2.0)
    d = rng.standard_normal((T, k))
    want = scored(x, k, how, None, d, 3.0)

    def value(v):
        w = scored(v, k, how)
        assert np.array_equal(w["experts"], want["experts"])
        return (w["weights"] * d).sum() + 3.0 * w["loss"]

    for t in range(T):
        for e in range(E):
            h = np.zeros_like(x)
            h[t, e] = 1e-5
            assert abs((value(x + h) - value(x - h)) / 2e-5 - want["d_logits"][t, e]) < 1e-8
