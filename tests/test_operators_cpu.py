"""The language-model operators' argument checks, without a GPU: the C entry points return
before anything is enqueued, and the binding refuses what is no device tensor."""
import ctypes

import pytest

import sampling_threshold_filtering_amd as stf
from sampling_threshold_filtering_amd.operators import Sampling

FAKE = 1 << 20  # never dereferenced: every call below is refused before a launch


def lib():
    return stf.load_library()


def test_scratch_queries():
    L = lib()
    for B, V in ((0, 1), (1, 1), (4096, 1 << 17), (7, 1 << 24)):
        assert L.profk_sample_tokens_scratch(B, V) >= 0
    for B, V in ((-1, 5), (1, 0), (1, (1 << 24) + 1)):
        assert L.profk_sample_tokens_scratch(B, V) == stf.PROFK_EINVAL
    for T, E in ((0, 1), (1, 1), (1 << 20, 1024)):
        assert L.profk_route_scratch(T, E) > 0
    for T, E in ((-1, 5), (1, 0), (1, 1025)):
        assert L.profk_route_scratch(T, E) == stf.PROFK_EINVAL


def test_sample_tokens_refusals():
    how = Sampling(1.0, 1.0, 0.0, 0, 0, None, None, None, None)

    def call(x=FAKE, dtype=0, B=2, V=10, ld=10, u=FAKE, h=how, tok=FAKE, lp=FAKE, scratch=FAKE, size=1 << 40):
        return lib().profk_sample_tokens(x, dtype, B, V, ld, u, ctypes.byref(h) if h else None, tok, lp, scratch, size,
                                         None)

    for kw in (dict(x=None), dict(dtype=3), dict(dtype=-1), dict(B=-1), dict(V=0), dict(ld=9), dict(u=None),
               dict(h=None), dict(tok=None), dict(lp=None)):
        assert call(**kw) == stf.PROFK_EINVAL, kw
    assert call(V=(1 << 24) + 1, ld=1 << 25) == stf.PROFK_EUNSUPPORTED
    assert call(B=1 << 31) == stf.PROFK_EUNSUPPORTED
    assert call(B=0, x=None, u=None, tok=None, lp=None, scratch=None, size=0) == stf.PROFK_OK
    need = lib().profk_sample_tokens_scratch(1, 1 << 20)
    if need:
        assert call(B=1, V=1 << 20, ld=1 << 20, size=need - 1) == stf.PROFK_ESCRATCH
        assert call(B=1, V=1 << 20, ld=1 << 20, scratch=None) == stf.PROFK_EINVAL
        assert call(B=1, V=1 << 20, ld=1 << 20, scratch=FAKE + 4) == stf.PROFK_EINVAL


def test_route_refusals():
    def call(x=FAKE, dtype=0, T=4, E=10, ld=10, mask=None, k=2, w=FAKE, e=FAKE, c=FAKE, r=FAKE, loss=None, s=FAKE,
             size=1 << 40):
        return lib().profk_route_tokens(x, dtype, T, E, ld, mask, k, 1, w, e, c, r, loss, s, size, None)

    for kw in (dict(x=None), dict(dtype=7), dict(T=-1), dict(E=0), dict(ld=9), dict(k=0), dict(k=11), dict(w=None),
               dict(e=None), dict(c=None), dict(r=None), dict(s=None), dict(s=FAKE + 8)):
        assert call(**kw) == stf.PROFK_EINVAL, kw
    assert call(E=1025, ld=2000) == stf.PROFK_EUNSUPPORTED
    assert call(E=100, ld=100, k=65) == stf.PROFK_EUNSUPPORTED
    assert call(T=1 << 31) == stf.PROFK_EUNSUPPORTED
    assert call(size=lib().profk_route_scratch(4, 10) - 1) == stf.PROFK_ESCRATCH

    def bal(e=FAKE, c=FAKE, r=FAKE, loss=FAKE, k=2):
        return lib().profk_balance_loss(FAKE, 0, 4, 10, 10, None, e, k, c, r, loss, FAKE, 1 << 40, None)

    for kw in (dict(e=None), dict(c=None), dict(r=None), dict(loss=None), dict(k=0)):
        assert bal(**kw) == stf.PROFK_EINVAL, kw


def test_gradient_refusals():
    def call(T=4, k=2, e=FAKE, dw=FAKE, c=FAKE, r=FAKE, out=FAKE):
        return lib().profk_route_tokens_grad(FAKE, 0, T, 10, 10, None, k, 1, e, dw, c, r, None, 1.0, out, None)

    for kw in (dict(out=None), dict(e=None), dict(r=None), dict(dw=None, c=None), dict(k=0), dict(T=-1)):
        assert call(**kw) == stf.PROFK_EINVAL, kw
    assert call(T=0, out=None) == stf.PROFK_OK

    def bal(c=FAKE, r=FAKE, out=FAKE):
        return lib().profk_balance_loss_grad(FAKE, 0, 4, 10, 10, None, 2, c, r, None, 1.0, out, None)

    for kw in (dict(c=None), dict(r=None), dict(out=None)):
        assert bal(**kw) == stf.PROFK_EINVAL, kw


def test_binding_takes_device_tensors_only():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 10))
    with pytest.raises(ValueError):
        stf.sample_tokens(x, torch.zeros(2))
    with pytest.raises(ValueError):
        stf.route_tokens(x, 2)
    with pytest.raises(ValueError):
        stf.balance_loss(x, torch.zeros((2, 1), dtype=torch.int64))
    with pytest.raises(ValueError):
        stf.route_tokens_grad(x, stf.Routing(None, torch.zeros((2, 1), dtype=torch.int64), None, None, None))
