"""Token sampling against its definition in 64 bits, row by row.

Tolerance of the log-probability: the kernel computes it in 64 bits from integer weights
of unit 2^-F of the largest, F = min(50, 62 - ceil(log2 V)); V of them are off by at most
V 2^-(F+1) of a mass of at least 1, and the result is rounded once to fp32 (2^-24 of it).
Tokens are equal unless the definition's decision is closer to its other side than that.
"""
import math

import numpy as np
import pytest

import sampling_threshold_filtering_amd as stf
from tests.operators_ref import sample_row

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]


def say(*a):
    print("[case]", *a, flush=True)


def weight_error(V):
    F = min(50, 62 - max(0, math.ceil(math.log2(V))))
    return V * 2.0 ** -(F + 1) + 1e-13 * V ** 0.5


def check(x, u, t=1.0, k=0, p=1.0, m=0.0, always=False, got=None):
    """x [B, V] device tensor, u [B] numpy; settings numbers or numpy arrays."""
    import torch
    B, V = x.shape
    ud = torch.from_numpy(np.asarray(u, np.float32)).cuda()

    def arg(v):
        return torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v

    def at(v, b):
        return v[b] if isinstance(v, np.ndarray) else v

    tok, lp = got if got is not None else stf.sample_tokens(x, ud, arg(t), arg(k), arg(p), arg(m))
    torch.cuda.synchronize()
    tok, lp = tok.cpu().numpy(), lp.cpu().numpy()
    rows = x.float().cpu().numpy()
    err = weight_error(V)
    compared = 0
    for b in range(B):
        f = lambda v: float(np.float32(at(v, b)))  # noqa: E731 (settings are fp32 numbers)
        et, el, margin = sample_row(rows[b], float(np.float32(u[b])), f(t), int(at(k, b)), f(p), f(m))
        if margin <= 2 * err and not always:
            continue
        compared += 1
        assert tok[b] == et, (b, tok[b], et, margin)
        if math.isfinite(el):
            assert abs(lp[b] - el) <= 2.0 ** -24 * abs(el) + 2 * err, (b, lp[b], el)
        else:
            assert (math.isnan(el) and math.isnan(lp[b])) or lp[b] == el
    assert compared >= B - 1 - B // 50
    return tok, lp


def logits(rng, B, V, dtype, spread=2.5, hot=True):
    import torch
    x = rng.standard_normal((B, V)) * spread
    if hot and V >= 8:
        for b in range(B):
            x[b, rng.integers(0, V, 5)] = spread * 4 + rng.standard_normal(5)
    return torch.from_numpy(x).to("cuda", dtype=getattr(torch, dtype))


SETTINGS = [dict(), dict(t=0.7, k=50, p=0.95), dict(t=1.3, p=0.99), dict(m=0.1), dict(t=0.8, k=7), dict(t=2.0, k=5000),
            dict(t=0.9, k=900, p=0.8, m=0.001), dict(t=0.0), dict(t=0.05, p=0.5), dict(t=30.0, p=0.3)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 3, 63, 64, 65, 1000, 4096, 4097, 32000])
def test_lengths(V, dtype):
    say("lengths", V, dtype)
    rng = np.random.default_rng(V)
    B = 5
    x = logits(rng, B, V, dtype)
    for s in SETTINGS:
        say(s)
        check(x, rng.random(B), **s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [50257, 131072, 262144])
def test_long_rows(V, dtype):
    rng = np.random.default_rng(V + 1)
    x = logits(rng, 3, V, dtype)
    for s in SETTINGS:
        say("long", V, dtype, s)
        check(x, rng.random(3), **s)


@pytest.mark.parametrize("B", [1, 2, 33, 300])
def test_batches_with_settings_per_row(B):
    rng = np.random.default_rng(B)
    V = 10007
    x = logits(rng, B, V, "bfloat16")
    t = rng.choice([0.0, 0.6, 1.0, 1.5], B).astype(np.float32)
    k = rng.choice([0, 1, 40, 1000, V, 6000], B).astype(np.int64)
    p = rng.choice([1.0, 0.9, 0.5, 0.0], B).astype(np.float32)
    m = rng.choice([0.0, 0.05, 1.0], B).astype(np.float32)
    say("rows", B)
    check(x, rng.random(B), t, k, p, m)
    check(x, rng.random(B), t.astype(np.float64), k.astype(np.int32), 0.9, m)


@pytest.mark.parametrize("V", [5, 4096, 5000, 20000])
@pytest.mark.parametrize("value", [0.0, -3.5, float(np.finfo(np.float32).min)])
def test_equal_entries_go_by_index(V, value):
    """One value everywhere (also the type's lowest, as masks use it): every weight is 2^F
    exactly, so every border is exact and ties go by index."""
    import torch
    x = torch.full((8, V), value, device="cuda")
    u = np.array([0.0, 0.25, 0.5, 0.75, 0.1, 0.9, 1 - 2.0 ** -24, 0.3], np.float32)
    for s in (dict(), dict(k=3), dict(k=4999), dict(p=0.5), dict(p=0.25, m=1.0), dict(t=3.0, k=17, p=0.6)):
        say("equal", V, value, s)
        check(x, u, always=True, **s)


def test_crowded_bins_are_split():
    """Tens of thousands of entries within one value bin, all different; and in two values."""
    import torch
    rng = np.random.default_rng(5)
    V = 40000
    x = torch.from_numpy((1.0 + 1e-5 * rng.standard_normal((4, V))).astype(np.float32)).cuda()
    y = torch.from_numpy(rng.choice([0.5, 0.5 + 2.0 ** -10], (4, V)).astype(np.float32)).cuda()
    z = torch.from_numpy((1e-30 * rng.standard_normal((4, V))).astype(np.float32)).cuda()
    for s in (dict(), dict(k=9000), dict(p=0.5), dict(t=0.5, k=30000, p=0.7)):
        say("crowded", s)
        check(x, rng.random(4), **s)
        check(y, rng.random(4), **s)
        check(z, rng.random(4), always=True, **s)  # every weight is 1 in 64 bits: exact borders


@pytest.mark.parametrize("dtype", TYPES)
def test_masks_infinities_and_nan(dtype):
    import torch
    rng = np.random.default_rng(9)
    V = 3001
    x = logits(rng, 8, V, dtype)
    x[0] = float("-inf")                                # nothing left
    x[1, :] = float("-inf")
    x[1, 2500] = -7.0                                   # one entry left
    x[2, rng.integers(0, V, 2900)] = float("-inf")      # few left
    x[3, [17, 2999]] = float("inf")                     # two share everything
    x[4, 100] = float("nan")
    x[5, rng.integers(0, V, 2000)] = torch.finfo(x.dtype).min
    x[6] = float("-inf")
    x[6, 5] = torch.finfo(x.dtype).min
    x[7, :] = torch.finfo(x.dtype).max
    for s in (dict(), dict(t=0.6, k=50, p=0.9), dict(m=0.2), dict(t=0.0), dict(t=1e-6), dict(t=1e4, p=0.7)):
        say("masks", dtype, s)
        tok, lp = check(x, rng.random(8), **s)
        assert tok[0] == -1 and lp[0] == -np.inf
        assert tok[1] == 2500 and lp[1] == 0.0
        assert tok[4] == -1 and np.isnan(lp[4])
        assert tok[3] in (17, 2999) and tok[6] == 5


def test_signed_zeros_tie():
    import torch
    x = torch.tensor([[-0.0, 0.0, -0.0, -1.0], [0.0, -0.0, -0.0, -1.0]], device="cuda")
    tok, _ = check(x, [0.0, 0.0], always=True)
    assert tok.tolist() == [0, 0]
    tok, _ = check(x, [0.0, 0.5], k=2, always=True)
    assert tok.tolist() == [0, 1]


def test_uniform_numbers_at_and_past_the_ends():
    import torch
    rng = np.random.default_rng(3)
    x = logits(rng, 6, 1000, "float32", hot=False)
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 5.0, -1.0, float("nan")]).cuda()
    tok, _ = stf.sample_tokens(x, u, top_k=10)
    order = torch.sort(x, dim=1, descending=True, stable=True)[1].cpu()
    want = [order[0, 0], order[1, 9], order[2, 9], order[3, 9], order[4, 0], order[5, 0]]
    assert tok.tolist() == [int(v) for v in want]


def test_rows_strided_offset_and_transposed():
    import torch
    rng = np.random.default_rng(4)
    for dtype in TYPES:
        wide = logits(rng, 7, 5003, dtype)
        for x in (wide[:, 1:], wide[:, 3:4003], wide[::2, 7:], wide.t()[:900].t(), wide[:, ::3],
                  wide[:1].expand(4, -1), wide.t()):
            say("strides", dtype, tuple(x.shape), x.stride())
            check(x, rng.random(x.shape[0]), t=0.9, k=40, p=0.9)
            check(x, rng.random(x.shape[0]), t=0.9, p=0.97)


def test_empty_batch_out_buffers_and_repeats():
    import torch
    x = torch.empty((0, 100), device="cuda")
    tok, lp = stf.sample_tokens(x, torch.empty(0, device="cuda"))
    assert tok.shape == (0,) and lp.shape == (0,)
    rng = np.random.default_rng(8)
    x = logits(rng, 9, 70001, "float16")
    u = torch.from_numpy(rng.random(9).astype(np.float32)).cuda()
    out = (torch.full((9,), -5, dtype=torch.int64, device="cuda"), torch.zeros(9, device="cuda"))
    got = stf.sample_tokens(x, u, 1.2, 0, 0.98, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    check(x, u.cpu().numpy(), 1.2, 0, 0.98, got=out)
    first = [t.clone() for t in out]
    for _ in range(3):
        a, b = stf.sample_tokens(x, u, 1.2, 0, 0.98)
        assert torch.equal(a, first[0]) and torch.equal(b, first[1])


def test_a_row_does_not_depend_on_its_batch():
    """Integer weights: the same row, alone and in batches of any size, gives the same bits."""
    import torch
    rng = np.random.default_rng(12)
    x = logits(rng, 200, 33000, "bfloat16", spread=1.5, hot=False)
    u = torch.from_numpy(rng.random(200).astype(np.float32)).cuda()
    whole = stf.sample_tokens(x, u, 1.1, 0, 0.99)
    for b in (0, 77, 199):
        one = stf.sample_tokens(x[b:b + 1], u[b:b + 1], 1.1, 0, 0.99)
        assert one[0].item() == whole[0][b].item() and one[1].item() == whole[1][b].item()
    part = stf.sample_tokens(x[:13], u[:13], 1.1, 0, 0.99)
    assert torch.equal(part[0], whole[0][:13]) and torch.equal(part[1], whole[1][:13])


def test_other_stream_and_graph():
    import torch
    rng = np.random.default_rng(10)
    x = logits(rng, 4, 40000, "bfloat16")
    u = torch.from_numpy(rng.random(4).astype(np.float32)).cuda()
    want = stf.sample_tokens(x, u, 0.8, 30, 0.9)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = stf.sample_tokens(x, u, 0.8, 30, 0.9)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = (torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        stf.sample_tokens(x, u, 0.8, 30, 0.9, out=out)
    for i in range(4):  # new inputs each replay, with the program's own calls between
        x.copy_(logits(rng, 4, 40000, "bfloat16"))
        u.copy_(torch.from_numpy(rng.random(4).astype(np.float32)))
        want = stf.sample_tokens(x, u, 0.8, 30, 0.9)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), i


def test_refusals():
    import torch
    x = torch.zeros((2, 10), device="cuda")
    u = torch.zeros(2, device="cuda")
    bad = [dict(temperature=-1.0), dict(top_k=-1), dict(top_p=1.5), dict(top_p=-0.1), dict(min_p=2.0),
           dict(temperature=float("nan")), dict(top_p=torch.zeros(3, device="cuda")), dict(top_p=torch.zeros(2)),
           dict(top_k=torch.zeros(2, device="cuda")), dict(temperature=torch.zeros(2, dtype=torch.int64, device="cuda"))]
    for kw in bad:
        with pytest.raises(ValueError):
            stf.sample_tokens(x, u, **kw)
    for xx, uu in ((x.double(), u), (x[0], u), (x, u.double()), (x, u[:1]), (x, u.cpu()),
                   (torch.zeros((2, 0), device="cuda"), u)):
        with pytest.raises(ValueError):
            stf.sample_tokens(xx, uu)
    with pytest.raises(ValueError):
        stf.sample_tokens(x, u, out=(torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda")))
