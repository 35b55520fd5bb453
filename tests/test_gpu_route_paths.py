"""Routing where the kernels part ways: selection keys that cannot tell neighbours apart, rows
with infinities, one block or many, four entries a load or one.

Compared as in test_gpu_route (the definition in 64 bits, its tolerances)."""
import numpy as np
import pytest

import sampling_threshold_filtering_amd as stf
from tests.test_gpu_route import TYPES, check_route, logits, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(5, 5), (16, 3), (60, 4), (64, 20), (128, 8), (192, 17), (256, 9), (300, 64), (1024, 33)])
def test_values_that_differ_in_their_last_bits(E, k):
    import torch
    rng = np.random.default_rng(E)
    T = 70
    one = np.float32(1.0).view(np.int32)
    x = (one + rng.integers(0, 6, (T, E))).astype(np.int32).view(np.float32)  # 1 + 0..5 steps of 2^-23
    x[10:20] *= -1
    x[20:30] = (rng.integers(0, 9, (10, E)) * 1e-45).astype(np.float32)       # the smallest numbers, zeros
    x[30:40, ::2] = rng.standard_normal((10, (E + 1) // 2)).astype(np.float32)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    for normalize in (True, False):
        say("close", E, k, normalize)
        check_route(torch.from_numpy(x).cuda(), k, normalize, d_weights=dw, d_loss=0.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [8, 60, 256, 700])
def test_infinite_and_nan_rows_do_not_touch_others(E, dtype):
    import torch
    rng = np.random.default_rng(E + 1)
    T, k = 90, 3
    x = logits(rng, T, E, dtype)
    clean = x.clone()
    x[7, 5] = float("inf")
    x[8, [2, 6]] = float("inf")
    x[9, 4] = float("nan")
    x[10, 3] = -torch.tensor(float("nan"), device="cuda")  # either sign
    bad = [7, 8, 9, 10]
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    for normalize in (True, False):
        say("bad rows", E, dtype, normalize)
        r = stf.route_tokens(x, k, normalize=normalize, balance=True)
        assert torch.isnan(r.weights[bad]).all() and torch.isnan(r.loss)
        assert r.experts[7, 0].item() == 5 and r.experts[8, :2].tolist() == [2, 6]
        assert r.experts[9, 0].item() == 4 and r.experts[10, 0].item() == 3
        good = [t for t in range(T) if t not in bad]
        want = stf.route_tokens(clean, k, normalize=normalize)
        assert torch.equal(r.weights[good], want.weights[good]) and torch.equal(r.experts[good], want.experts[good])
        g = stf.route_tokens_grad(x, r, dw, None, normalize=normalize)
        assert torch.isnan(g[[7, 9]]).any(dim=1).all()
        assert torch.equal(g[good], stf.route_tokens_grad(clean, want, dw, None, normalize=normalize)[good])
        mask[bad] = False  # masked, they count nowhere
        check_route(clean, k, normalize, mask, dw, 0.2)
        m = stf.route_tokens(x, k, normalize=normalize, mask=mask, balance=True)
        w = stf.route_tokens(clean, k, normalize=normalize, mask=mask, balance=True)
        assert all(torch.equal(a, b) for a, b in zip(m, w))
        mask[bad] = True


@pytest.mark.parametrize("T", [15, 16, 17, 63, 64, 65, 255, 256, 257, 1023, 1025])
@pytest.mark.parametrize("E", [12, 61, 64, 600])
def test_one_block_and_many(T, E):
    import torch
    rng = np.random.default_rng(T * 1000 + E)
    x = logits(rng, T, E, "float16")
    dw = torch.from_numpy(rng.standard_normal((T, 2)).astype(np.float32)).cuda()
    mask = torch.from_numpy(rng.random(T) < 0.9).cuda()
    say("blocks", T, E)
    check_route(x, 2, True, mask, dw, 0.3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [4, 64, 160, 256, 512, 1024])
def test_four_at_a_time_and_one_give_the_same_choice(E, dtype):
    """The same rows at another alignment: the choice and the counts are equal, the weights
    within the rounding of sums in another order."""
    import torch
    rng = np.random.default_rng(E + 3)
    T, k = 133, min(8, E)
    x = logits(rng, T, E, dtype)
    wide = torch.zeros((T, E + 3), dtype=x.dtype, device="cuda")
    wide[:, 1:E + 1] = x
    a = stf.route_tokens(x, k, balance=True)
    b = stf.route_tokens(wide[:, 1:E + 1], k, balance=True)
    assert torch.equal(a.experts, b.experts) and torch.equal(a.counts, b.counts) and torch.equal(a.rows, b.rows)
    assert torch.equal(a.weights, b.weights)  # by the chosen entries' exponentials alone, in the same order
    say("quad", E, dtype)
    check_route(wide[:, 1:E + 1], k, False, d_loss=0.1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [191, 192, 193, 383, 384, 385, 512, 513, 767, 768, 769])
def test_expert_counts_at_the_limits_of_each_layout(E, dtype):
    import torch
    rng = np.random.default_rng(E + 5)
    T, k = 75, 40
    x = logits(rng, T, E, dtype)
    x[3] = 0.0
    x[4, E // 2:] = float("-inf")
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    say("limits", E, dtype)
    for normalize in (True, False):
        check_route(x, k, normalize, d_weights=dw, d_loss=0.4)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,k", [(20, 3), (33, 5), (64, 8)])
def test_long_batches_against_their_parts_and_64_bits(E, k, dtype):
    """From 65536 tokens on another layout takes the rows: the choice equals that of two
    shorter batches, and the gradient and the loss the formula's in 64 bits (their error: the
    exponentials', 4 h and |d| h for the difference, twice for p and a sum over a row's
    entries, and half a step of the logits' type)."""
    import torch
    rng = np.random.default_rng(E)
    T = 65536 + 77
    x = logits(rng, T, E, dtype)
    mask = torch.from_numpy(rng.random(T) < 0.9).cuda()
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    d_loss = 0.01 * T
    say("long", E, k, dtype)
    r = stf.route_tokens(x, k, normalize=False, mask=mask, balance=True)
    g = stf.route_tokens_grad(x, r, dw, d_loss, normalize=False, mask=mask)
    a = stf.route_tokens(x[:30000], k, normalize=False, mask=mask[:30000])
    b = stf.route_tokens(x[30000:], k, normalize=False, mask=mask[30000:])
    assert torch.equal(r.experts, torch.cat([a.experts, b.experts]))
    assert torch.equal(r.counts, a.counts + b.counts) and int(r.rows) == int(a.rows) + int(b.rows)
    p = torch.softmax(x.double(), dim=1) * mask.unsqueeze(1)
    n = int(mask.sum())
    f = r.counts.double() / (n * k)
    tol = (64 + 4 * 20) * 2.0 ** -24
    assert float((x.float().amax(1) - x.float().amin(1)).max()) <= 20
    w = p.gather(1, r.experts.clamp(min=0)) * (r.experts >= 0)
    assert ((r.weights.double() - w).abs() <= tol * w).all()
    loss = float((E * f * p.sum(dim=0) / n).sum())
    assert abs(float(r.loss) - loss) <= tol * loss
    d = torch.zeros_like(p).scatter_add_(1, r.experts.clamp(min=0), dw.double() * (r.experts >= 0))
    want = p * (d - (p * d).sum(1, keepdim=True)) + d_loss * E / n * p * (f - (p * f).sum(1, keepdim=True))
    big = d.abs().amax(1, keepdim=True)
    size = 2 * big * p + d_loss * E / n * p * (f + (p * f).sum(1, keepdim=True))
    half = torch.finfo(x.dtype).eps / 2
    least = float(torch.finfo(x.dtype).tiny) * 2 * half if x.dtype == torch.float16 else 1e-38
    assert ((g.double() - want).abs() <= 2 * tol * size + half * (want.abs() + 2 * tol * size) + least).all()


def test_many_slots_of_one_expert_and_a_long_batch():
    import torch
    T, E, k = 150000, 8, 2
    x = torch.zeros((T, E), device="cuda")
    x[:, 3] = 5.0
    x[::2, 6] = 4.0
    r = stf.route_tokens(x, k, balance=True)
    assert r.counts.tolist() == [T // 2, 0, 0, T, 0, 0, T // 2, 0]
    p = torch.softmax(x.double(), dim=1)
    loss = float((E * r.counts.double() / (T * k) * p.mean(dim=0)).sum())
    # lane sums of at most 150000 / (512 blocks * 256 rows) + 1 = 3 terms, 4 exchanges, beside the weights' error
    assert abs(float(r.loss) - loss) <= (64 + 4 * 5 + 8) * 2.0 ** -24 * loss


def test_loss_gradient_given_on_the_device_and_scaled():
    import torch
    rng = np.random.default_rng(5)
    x = logits(rng, 500, 40, "float32")
    r = stf.route_tokens(x, 3, balance=True)
    for v in (0.0, 1e-20, 1e20, -3.0):
        g = stf.route_tokens_grad(x, r, None, v)
        assert torch.equal(g, stf.route_tokens_grad(x, r, None, torch.tensor([v], device="cuda")))
    assert torch.isnan(stf.route_tokens_grad(x, r, None, float("nan"))).all()
