"""Token sampling where the kernels part ways: counters and lists that overflow, lengths on
both sides of what a workgroup holds in registers, rows of each kind in one batch.

Compared as in test_gpu_tokens (the definition in 64 bits, its tolerance)."""
import numpy as np
import pytest

import sampling_threshold_filtering_amd as stf
from tests.test_gpu_tokens import SETTINGS, check, logits, say

pytestmark = pytest.mark.gpu

# 4, 8 and 16 vectors of 16 bytes for each of 1024 threads: entries of 4 and of 2 bytes
EDGES = {"float32": (16384, 32768, 65536), "bfloat16": (32768, 65536, 131072), "float16": (32768, 131072)}


@pytest.mark.parametrize("dtype", sorted(EDGES))
@pytest.mark.parametrize("off", [-7, -1, 0, 1, 9])
def test_lengths_at_the_register_limits(dtype, off):
    rng = np.random.default_rng(100 + off)
    for edge in EDGES[dtype]:
        x = logits(rng, 2, edge + off + 3, dtype)
        for shift in (0, 1, 3):  # the row's first and last entries outside of whole vectors
            y = x[:, shift:shift + edge + off]
            say("edge", dtype, edge, off, shift)
            check(y, rng.random(2), t=0.9, p=0.97)
            check(y, rng.random(2), t=1.1, k=700, m=0.001)
            check(y, rng.random(2), t=0.0)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_a_value_that_fills_its_counter(dtype):
    """65535 and 65536 equal entries, and far more: all weights are 1, so borders are exact."""
    import torch
    rng = np.random.default_rng(1)
    for V in (65535, 65536, 65537, 131071, 200001):
        x = torch.full((4, V), 1.5, device="cuda").to(getattr(torch, dtype))
        x[1] = -0.0                       # and a row of both zeros
        x[1, ::3] = 0.0
        x[2, rng.integers(0, V, 50)] = float("-inf")
        u = np.array([0.0, 0.5, 0.999, 1 - 2.0 ** -24], np.float32)
        for s in (dict(), dict(k=65536), dict(k=3), dict(p=0.75, t=2.0), dict(t=0.0)):
            say("full counter", dtype, V, s)
            check(x, u, always=True, **s)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_overflowed_rows_beside_ordinary_ones(dtype):
    import torch
    rng = np.random.default_rng(2)
    B, V = 70, 140000
    x = logits(rng, B, V, dtype)
    heavy = rng.random(B) < 0.4
    heavy[0] = heavy[-1] = True
    for b in np.flatnonzero(heavy):  # one value nearly everywhere, near the top
        x[b, torch.from_numpy(rng.random(V) < 0.9).cuda()] = 3.0
    for s in (dict(), dict(t=0.7, k=50, p=0.95), dict(t=1.2, p=0.9, m=0.01)):
        say("mixed overflow", dtype, s)
        check(x, rng.random(B), **s)


def test_crowded_lists_beside_ordinary_rows():
    """fp32: more than 1024 entries of a value bin, in some rows."""
    import torch
    rng = np.random.default_rng(3)
    B, V = 66, 9001
    x = logits(rng, B, V, "float32")
    for b in range(0, B, 3):
        x[b] = torch.from_numpy((2.0 + 1e-6 * rng.standard_normal(V)).astype(np.float32)).cuda()
    x[4] = float("inf")
    x[5, 7:8000] = float("inf")
    x[7] = 0.25
    for s in (dict(), dict(k=2000), dict(t=0.8, p=0.5), dict(m=0.5), dict(t=0.0)):
        say("crowded", s)
        tok, _ = check(x, rng.random(B), **s)
        assert tok[5] >= 7
    tok, lp = stf.sample_tokens(x, torch.zeros(B, device="cuda"), temperature=0.0)
    assert tok[4].item() == 0 and tok[5].item() == 7 and tok[7].item() == 0 and (lp == 0).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("V", [700, 20000, 140000])
def test_infinities_and_temperatures_at_the_ends(V, dtype):
    import torch
    rng = np.random.default_rng(V)
    x = logits(rng, 6, V, dtype)
    x[0, [5, V - 1, V // 2]] = float("inf")
    x[1, ::2] = float("inf")
    x[2, :] = float("-inf")
    x[2, V - 2] = torch.finfo(x.dtype).min
    x[3, 3:] = torch.finfo(x.dtype).min
    x[4, 1] = torch.finfo(x.dtype).max
    for s in (dict(), dict(t=1e-30), dict(t=1e-6, k=9), dict(t=1e6, p=0.6), dict(t=0.0), dict(t=0.5, m=1.0)):
        say("ends", V, dtype, s)
        tok, _ = check(x, rng.random(6), **s)
        assert tok[0] in (5, V - 1, V // 2) and tok[1] % 2 == 0 and tok[2] == V - 2


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_top_k_at_every_border_of_a_small_row(dtype):
    """k through ties and through the groups of neighbouring values."""
    import torch
    rng = np.random.default_rng(6)
    V = 3000
    x = torch.from_numpy(np.round(rng.standard_normal((1, V)) * 8) / 8).to("cuda", dtype=getattr(torch, dtype))
    x = x.expand(64, -1).contiguous()
    k = np.unique(np.concatenate([np.arange(1, 33), rng.integers(33, V, 32)]))[:64].astype(np.int64)
    k = np.concatenate([k, np.full(64 - k.size, V, np.int64)])
    check(x, rng.random(64), t=1.0, k=k)
    check(x, rng.random(64), t=0.7, k=k, p=0.8, m=0.02)


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("V", [40000, 140000])
def test_rows_alone_and_in_batches_have_the_same_bits(V, dtype):
    import torch
    rng = np.random.default_rng(V + 7)
    x = logits(rng, 40, V, dtype, spread=1.5, hot=False)
    u = torch.from_numpy(rng.random(40).astype(np.float32)).cuda()
    for kw in (dict(temperature=1.1, top_p=0.99), dict(temperature=0.9, top_k=300, min_p=0.001)):
        whole = stf.sample_tokens(x, u, **kw)
        wide = torch.zeros((40, V + 5), dtype=x.dtype, device="cuda")
        wide[:, 3:V + 3] = x
        moved = stf.sample_tokens(wide[:, 3:V + 3], u, **kw)   # another alignment
        assert torch.equal(moved[0], whole[0]) and torch.equal(moved[1], whole[1])
        for b in (0, 39):
            one = stf.sample_tokens(x[b:b + 1], u[b:b + 1], **kw)
            assert one[0].item() == whole[0][b].item() and one[1].item() == whole[1][b].item()


def test_settings_over_a_long_row_of_floats():
    rng = np.random.default_rng(11)
    x = logits(rng, 2, 300001, "float32", spread=1.5, hot=False)
    for s in SETTINGS:
        say("long floats", s)
        check(x, rng.random(2), **s)
