"""The token losses where a mask's bytes, a margin, a ratio or a setting is as far out as it may be.

Tolerances as in losses_ref.py.  Where a result has to be what another call gives, the two calls
do the same arithmetic on the rows that count, and are compared bit for bit.
"""
import numpy as np
import pytest

import sampling_threshold_filtering_amd as stf
from tests import losses_ref as ref
from tests.test_gpu_loss_edges import policy_inputs
from tests.test_gpu_token_losses import TYPES, H, batch, close, host, say, some_tokens, values

pytestmark = pytest.mark.gpu

INF = float("inf")
# rows a wavefront each, a workgroup each, in slices
SIZES = [(700, 300), (300, 9000), (40, 40000)]


def same(a, b):
    import torch
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("T,V", SIZES)
def test_any_mask_byte_but_zero_is_set(T, V):
    import torch
    x, tokens, old, adv, w, _ = policy_inputs(T, V, "bfloat16", T, True)
    d = torch.randn(T, device="cuda")
    offsets = torch.tensor([0, T // 4, T // 3, T // 2, T], device="cuda")
    some = torch.tensor([0, 1, 2, 4, 0x80, 0xFE, 0, 0xFF], dtype=torch.uint8, device="cuda")
    byte = some.repeat(T // 8 + 1)[:T]
    say("mask bytes", T, V)

    def step(mask):
        p, g = stf.policy_loss_and_grad(x, tokens, old, adv, ref_logprobs=old, kl_weight=0.1, mask=mask)
        q, h = stf.policy_loss_and_grad(x, tokens, old, adv, weights=w, mask=mask)
        z = stf.preference_loss(x, tokens, offsets, old, mask)
        return (*p, g, *q, h, *stf.policy_loss(x, tokens, old, adv, mask=mask), *z,
                stf.preference_loss_grad(x, tokens, z, 1.0, mask), stf.token_logprobs(x, tokens, mask),
                stf.token_logprobs_grad(x, tokens, d, mask))

    odd = step(byte.view(torch.bool))
    assert int(odd[4]) == int((byte != 0).sum())  # the live rows
    assert same(odd, step(byte != 0))
