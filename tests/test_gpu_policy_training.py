"""The operators as a training run uses them: a small mixture-of-experts model that routes by
scores draws tokens, scores them, and learns from a policy loss and from preferences.  Every
parameter's gradient against the same model in 64 bits by plain operations."""
import pytest

import sampling_threshold_filtering_amd as stf

pytestmark = pytest.mark.gpu
VOCAB, WIDTH, EXPERTS, CHOSEN, GROUPS = 50, 24, 12, 3, 4


def parameters(seed):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda") * shape[-2] ** -0.5

    return dict(embed=normal(VOCAB, WIDTH), router=normal(WIDTH, EXPERTS), up=normal(EXPERTS, WIDTH, WIDTH),
                head=normal(WIDTH, VOCAB))


def experts_of(p, x, weights, experts):
    import torch
    out = torch.zeros_like(x)
    for e in range(EXPERTS):
        token, slot = (experts == e).nonzero(as_tuple=True)
        y = torch.tanh(x[token] @ p["up"][e])
        out = out.index_add(0, token, y * weights[token, slot].unsqueeze(1))
    return x + out


def forward(p, tokens, mask, bias):
    x = p["embed"][tokens]
    r = stf.route_tokens(x @ p["router"], CHOSEN, scores="sigmoid", bias=bias, groups=GROUPS, top_groups=2, scale=1.5,
                         mask=mask, balance=True)
    return experts_of(p, x, r.weights, r.experts) @ p["head"], r


def plain_forward(p, tokens, mask, experts, counts, rows):
    """The same in the parameters' type, with the choice given."""
    import torch
    x = p["embed"][tokens]
    s = torch.sigmoid(x @ p["router"])
    w = s.gather(1, experts.clamp(min=0)) * mask.unsqueeze(1)
    w = 1.5 * w / w.sum(1, keepdim=True).clamp(min=1e-300)
    share = (s / s.sum(1, keepdim=True))[mask].sum(0) / rows
    balance = EXPERTS * (counts.double() / (rows * CHOSEN) * share).sum()
    return experts_of(p, x, w, experts) @ p["head"], balance


def check_gradients(p, q, tol):
    for name in p:
        g, want = p[name].grad.double(), q[name].grad
        assert float((g - want).norm()) <= tol * float(want.norm()), name


def test_a_policy_step_and_a_preference_step():
    import torch
    p = {n: v.requires_grad_() for n, v in parameters(0).items()}
    q = {n: v.detach().double().requires_grad_() for n, v in p.items()}
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    T = 600
    prompt = torch.randint(0, VOCAB, (T,), generator=gen, device="cuda")
    mask = torch.rand(T, generator=gen, device="cuda") < 0.9
    bias = torch.zeros(EXPERTS, device="cuda")
    for _ in range(4):  # the bias follows the loads, as a balance without a loss
        with torch.no_grad():
            logits, r = forward(p, prompt, mask, bias)
        bias = bias + 0.02 * torch.sign(r.counts.float().mean() - r.counts.float())
    assert int(r.rows) == int(mask.sum()) and int(r.counts.sum()) == CHOSEN * int(r.rows)
    drawn, old = stf.sample_tokens(logits, torch.rand(T, generator=gen, device="cuda"))
    assert torch.allclose(stf.token_logprobs(logits, drawn), old, rtol=1e-5, atol=1e-6)
    old = old + 0.3 * torch.randn(T, generator=gen, device="cuda")
    reference = old + 0.2 * torch.randn(T, generator=gen, device="cuda")
    adv = torch.randn(T, generator=gen, device="cuda")
    # Gradients are sums of a few hundred terms in fp32 with library products between: a relative
    # 2^-24 of each, some dozens deep, so 1e-5 of the norm holds them with room; a wrong term shows
    # at 1 / 600 and above.
    tol = 1e-5

    logits, r = forward(p, prompt, mask, bias)
    loss = stf.policy_loss(logits, drawn, old, adv, ref_logprobs=reference, mask=mask, kl_weight=0.1)
    (loss.loss + 0.05 * r.loss).backward()
    z, balance = plain_forward(q, prompt, mask, r.experts, r.counts, r.rows)
    lp = torch.log_softmax(z, 1).gather(1, drawn[:, None])[:, 0]
    ratio, a, k = torch.exp(lp - old.double()), adv.double(), reference.double() - lp
    terms = -torch.minimum(ratio * a, ratio.clamp(0.8, 1.2) * a) + 0.1 * (torch.expm1(k) - k)
    want = terms[mask].mean()
    assert abs(float(loss.loss) - float(want)) < 1e-5 and abs(float(r.loss) - float(balance)) < 1e-5
    (want + 0.05 * balance).backward()
    check_gradients(p, q, tol)

    for v in (*p.values(), *q.values()):
        v.grad = None
    offsets = torch.tensor([0, 100, 260, 300, 301, 450, 600], device="cuda")
    logits, r = forward(p, prompt, mask, bias)
    loss = stf.preference_loss(logits, drawn, offsets, reference, mask, beta=0.3, smoothing=0.1)
    loss.loss.backward()
    z, _ = plain_forward(q, prompt, mask, r.experts, r.counts, r.rows)
    gap = (torch.log_softmax(z, 1).gather(1, drawn[:, None])[:, 0] - reference.double()) * mask
    d = torch.stack([gap[offsets[i]:offsets[i + 1]].sum() for i in range(6)])
    m = 0.3 * (d[:3] - d[3:])
    want = -(0.9 * torch.nn.functional.logsigmoid(m) + 0.1 * torch.nn.functional.logsigmoid(-m)).mean()
    assert abs(float(loss.loss) - float(want)) < 1e-5 * max(1.0, float(want))
    want.backward()
    check_gradients(p, q, tol)
