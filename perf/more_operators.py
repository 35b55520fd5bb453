"""The operators that train a policy on the tokens it drew: what is timed and what they compute.

Four operators over rows of logits, next to the sampling and the routing:
  logprobs    the log-probability of given tokens, forward or forward and gradient
  policy      the clipped policy loss with a KL term, loss and gradient
  preference  the loss of pairs of sequences (log ratios to a reference), loss and gradient
  scored      routing by softmax or sigmoid scores with a bias for balance, groups of experts and
              a scale, forward or forward and gradient
Each has a plain form here, in elementary torch operations, and a definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
CLIP_LOW, CLIP_HIGH = 0.2, 0.28
BETA = 0.1


def listed():
    return [
        # one drawn token scored; all latency
        {"name": "logprobs-one", "op": "logprobs", "T": 1, "V": 32000, "pad": 0, "dtype": "bf16", "train": False,
         "blocked": 0.0, "masked": 0.0, "temperature": 1.0},
        # a reference model's pass over a batch of answers: odd length, padded rows, 32-bit logits
        {"name": "logprobs-score", "op": "logprobs", "T": 4099, "V": 50257, "pad": 47, "dtype": "fp32", "train": False,
         "blocked": 0.0, "masked": 0.3, "temperature": 1.0},
        # a training step on given tokens, with a gradient for each log-probability
        {"name": "logprobs-train", "op": "logprobs", "T": 4096, "V": 131072, "pad": 0, "dtype": "bf16", "train": True,
         "blocked": 0.0, "masked": 0.0, "temperature": 0.8},
        # a short answer's step: few rows, so each row is several workgroups' work
        {"name": "policy-small", "op": "policy", "T": 48, "V": 32000, "pad": 0, "dtype": "bf16", "blocked": 0.0,
         "masked": 0.0, "temperature": 1.0, "kl": 0.04, "weights": False},
        # answers of a grammar that blocks a third of the vocabulary, odd length, prompts masked,
        # 16-bit floats of a short range
        {"name": "policy-ragged", "op": "policy", "T": 3001, "V": 50257, "pad": 0, "dtype": "fp16", "blocked": 0.33,
         "masked": 0.4, "temperature": 0.7, "kl": 0.04, "weights": True},
        # a large batch of long answers, every token the same share, no reference
        {"name": "policy-large", "op": "policy", "T": 8192, "V": 131072, "pad": 0, "dtype": "bf16", "blocked": 0.0,
         "masked": 0.0, "temperature": 1.0, "kl": 0.0, "weights": False},
        # two pairs of short sequences, 32-bit logits
        {"name": "preference-small", "op": "preference", "pairs": 2, "T": 150, "V": 32000, "pad": 0, "dtype": "fp32",
         "blocked": 0.0, "masked": 0.3, "average": False, "smoothing": 0.0},
        # an ordinary batch of pairs with their prompts masked, padded rows
        {"name": "preference-large", "op": "preference", "pairs": 16, "T": 12000, "V": 65536, "pad": 24,
         "dtype": "bf16", "blocked": 0.0, "masked": 0.4, "average": False, "smoothing": 0.1},
        # a decode step of a few sequences: sigmoid scores, half of the groups
        {"name": "scored-decode", "op": "scored", "T": 8, "E": 256, "k": 8, "dtype": "fp32", "train": False,
         "scores": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "best": 2, "normalize": True, "scale": 2.5,
         "masked": 0.0, "off": 0},
        # a prompt through a router of softmax scores, a group by its best expert
        {"name": "scored-prompt", "op": "scored", "T": 8192, "E": 160, "k": 6, "dtype": "bf16", "train": False,
         "scores": "softmax", "bias": False, "groups": 8, "top_groups": 3, "best": 1, "normalize": False,
         "scale": 16.0, "masked": 0.0, "off": 0},
        # a training step on padded sequences: odd sizes, two experts switched off
        {"name": "scored-ragged", "op": "scored", "T": 10007, "E": 60, "k": 4, "dtype": "fp32", "train": True,
         "scores": "softmax", "bias": True, "groups": 6, "top_groups": 3, "best": 2, "normalize": True, "scale": 1.0,
         "masked": 0.2, "off": 2},
        # a training step of a large batch over many experts
        {"name": "scored-train", "op": "scored", "T": 65536, "E": 256, "k": 8, "dtype": "bf16", "train": True,
         "scores": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "best": 2, "normalize": True, "scale": 2.5,
         "masked": 0.0, "off": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "policy", "preference", "scored"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    masked = rng.choice([0.0, rng.uniform(0.05, 0.7)])
    if op == "scored":
        groups = _log_int(rng, 1, 16)
        E = groups * _log_int(rng, 2, 512 // groups)
        top = rng.randint((groups + 2) // 3, groups)
        case = {"op": op, "T": _log_int(rng, 1, min(131072, (1 << 24) // E)), "E": E,
                "k": _log_int(rng, 1, min(E * top // groups, 16)), "dtype": dtype, "train": rng.random() < 0.6,
                "scores": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.7, "groups": groups,
                "top_groups": top, "best": rng.choice([1, 2]), "normalize": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5, 16.0]), "masked": masked,
                "off": rng.choice([0, 0, rng.randrange(E // 3 + 1)])}
        return case
    V = _log_int(rng, 512, 262144)
    case = {"op": op, "T": _log_int(rng, 4 if op == "preference" else 1, min(32768, (1 << 28) // V)), "V": V,
            "pad": rng.choice([0, 0, 1, 24, 63]), "dtype": dtype,
            "blocked": rng.choice([0.0, 0.0, rng.uniform(0.05, 0.9)]), "masked": masked}
    if op == "logprobs":
        case["train"] = rng.random() < 0.5
    if op == "policy":
        case["kl"] = rng.choice([0.0, 0.02, 0.1])
        case["weights"] = rng.random() < 0.5
    if op == "preference":
        case["pairs"] = _log_int(rng, 1, max(1, case["T"] // 4))
        case["average"] = rng.random() < 0.5
        case["smoothing"] = rng.choice([0.0, 0.1])
    else:
        case["temperature"] = rng.choice([0.6, 0.8, 1.0, 1.2])
    return case


# ---------------------------------------------------------------------------------------
# inputs

def _grad_scale(case):
    """What the loss is multiplied by in the step: 16-bit floats of a short range are trained with
    the loss scaled up, so that gradients stay normal."""
    return 64.0 * case["T"] if case["dtype"] == "fp16" else 1.0


def _draw_tokens(x, temperature, gen):
    """Tokens drawn from the rows, and their log-probabilities; a slice of rows at a time."""
    tokens, lp = [], []
    for rows in x.split(max(1, (1 << 28) // x.shape[1])):
        z = rows.float() / temperature
        noise = torch.empty_like(z).exponential_(generator=gen)
        a = (z - noise.log_()).argmax(dim=1)
        tokens.append(a)
        lp.append(z.gather(1, a.unsqueeze(1)).squeeze(1) - torch.logsumexp(z, dim=1))
    return torch.cat(tokens), torch.cat(lp)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case, "mask": None}
    T = case["T"]
    if case["op"] == "scored":
        E, k = case["E"], case["k"]
        # a router's logits: tokens differ, and some experts are liked better than others
        x = torch.randn((T, E), generator=gen, device="cuda") * 1.5 + torch.randn(E, generator=gen, device="cuda") * 0.7
        if case["off"]:
            x[:, torch.randperm(E, generator=gen, device="cuda")[:case["off"]]] = float("-inf")
        s["logits"] = x.to(dt)
        # what keeps the load even, as training leaves it
        s["bias"] = torch.randn(E, generator=gen, device="cuda") * 0.05 if case["bias"] else None
        if case["masked"] > 0:
            s["mask"] = torch.rand(T, generator=gen, device="cuda") >= case["masked"]
        if case["train"]:
            s["d_weights"] = torch.randn((T, k), generator=gen, device="cuda")
            s["d_loss"] = 0.01 * (case["T"] if case["dtype"] == "fp16" else 1)
        return s
    V = case["V"]
    # a vocabulary's logits: a body, and a few tokens per row that the context favours
    x = torch.randn((T, V), generator=gen, device="cuda").mul_(2.0)
    hot = torch.randint(0, V, (T, 24), generator=gen, device="cuda")
    x.scatter_(1, hot, 10.0 + 1.5 * x.gather(1, hot))
    if case["blocked"] > 0:  # by a grammar
        x.masked_fill_(torch.rand((T, V), generator=gen, device="cuda") < case["blocked"], float("-inf"))
    store = torch.zeros((T, V + case["pad"]), dtype=dt, device="cuda")
    store[:, :V] = x
    del x
    s["logits"] = store[:, :V]
    s["tokens"], lp = _draw_tokens(s["logits"], case.get("temperature", 1.0), gen)
    if case["op"] == "preference":
        S = 2 * case["pairs"]
        cut = torch.randint(0, T + 1, (S - 1,), generator=gen, device="cuda").sort()[0]
        end = torch.full((1,), T, device="cuda")
        s["offsets"] = torch.cat([torch.zeros_like(end), cut, end])
        if case["masked"] > 0:  # each sequence's prompt
            start, length = s["offsets"][:-1], s["offsets"].diff()
            t = torch.arange(T, device="cuda")
            of = torch.searchsorted(s["offsets"], t, right=True) - 1
            s["mask"] = t >= start[of] + (length[of] * case["masked"]).long()
        s["ref"] = lp + 0.3 * torch.randn(T, generator=gen, device="cuda")
        s["d_loss"] = _grad_scale(case)
        return s
    if case["masked"] > 0:
        s["mask"] = torch.rand(T, generator=gen, device="cuda") >= case["masked"]
    if case["op"] == "logprobs":
        if case["train"]:
            s["d_logprobs"] = torch.randn(T, generator=gen, device="cuda") / T * _grad_scale(case)
        return s
    # the policy has moved since it drew; a ratio within 32 bits of a clipping border may fall on
    # either side of it, so none is put there
    moved = 0.2 * torch.randn(T, generator=gen, device="cuda")
    for border in (math.log1p(-CLIP_LOW), math.log1p(CLIP_HIGH)):
        moved = torch.where((moved - border).abs() < 1e-4, moved + 3e-4, moved)
    s["old"] = lp - moved
    s["advantages"] = torch.randn(T, generator=gen, device="cuda")
    s["ref"] = lp + 0.3 * torch.randn(T, generator=gen, device="cuda") if case["kl"] > 0 else None
    s["weights"] = None
    if case["weights"]:  # each answer the same share, whatever its length
        length = torch.randint(20, 2000, (T,), generator=gen, device="cuda").float()
        s["weights"] = 1.0 / (length * max(1, T // 500))
    s["d_loss"] = _grad_scale(case)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---------------------------------------------------------------------------------------
# plain forms: entries in 32 bits; what there is once a row (sums of long rows, the token's own
# probability and its complement, ratios next to a border) in 64

def _rows(s, tokens, temperature):
    """exp(row - top), the rows' sums, tokens' logprobs and probabilities."""
    x = s["logits"].float()
    top = x.amax(dim=1, keepdim=True)
    e = torch.exp((x - top) / temperature)
    total = e.sum(dim=1, dtype=torch.float64)
    at = tokens.unsqueeze(1)
    lp = ((x.gather(1, at).double() - top.double()) / temperature).squeeze(1) - torch.log(total)
    return e, total, lp


def _token_grad(s, e, total, lp, c, temperature):
    """c (one at the token - p) / temperature, c a number per row in 64 bits."""
    c = c / temperature
    g = e * (-c / total).float().unsqueeze(1)
    g.scatter_(1, s["tokens"].unsqueeze(1), (c * -torch.expm1(lp)).float().unsqueeze(1))
    return g.to(s["logits"].dtype)


def _live(s):
    live = torch.ones(s["tokens"].shape, dtype=torch.bool, device=s["tokens"].device)
    return live if s["mask"] is None else s["mask"]


def _logprobs(s):
    case, live = s["case"], _live(s)
    e, total, lp = _rows(s, s["tokens"], case["temperature"])
    out = {"logprobs": torch.where(live, lp, torch.zeros_like(lp)).float()}
    if case["train"]:
        d = s["d_logprobs"].double()
        out["d_logits"] = _token_grad(s, e, total, lp, torch.where(live, d, torch.zeros_like(d)), case["temperature"])
    return out


def _policy(s):
    case, live = s["case"], _live(s)
    e, total, lp = _rows(s, s["tokens"], case["temperature"])
    n = live.sum()
    w = s["weights"].double() if s["weights"] is not None else 1.0 / n.clamp(min=1).double()
    w = torch.where(live, w, torch.zeros_like(lp))
    a = s["advantages"].double()
    r = torch.exp(lp - s["old"].double())
    cut = r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    clipped = cut * a < r * a
    loss = -torch.where(clipped, cut * a, r * a)
    c = torch.where(clipped, torch.zeros_like(r), -r * a)
    kl = torch.zeros_like(lp)
    if s["ref"] is not None:
        q = s["ref"].double() - lp
        kl = torch.expm1(q) - q
        loss = loss + case["kl"] * kl
        c = c - case["kl"] * torch.expm1(q)
    return {"loss": (w * loss).sum().float(), "kl": (w * kl).sum().float(), "clipped": (clipped & live).sum(), "rows": n,
            "logprobs": torch.where(live, lp, torch.zeros_like(lp)).float(),
            "d_logits": _token_grad(s, e, total, lp, w * c * s["d_loss"], case["temperature"])}


def _preference(s):
    case, live = s["case"], _live(s)
    P, T = case["pairs"], case["T"]
    e, total, lp = _rows(s, s["tokens"], 1.0)
    of = torch.searchsorted(s["offsets"], torch.arange(T, device=lp.device), right=True) - 1
    zero = torch.zeros(2 * P, dtype=torch.float64, device=lp.device)
    own_lp = torch.where(live, lp, torch.zeros_like(lp))
    sums = zero.scatter_add(0, of, own_lp)
    ratio = zero.scatter_add(0, of, torch.where(live, lp - s["ref"].double(), torch.zeros_like(lp)))
    length = zero.scatter_add(0, of, live.double()).clamp(min=1)
    share = 1.0 / length if case["average"] else torch.ones_like(length)
    z = BETA * (ratio[:P] * share[:P] - ratio[P:] * share[P:])
    t = case["smoothing"]
    loss = ((1 - t) * torch.logaddexp(zero[:P], -z) + t * torch.logaddexp(zero[:P], z)).mean()
    slope = BETA / P * (torch.sigmoid(z) - (1 - t))
    c = (torch.cat([slope, -slope]) * share)[of]
    c = torch.where(live, c * s["d_loss"], torch.zeros_like(c))
    return {"loss": loss.float(), "margins": z.float(), "sequence_logprobs": (sums * share).float(), "rows": live.sum(),
            "logprobs": own_lp.float(), "d_logits": _token_grad(s, e, total, lp, c, 1.0)}


def _scored(s):
    case, logits = s["case"], s["logits"]
    T, E, k, groups = case["T"], case["E"], case["k"], case["groups"]
    x = logits.double()  # in 64 bits: a choice next to a border is decided by the last bits
    there = x > float("-inf")
    live = there.any(dim=1)
    if s["mask"] is not None:
        live = live & s["mask"]
    if case["scores"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        top = torch.where(live, x.amax(dim=1), torch.zeros_like(x[:, 0])).unsqueeze(1)
        score = torch.exp(x - top)
        score = score / score.sum(dim=1, keepdim=True)
    score = torch.where(live.unsqueeze(1), score, torch.zeros_like(score))
    none = torch.full_like(score, float("-inf"))
    choice = torch.where(there, score + s["bias"].double() if s["bias"] is not None else score, none)
    if case["top_groups"] < groups:
        by_group = choice.view(T, groups, E // groups)
        best = by_group.sort(dim=2, descending=True)[0][:, :, :case["best"]]
        some = best > float("-inf")
        value = torch.where(some, best, torch.zeros_like(best)).sum(dim=2)
        value = torch.where(some.any(dim=2), value, torch.full_like(value, float("-inf")))
        order = value.sort(dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order, True)
        choice = torch.where(kept.unsqueeze(2), by_group, none.view(by_group.shape)).view(T, E)
    val, idx = choice.sort(dim=1, descending=True, stable=True)
    taken = (val[:, :k] > float("-inf")) & live.unsqueeze(1)
    at = idx[:, :k]
    experts = torch.where(taken, at, torch.full_like(at, -1))
    weights = torch.where(taken, score.gather(1, at), torch.zeros_like(val[:, :k]))
    if case["normalize"]:
        total = weights.sum(dim=1, keepdim=True)
        weights = weights / torch.where(total > 0, total, torch.ones_like(total))
    slot = torch.where(taken, at, torch.full_like(at, E)).reshape(-1)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=x.device).scatter_add_(0, slot, torch.ones_like(slot))[:E]
    rows = live.sum()
    out = {"weights": (case["scale"] * weights).float(), "experts": experts, "counts": counts, "rows": rows}
    if not case["train"]:
        return out
    n = rows.clamp(min=1).double()
    total = score.sum(dim=1, keepdim=True)
    p = score / torch.where(total > 0, total, torch.ones_like(total))
    f = counts.double() / (n * k)
    out["loss"] = (E * (f * p.sum(dim=0) / n).sum()).float()
    d = torch.where(taken, case["scale"] * s["d_weights"].double(), torch.zeros_like(weights))
    g = (s["d_loss"] * E) * p * (f - (p * f).sum(dim=1, keepdim=True)) / n
    if case["normalize"]:
        g = g.scatter_add(1, at, weights * (d - (weights * d).sum(dim=1, keepdim=True)))
    elif case["scores"] == "sigmoid":
        g = g.scatter_add(1, at, weights * d)
    else:
        g = g.scatter_add(1, at, weights * d) - p * (weights * d).sum(dim=1, keepdim=True)
    if case["scores"] == "sigmoid":
        g = g / (1.0 + torch.exp(x))
    out["d_logits"] = g.to(logits.dtype)
    return out


def run(state):
    case = state["case"]
    if not own:
        return {"logprobs": _logprobs, "policy": _policy, "preference": _preference, "scored": _scored}[case["op"]](state)
    import sampling_threshold_filtering_amd as stf
    logits, mask = state["logits"], state["mask"]
    if case["op"] == "logprobs":
        out = {"logprobs": stf.token_logprobs(logits, state["tokens"], mask=mask, temperature=case["temperature"])}
        if case["train"]:
            out["d_logits"] = stf.token_logprobs_grad(logits, state["tokens"], state["d_logprobs"], mask=mask,
                                                      temperature=case["temperature"])
        return out
    if case["op"] == "policy":
        r, d_logits = stf.policy_loss_and_grad(
            logits, state["tokens"], state["old"], state["advantages"], ref_logprobs=state["ref"],
            weights=state["weights"], mask=mask, clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_weight=case["kl"],
            temperature=case["temperature"], d_loss=state["d_loss"])
        return {"loss": r.loss, "kl": r.kl, "clipped": r.clipped, "rows": r.rows, "logprobs": r.logprobs,
                "d_logits": d_logits}
    if case["op"] == "preference":
        r = stf.preference_loss(logits, state["tokens"], state["offsets"], ref_logprobs=state["ref"], mask=mask,
                                beta=BETA, smoothing=case["smoothing"], average=case["average"])
        d_logits = stf.preference_loss_grad(logits, state["tokens"], r, d_loss=state["d_loss"], mask=mask)
        return {"loss": r.loss, "margins": r.margins, "sequence_logprobs": r.sequence_logprobs, "rows": r.rows,
                "logprobs": r.logprobs, "d_logits": d_logits}
    r = stf.route_tokens(logits, case["k"], normalize=case["normalize"], mask=mask, balance=case["train"],
                         scores=case["scores"], bias=state["bias"], groups=case["groups"],
                         top_groups=case["top_groups"], group_best=case["best"], scale=case["scale"])
    out = {"weights": r.weights, "experts": r.experts, "counts": r.counts, "rows": r.rows}
    if case["train"]:
        out["loss"] = r.loss
        out["d_logits"] = stf.route_tokens_grad(logits, r, d_weights=state["d_weights"], d_loss=state["d_loss"],
                                                normalize=case["normalize"], mask=mask, scores=case["scores"],
                                                scale=case["scale"])
    return out


# ---------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    size, T, masked = SIZE[case["dtype"]], case["T"], case["masked"]
    mask = T if masked > 0 else 0
    if case["op"] == "scored":
        E, k = case["E"], case["k"]
        # a score, its bias, one comparison for the choice and one for the group
        by, fl = T * E * size + mask + T * k * 12 + E * (12 if case["bias"] else 8), 8 * T * E
        if case["train"]:
            by += T * E * size + T * k * 4
            fl += 8 * T * E
        return {"bytes": by, "flops": fl}
    V = case["V"]
    read = int(T * (1 - masked) * V) * size  # rows that take no part need not be read
    rows = mask + T * (8 + 4)
    fl = 4 * int(T * (1 - masked) * V)  # difference, exponential, sum, maximum
    if case["op"] == "logprobs":
        if not case["train"]:
            return {"bytes": read + rows, "flops": fl}
        return {"bytes": read + rows + T * 4 + T * V * size, "flops": fl + 2 * T * V}
    if case["op"] == "policy":
        rows += T * (8 + (4 if case["kl"] > 0 else 0) + (4 if case["weights"] else 0))
    else:
        rows += T * 4 + case["pairs"] * (16 + 12)
    return {"bytes": read + rows + T * V * size, "flops": fl + 2 * T * V}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rows(s, temperature, coefficient):
    """coefficient(lp) -> a number per row; (lp, gradient or None), row by row in slices."""
    x, tokens = s["logits"], s["tokens"]
    step = max(1, (1 << 26) // x.shape[1])
    spans = [(i, min(i + step, x.shape[0])) for i in range(0, x.shape[0], step)]
    lp = torch.cat([torch.log_softmax(x[i:j].double() / temperature, dim=1)[torch.arange(j - i), tokens[i:j]]
                    for i, j in spans]).cpu()
    c = coefficient(lp)
    if c is None or x.numel() > 1 << 28:  # beyond that the gradient takes too long
        return lp, None
    grad = torch.empty(x.shape, dtype=torch.float64)
    for i, j in spans:
        # at the token: one minus its probability, as the sum of the others'
        others = torch.softmax(x[i:j].double() / temperature, dim=1)
        pick = tokens[i:j].unsqueeze(1)
        others.scatter_(1, pick, 0.0)
        rest = others.sum(dim=1, keepdim=True)
        direction = (-others).scatter_(1, pick, rest)
        grad[i:j] = (direction * (c[i:j].to(x.device) / temperature).unsqueeze(1)).cpu()
    return lp, grad


def _exact_policy(case, s):
    T = case["T"]
    live = s["mask"].cpu().numpy() if s["mask"] is not None else np.ones(T, bool)
    old, adv = s["old"].cpu().numpy().astype(np.float64), s["advantages"].cpu().numpy().astype(np.float64)
    n = int(live.sum())
    w = s["weights"].cpu().numpy().astype(np.float64) if s["weights"] is not None else np.full(T, 1 / max(n, 1))
    w = np.where(live, w, 0.0)
    out = {}

    def coefficient(lp):
        lp = lp.numpy()
        ratio = np.exp(lp - old)
        over = ((adv > 0) & (ratio > 1 + CLIP_HIGH)) | ((adv < 0) & (ratio < 1 - CLIP_LOW))
        value = -adv * np.where(over, np.where(adv > 0, 1 + CLIP_HIGH, 1 - CLIP_LOW), ratio)
        slope = np.where(over, 0.0, -adv * ratio)
        gap = np.zeros(T)
        if s["ref"] is not None:
            q = s["ref"].cpu().numpy().astype(np.float64) - lp
            gap = np.expm1(q) - q
            value, slope = value + case["kl"] * gap, slope + case["kl"] * -np.expm1(q)
        out.update(loss=torch.tensor(float(w @ value), dtype=torch.float64),
                   kl=torch.tensor(float(w @ gap), dtype=torch.float64),
                   clipped=torch.tensor(int((over & live).sum())), rows=torch.tensor(n))
        return torch.from_numpy(w * slope * s["d_loss"])

    lp, grad = _exact_rows(s, case["temperature"], coefficient)
    return {**out, "logprobs": torch.where(torch.from_numpy(live), lp, torch.zeros_like(lp)), "d_logits": grad}


def _exact_preference(case, s):
    T, P, t = case["T"], case["pairs"], case["smoothing"]
    live = s["mask"].cpu().numpy() if s["mask"] is not None else np.ones(T, bool)
    ref, offsets = s["ref"].cpu().numpy().astype(np.float64), s["offsets"].cpu().numpy()
    out = {}

    def coefficient(lp):
        lp = lp.numpy()
        sums, ratios, share = np.zeros(2 * P), np.zeros(2 * P), np.ones(2 * P)
        spans = [np.arange(offsets[i], offsets[i + 1])[live[offsets[i]:offsets[i + 1]]] for i in range(2 * P)]
        for i, rows in enumerate(spans):
            if case["average"]:
                share[i] = 1 / max(rows.size, 1)
            sums[i], ratios[i] = share[i] * lp[rows].sum(), share[i] * (lp[rows] - ref[rows]).sum()
        z = BETA * (ratios[:P] - ratios[P:])
        log_up, log_down = np.logaddexp(0, -z), np.logaddexp(0, z)  # -log of a sigmoid and of its complement
        slope = BETA / P * (t / (1 + np.exp(-z)) - (1 - t) / (1 + np.exp(z)))
        c = np.zeros(T)
        for i, rows in enumerate(spans):
            c[rows] = (slope[i] if i < P else -slope[i - P]) * share[i]
        out.update(loss=torch.tensor(float(((1 - t) * log_up + t * log_down).mean()), dtype=torch.float64),
                   margins=torch.from_numpy(z), sequence_logprobs=torch.from_numpy(sums),
                   rows=torch.tensor(int(live.sum())))
        return torch.from_numpy(c * s["d_loss"])

    lp, grad = _exact_rows(s, 1.0, coefficient)
    return {**out, "logprobs": torch.where(torch.from_numpy(live), lp, torch.zeros_like(lp)), "d_logits": grad}


def _exact_logprobs(case, s):
    live = s["mask"].cpu() if s["mask"] is not None else torch.ones(case["T"], dtype=torch.bool)
    d = torch.where(live, s["d_logprobs"].cpu().double(), torch.zeros((), dtype=torch.float64)) if case["train"] else None
    lp, grad = _exact_rows(s, case["temperature"], lambda _: d)
    out = {"logprobs": torch.where(live, lp, torch.zeros_like(lp))}
    if case["train"]:
        out["d_logits"] = grad
    return out


def _exact_scored(case, s):
    x = s["logits"].float().cpu().numpy().astype(np.float64)
    (T, E), k, groups = x.shape, case["k"], case["groups"]
    live = (x > -np.inf).any(axis=1)
    if s["mask"] is not None:
        live &= s["mask"].cpu().numpy()
    p = np.zeros_like(x)
    e = np.exp(x[live] - x[live].max(axis=1, keepdims=True, initial=-np.inf))
    p[live] = e / e.sum(axis=1, keepdims=True)
    falling = np.ones_like(x)  # ds/dx = s times this, for scores that do not depend on each other
    if case["scores"] == "sigmoid":
        with np.errstate(over="ignore"):
            score, falling = 1 / (1 + np.exp(-x)), 1 / (1 + np.exp(x))
        score[~live] = 0
        total = score.sum(axis=1, keepdims=True)
        p = np.divide(score, total, out=np.zeros_like(score), where=total > 0)
    else:
        score = p
    c = score + (s["bias"].cpu().numpy().astype(np.float64) if s["bias"] is not None else 0.0)
    c[x == -np.inf] = -np.inf
    if case["top_groups"] < groups:
        member = -np.sort(-c.reshape(T, groups, E // groups), axis=2)[:, :, :case["best"]]
        value = np.where(member > -np.inf, member, 0).sum(axis=2)
        value[member[:, :, 0] == -np.inf] = -np.inf
        left_out = np.argsort(-value, axis=1, kind="stable")[:, case["top_groups"]:]
        struck = np.zeros((T, groups), bool)
        np.put_along_axis(struck, left_out, True, axis=1)
        c[np.repeat(struck, E // groups, axis=1)] = -np.inf
    order = np.argsort(-c, axis=1, kind="stable")[:, :k]
    taken = (np.take_along_axis(c, order, axis=1) > -np.inf) & live[:, None]
    experts = np.where(taken, order, -1)
    w = np.where(taken, np.take_along_axis(score, order, axis=1), 0.0)
    if case["normalize"]:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    counts = np.bincount(order[taken], minlength=E)
    n = int(live.sum())
    out = {"weights": torch.from_numpy(case["scale"] * w), "experts": torch.from_numpy(experts),
           "counts": torch.from_numpy(counts), "rows": torch.tensor(n)}
    if not case["train"]:
        return out
    f = counts / max(n * k, 1)
    out["loss"] = torch.tensor(E * float(f @ p.sum(axis=0)) / max(n, 1), dtype=torch.float64)
    grad = s["d_loss"] * E / max(n, 1) * p * (f[None, :] - (p @ f)[:, None])
    d = np.where(taken, s["d_weights"].cpu().numpy().astype(np.float64) * case["scale"], 0.0)
    rows = np.arange(T)[:, None]
    if case["normalize"]:
        grad[rows, order] += w * (d - (w * d).sum(axis=1, keepdims=True))
    elif case["scores"] == "sigmoid":
        grad[rows, order] += w * d
    else:
        g = np.zeros_like(p)
        g[rows, order] = d
        grad += p * (g - (p * g).sum(axis=1, keepdims=True))
    out["d_logits"] = torch.from_numpy(grad * falling)
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    return {"logprobs": _exact_logprobs, "policy": _exact_policy, "preference": _exact_preference,
            "scored": _exact_scored}[case["op"]](case, s)
