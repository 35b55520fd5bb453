"""Language-model operators over rows of logits: thin binding, like the top-k's.

  sample_tokens      a token per row: temperature, top-k, top-p, min-p, given uniform numbers
  route_tokens       the k experts of a token, gate weights, per-expert counts, balance loss
  balance_loss       the balance loss and counts of a choice made elsewhere
  token_logprobs     the log-probabilities of given tokens
  policy_loss        the clipped policy loss of drawn tokens, with a KL term
  preference_loss    the loss of pairs of sequences, by their log ratios to a reference
  *_grad             their gradients with respect to the logits

Formulas, ties, empty rows and limits: include/profk.h.  Every call is enqueued on the
current stream of the logits' device and waits for nothing; outputs and scratch come from
torch's allocator, so calls may be captured into a graph without a first call.
All but sample_tokens are differentiable (backward, once) with respect to the logits, where
those require a gradient; a forward-mode tangent is refused.  Their other inputs, sample_tokens'
results and the gradients by name are constants to autograd.

The checks of arguments, the outputs and the library's call are one compiled step
(csrc/operators_binding.cpp): a call takes 3 to 60 us on the GPU, and from Python the same
steps took 9 to 15 us.  There is no other path when it has not been built.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import sampling_threshold_filtering_amd as _profk


class Sampling(ctypes.Structure):
    """profk_sampling"""
    _fields_ = [
        ("temperature", ctypes.c_float), ("top_p", ctypes.c_float), ("min_p", ctypes.c_float),
        ("reserved", ctypes.c_int32), ("top_k", ctypes.c_int64),
        ("row_temperature", ctypes.c_void_p), ("row_top_k", ctypes.c_void_p), ("row_top_p", ctypes.c_void_p),
        ("row_min_p", ctypes.c_void_p),
    ]


class ScoringSettings(ctypes.Structure):
    """profk_scoring"""
    _fields_ = [
        ("scores", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
        ("group_best", ctypes.c_int32), ("scale", ctypes.c_float), ("normalize", ctypes.c_int32), ("bias", ctypes.c_void_p),
    ]


class PolicySettings(ctypes.Structure):
    """profk_policy"""
    _fields_ = [
        ("old_logprobs", ctypes.c_void_p), ("advantages", ctypes.c_void_p), ("ref_logprobs", ctypes.c_void_p),
        ("weights", ctypes.c_void_p), ("clip_low", ctypes.c_double), ("clip_high", ctypes.c_double),
        ("kl_weight", ctypes.c_double),
    ]


class PreferenceSettings(ctypes.Structure):
    """profk_preference"""
    _fields_ = [
        ("offsets", ctypes.c_void_p), ("ref_logprobs", ctypes.c_void_p), ("pairs", ctypes.c_int64),
        ("beta", ctypes.c_double), ("smoothing", ctypes.c_double), ("margin", ctypes.c_double), ("average", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class Routing(NamedTuple):
    """weights [T, k] float32, experts [T, k] int64 (-1: none), counts [E] int64, rows int64
    (the live rows), loss float32 or None."""
    weights: object
    experts: object
    counts: object
    rows: object
    loss: Optional[object]


class Balance(NamedTuple):
    """loss float32, counts [E] int64, rows int64 (the live rows), k (slots per row)."""
    loss: object
    counts: object
    rows: object
    k: int


class PolicyLoss(NamedTuple):
    """loss float32, logprobs [T] float32, kl float32 (the weighted sum of e^q - 1 - q), clipped
    int64 (live rows whose ratio is clipped), rows int64 (the live rows)."""
    loss: object
    logprobs: object
    kl: object
    clipped: object
    rows: object


class PreferenceLoss(NamedTuple):
    """loss float32, margins [pairs] float32, sequence_logprobs [2 * pairs] float32, rows int64
    (the live rows), logprobs [T] float32, coefficients [T] float32 (dloss / dlogprobs)."""
    loss: object
    margins: object
    sequence_logprobs: object
    rows: object
    logprobs: object
    coefficients: object


# set together, at first use; the last two are looked up once (0.1 us each time)
_module = _torch = _stream = _device = None


def _native():
    global _module, _torch, _stream, _device
    if _module is None:
        _profk.load_library()
        import torch  # the compiled step uses its libraries
        try:
            from sampling_threshold_filtering_amd import _operators
        except ImportError as e:
            raise ImportError("the operators' binding is missing: build it with "
                              "`python -m sampling_threshold_filtering_amd.build_native`") from e
        _torch = torch
        _stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or functools.partial(_profk._raw_stream, torch)
        _device = getattr(torch._C, "_cuda_getDevice", None) or functools.partial(_profk._current_device, torch)
        _module = _operators
    return _module


def _check_device(torch, x):
    if not (isinstance(x, torch.Tensor) and x.is_cuda):
        raise ValueError("logits must be a 2-D float32, float16 or bfloat16 device tensor")


def _call(x, fn, *args):
    """fn(*args, the current stream of x's device); raises ProfkError for a status"""
    torch = _torch
    if not (isinstance(x, torch.Tensor) and x.is_cuda):
        _check_device(torch, x)
    di = x.get_device()
    if di == _device():
        r = fn(*args, _stream(di))
    else:
        with torch.cuda.device(di):
            r = fn(*args, _stream(di))
    if r.__class__ is int:
        _profk._check(r)
    return r


def sample_tokens(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None):
    """One token per row of logits [B, V] (fp32, fp16 or bf16; rows may be strided) from
    uniform numbers u [B] float32 in [0, 1): (tokens int64 [B], logprobs float32 [B]).

    Applied in this order: temperature, top_k, top_p, min_p, each a number or a tensor of
    B values.  temperature 0 is greedy; top_k 0, top_p 1 and min_p 0 are off.  The token is
    the quantile u of what is left, counted from the likeliest down (u = 0: the likeliest;
    ties to the lower index); its logprob is of that renormalised distribution.  A row with
    no entry above -inf, or with a NaN, gives token -1.  The log-probabilities are constants:
    no gradient reaches the logits.  `out=(tokens, logprobs)` reuses caller buffers."""
    return _call(logits, (_module or _native()).sample, logits, u, temperature, top_k, top_p, min_p, out)


def _route(logits, k, normalize, mask, balance, scores, bias, groups, top_groups, group_best, scale):
    module = _module or _native()
    # (Routing._make does this too, in 0.3 us more)
    if scores == "softmax" and bias is None and scale == 1.0 and (top_groups is None or top_groups == groups) \
            and groups == 1 and group_best in (1, 2):
        return tuple.__new__(Routing, _call(logits, module.route, logits, k, normalize, mask, balance))
    return tuple.__new__(Routing, _call(logits, module.scored, logits, k, normalize, mask, balance, scores, bias, groups,
                                        top_groups, group_best, scale))


def route_tokens(logits, k: int, normalize: bool = True, mask=None, balance: bool = False, scores: str = "softmax",
                 bias=None, groups: int = 1, top_groups: Optional[int] = None, group_best: int = 2,
                 scale: float = 1.0) -> Routing:
    """The k experts of each token from router logits [T, E] (fp32, fp16 or bf16; rows may be
    strided): a Routing.  Experts by logit, descending, ties to the lower index; gate weights
    are the softmax's, divided by the chosen ones' sum with `normalize`.  Tokens whose `mask`
    ([T] bool) is False, and rows of -inf alone, get expert -1 and weight 0 and count nowhere;
    a logit of -inf is never chosen.  With `balance`, loss = E sum_e f_e P_e with f_e the share
    of slots that expert e got and P_e its mean probability.  weights and loss are
    differentiable with respect to the logits (the choice and the counts are constants).

    Routing by scores: `scores` "sigmoid" takes s = sigmoid(logit) in place of the softmax (its
    probability is then s / sum s).  The choice is by s + `bias` ([E] float32, a constant), ties
    to the lower index.  With `top_groups` of `groups` (equal groups of neighbours), a group's
    score is the sum of its `group_best` (1 or 2) largest of those, and only the best groups'
    experts are chosen from.  The gate weights are s, with `normalize` over the chosen ones' sum,
    times `scale`; the bias is not among them.  An expert of bias -inf is never chosen."""
    if logits.requires_grad:
        import torch
        if torch.is_grad_enabled():
            return _route_function().route(logits, k, normalize, mask, balance, scores, bias, groups, top_groups,
                                           group_best, scale)
    return _route(logits, k, normalize, mask, balance, scores, bias, groups, top_groups, group_best, scale)


def route_tokens_grad(logits, routing: Routing, d_weights=None, d_loss=None, normalize: bool = True, mask=None,
                      scores: str = "softmax", scale: float = 1.0):
    """The gradient with respect to the logits (their type, contiguous) of a scalar whose
    gradients are d_weights [T, k] float32 and d_loss (a number or one float32 value) with
    respect to route_tokens' weights and loss; either may be None.  The other arguments are
    those of the call that gave `routing`."""
    if d_weights is None and d_loss is None:
        import torch
        _check_device(torch, logits)
        return torch.zeros(logits.shape, dtype=logits.dtype, device=logits.device)
    return _call(logits, (_module or _native()).route_grad, logits, routing.experts, routing.counts, routing.rows,
                 d_weights, d_loss, normalize, mask, scores, scale)


def _balance(logits, experts, mask):
    loss, counts, rows = _call(logits, (_module or _native()).balance, logits, experts, mask)
    return Balance(loss, counts, rows, experts.shape[1])


def balance_loss(logits, experts, mask=None) -> Balance:
    """route_tokens' balance loss and per-expert counts for a choice made elsewhere: experts
    [T, k] int64, entries outside [0, E) dropped slots.  The loss is differentiable with
    respect to the logits."""
    if logits.requires_grad:
        import torch
        if torch.is_grad_enabled():
            return _route_function().balance(logits, experts, mask)
    return _balance(logits, experts, mask)


def balance_loss_grad(logits, balance: Balance, d_loss=1.0, mask=None):
    """The gradient with respect to the logits (their type, contiguous) of a scalar whose
    gradient with respect to balance_loss' loss is d_loss (a number or one float32 value)."""
    return _call(logits, (_module or _native()).balance_grad, logits, balance.k, balance.counts, balance.rows, d_loss,
                 mask)


def token_logprobs(logits, tokens, mask=None, temperature=1.0):
    """The log-probability [T] float32 of each row's token (tokens [T] int64) under the softmax
    of logits [T, V] / temperature (fp32, fp16 or bf16; rows may be strided).  Rows whose `mask`
    ([T] bool) is False or whose token is outside [0, V) give 0; a token whose logit is -inf
    gives -inf, a row with a NaN or +inf NaN.  Differentiable with respect to the logits."""
    if logits.requires_grad:
        import torch
        if torch.is_grad_enabled():
            return _loss_functions().logprobs(logits, tokens, mask, temperature)
    return _call(logits, (_module or _native()).token_logprobs, logits, tokens, mask, temperature)


def token_logprobs_grad(logits, tokens, d_logprobs, mask=None, temperature=1.0, d_loss=1.0):
    """The gradient with respect to the logits (their type, contiguous) of a scalar whose
    gradients with respect to token_logprobs' result are d_loss (a number or one float32 value)
    times d_logprobs [T] float32.  A row of d_logprobs 0 and one whose token has logit -inf get
    0.  One pass over the logits; the forward pass need not have run."""
    return _call(logits, (_module or _native()).token_logprobs_grad, logits, tokens, d_logprobs, d_loss, mask, temperature)


def _policy(logits, tokens, old_logprobs, advantages, ref_logprobs, weights, mask, clip_low, clip_high, kl_weight,
            temperature, d_loss):
    return _call(logits, (_module or _native()).policy, logits, tokens, old_logprobs, advantages, ref_logprobs, weights,
                 mask, clip_low, clip_high, kl_weight, temperature, d_loss)


def policy_loss(logits, tokens, old_logprobs, advantages, ref_logprobs=None, weights=None, mask=None, clip_low=0.2,
                clip_high=0.2, kl_weight=0.0, temperature=1.0) -> PolicyLoss:
    """The clipped policy loss of tokens [T] int64 that a policy of log-probabilities
    old_logprobs drew, under logits [T, V] / temperature: a PolicyLoss.  With r = exp(logprob -
    old), advantage A and q = ref - logprob, its loss is the sum over live rows of
      weight (-min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_weight (e^q - 1 - q))
    with weights [T], or 1 / (the number of live rows) without them; no last term without
    ref_logprobs.  The values per row are float32.  Rows whose `mask` ([T] bool) is False or
    whose token is outside [0, V) take no part; a token whose logit is -inf adds nothing.  Only
    loss is differentiable, and only with respect to the logits."""
    if logits.requires_grad:
        import torch
        if torch.is_grad_enabled():
            return _loss_functions().policy(logits, tokens, old_logprobs, advantages, ref_logprobs, weights, mask,
                                            clip_low, clip_high, kl_weight, temperature)
    return PolicyLoss(*_policy(logits, tokens, old_logprobs, advantages, ref_logprobs, weights, mask, clip_low,
                               clip_high, kl_weight, temperature, None)[:5])


def policy_loss_and_grad(logits, tokens, old_logprobs, advantages, ref_logprobs=None, weights=None, mask=None,
                         clip_low=0.2, clip_high=0.2, kl_weight=0.0, temperature=1.0, d_loss=1.0):
    """(policy_loss of the same arguments, its gradient with respect to the logits) in one pass:
    the gradient (the logits' type, contiguous) of a scalar whose gradient with respect to the
    loss is d_loss, a number or one float32 value."""
    if d_loss is None:
        raise ValueError("d_loss must be a number or one float32 value")
    r = _policy(logits, tokens, old_logprobs, advantages, ref_logprobs, weights, mask, clip_low, clip_high, kl_weight,
                temperature, d_loss)
    return PolicyLoss(*r[:5]), r[5]


def _preference(logits, tokens, offsets, ref_logprobs, mask, beta, smoothing, margin, average, temperature):
    return PreferenceLoss(*_call(logits, (_module or _native()).preference, logits, tokens, offsets, ref_logprobs, mask,
                                 beta, smoothing, margin, average, temperature))


def preference_loss(logits, tokens, offsets, ref_logprobs=None, mask=None, beta=0.1, smoothing=0.0, margin=0.0,
                    average=False, temperature=1.0) -> PreferenceLoss:
    """The loss of pairs of sequences, the first preferred: a PreferenceLoss.  Sequence s is rows
    offsets[s] .. offsets[s + 1] of logits [T, V] and tokens [T] (offsets [2 * pairs + 1] int64 on
    the device); pair i is sequences i and pairs + i.  With D the sum over a sequence's live rows
    of logprob - ref_logprobs [T] (`average`: the mean), z = beta (D_i - D_{pairs + i}) - margin
    and loss = mean of -(1 - smoothing) ln sigmoid(z) - smoothing ln sigmoid(-z).  Rows whose
    `mask` ([T] bool) is False or whose token is outside [0, V) take no part; a token whose logit
    is -inf adds nothing.  Only loss is differentiable, and only with respect to the logits."""
    if logits.requires_grad:
        import torch
        if torch.is_grad_enabled():
            return _loss_functions().preference(logits, tokens, offsets, ref_logprobs, mask, beta, smoothing, margin,
                                                average, temperature)
    return _preference(logits, tokens, offsets, ref_logprobs, mask, beta, smoothing, margin, average, temperature)


def preference_loss_grad(logits, tokens, preference: PreferenceLoss, d_loss=1.0, mask=None, temperature=1.0):
    """The gradient with respect to the logits (their type, contiguous) of a scalar whose
    gradient with respect to preference_loss' loss is d_loss (a number or one float32 value).
    The other arguments are those of the call that gave `preference`."""
    return token_logprobs_grad(logits, tokens, preference.coefficients, mask, temperature, d_loss)


_functions = None


def _route_function():
    """The autograd functions, made at first use so that importing the package needs no torch."""
    global _functions
    if _functions is not None:
        return _functions
    import torch

    class RouteFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, k, normalize, mask, balance, scores, bias, groups, top_groups, group_best, scale):
            r = _route(logits, k, normalize, mask, balance, scores, bias, groups, top_groups, group_best, scale)
            ctx.save_for_backward(logits, mask, r.experts, r.counts, r.rows)
            ctx.normalize, ctx.scores, ctx.scale = normalize, scores, scale
            ctx.mark_non_differentiable(r.experts, r.counts, r.rows)
            ctx.set_materialize_grads(False)
            return tuple(r)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, d_weights, d_experts, d_counts, d_rows, d_loss):
            logits, mask, experts, counts, rows = ctx.saved_tensors
            if d_weights is None and d_loss is None:
                return (None,) * 11
            r = Routing(None, experts, counts, rows, None)
            return (route_tokens_grad(logits, r, d_weights, d_loss, ctx.normalize, mask, ctx.scores, ctx.scale),) + (None,) * 10

    class BalanceFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, experts, mask):
            b = _balance(logits, experts, mask)
            ctx.save_for_backward(logits, mask, b.counts, b.rows)
            ctx.k = b.k
            ctx.mark_non_differentiable(b.counts, b.rows)
            ctx.set_materialize_grads(False)
            return b.loss, b.counts, b.rows

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, d_loss, d_counts, d_rows):
            if d_loss is None:
                return None, None, None
            logits, mask, counts, rows = ctx.saved_tensors
            return balance_loss_grad(logits, Balance(None, counts, rows, ctx.k), d_loss, mask), None, None

    class Functions:
        @staticmethod
        def route(*args):
            return Routing(*RouteFunction.apply(*args))

        @staticmethod
        def balance(logits, experts, mask):
            return Balance(*BalanceFunction.apply(logits, experts, mask), experts.shape[1])

    _functions = Functions
    return _functions


_losses = None


def _loss_functions():
    """As _route_function, of the losses over given tokens."""
    global _losses
    if _losses is not None:
        return _losses
    import torch

    class LogprobsFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, tokens, mask, temperature):
            ctx.save_for_backward(logits, tokens, mask)
            ctx.temperature = temperature
            return _call(logits, (_module or _native()).token_logprobs, logits, tokens, mask, temperature)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, d_logprobs):
            logits, tokens, mask = ctx.saved_tensors
            return token_logprobs_grad(logits, tokens, d_logprobs, mask, ctx.temperature), None, None, None

    class PolicyFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, tokens, old, advantages, ref, weights, mask, *settings):
            ctx.save_for_backward(logits, tokens, old, advantages, ref, weights, mask)
            ctx.settings = settings
            r = _policy(logits, tokens, old, advantages, ref, weights, mask, *settings, None)[:5]
            ctx.mark_non_differentiable(*r[1:])
            ctx.set_materialize_grads(False)
            return r

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, d_loss, *constants):
            if d_loss is None:
                return (None,) * 11
            # the loss again, beside the gradient: one pass over the logits either way
            return (_policy(*ctx.saved_tensors, *ctx.settings, d_loss)[5],) + (None,) * 10

    class PreferenceFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, tokens, offsets, ref, mask, *settings):
            r = _preference(logits, tokens, offsets, ref, mask, *settings)
            ctx.save_for_backward(logits, tokens, mask, r.coefficients)
            ctx.temperature = settings[-1]
            ctx.mark_non_differentiable(*r[1:])
            ctx.set_materialize_grads(False)
            return tuple(r)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, d_loss, *constants):
            if d_loss is None:
                return (None,) * 10
            logits, tokens, mask, coefficients = ctx.saved_tensors
            return (token_logprobs_grad(logits, tokens, coefficients, mask, ctx.temperature, d_loss),) + (None,) * 9

    class Functions:
        logprobs = staticmethod(LogprobsFunction.apply)

        @staticmethod
        def policy(*args):
            return PolicyLoss(*PolicyFunction.apply(*args))

        @staticmethod
        def preference(*args):
            return PreferenceLoss(*PreferenceFunction.apply(*args))

    _losses = Functions
    return _losses
