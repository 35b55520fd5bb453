"""Language-model operators over rows of logits: thin binding, like the top-k's.

  sample_tokens      a token per row: temperature, top-k, top-p, min-p, given uniform numbers
  route_tokens       the k experts of a token, gate weights, per-expert counts, balance loss
  balance_loss       the balance loss and counts of a choice made elsewhere
  *_grad             their gradients with respect to the logits

Formulas, ties, empty rows and limits: include/profk.h.  Every call is enqueued on the
current stream of the logits' device and waits for nothing; outputs and scratch come from
torch's allocator, so calls may be captured into a graph without a first call.
route_tokens and balance_loss are differentiable (backward, once) where the logits require a
gradient; a forward-mode tangent is refused.  sample_tokens' results and the gradients by name
are constants to autograd.

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


def _route(logits, k, normalize, mask, balance):
    # (Routing._make does this too, in 0.3 us more)
    return tuple.__new__(Routing, _call(logits, (_module or _native()).route, logits, k, normalize, mask, balance))


def route_tokens(logits, k: int, normalize: bool = True, mask=None, balance: bool = False) -> Routing:
    """The k experts of each token from router logits [T, E] (fp32, fp16 or bf16; rows may be
    strided): a Routing.  Experts by logit, descending, ties to the lower index; gate weights
    are the softmax's, divided by the chosen ones' sum with `normalize`.  Tokens whose `mask`
    ([T] bool) is False, and rows of -inf alone, get expert -1 and weight 0 and count nowhere;
    a logit of -inf is never chosen.  With `balance`, loss = E sum_e f_e P_e with f_e the share
    of slots that expert e got and P_e its mean probability.  weights and loss are
    differentiable with respect to the logits (the choice and the counts are constants)."""
    if logits.requires_grad:
        import torch
        if torch.is_grad_enabled():
            return _route_function().route(logits, k, normalize, mask, balance)
    return _route(logits, k, normalize, mask, balance)


def route_tokens_grad(logits, routing: Routing, d_weights=None, d_loss=None, normalize: bool = True, mask=None):
    """The gradient with respect to the logits (their type, contiguous) of a scalar whose
    gradients are d_weights [T, k] float32 and d_loss (a number or one float32 value) with
    respect to route_tokens' weights and loss; either may be None.  The other arguments are
    those of the call that gave `routing`."""
    if d_weights is None and d_loss is None:
        import torch
        _check_device(torch, logits)
        return torch.zeros(logits.shape, dtype=logits.dtype, device=logits.device)
    return _call(logits, (_module or _native()).route_grad, logits, routing.experts, routing.counts, routing.rows,
                 d_weights, d_loss, normalize, mask)


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


_functions = None


def _route_function():
    """The autograd functions, made at first use so that importing the package needs no torch."""
    global _functions
    if _functions is not None:
        return _functions
    import torch

    class RouteFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, k, normalize, mask, balance):
            r = _route(logits, k, normalize, mask, balance)
            ctx.save_for_backward(logits, mask, r.experts, r.counts, r.rows)
            ctx.normalize = normalize
            ctx.mark_non_differentiable(r.experts, r.counts, r.rows)
            ctx.set_materialize_grads(False)
            return tuple(r)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, d_weights, d_experts, d_counts, d_rows, d_loss):
            logits, mask, experts, counts, rows = ctx.saved_tensors
            if d_weights is None and d_loss is None:
                return None, None, None, None, None
            r = Routing(None, experts, counts, rows, None)
            return route_tokens_grad(logits, r, d_weights, d_loss, ctx.normalize, mask), None, None, None, None

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
        def route(logits, k, normalize, mask, balance):
            return Routing(*RouteFunction.apply(logits, k, normalize, mask, balance))

        @staticmethod
        def balance(logits, experts, mask):
            return Balance(*BalanceFunction.apply(logits, experts, mask), experts.shape[1])

    _functions = Functions
    return _functions
