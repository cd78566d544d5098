"""Losses on log-probabilities, on one GB300: the clipped policy loss with a KL
term (over tokens, or from rows of logits with the logits' gradient) and the
loss over pairs of sequences.

The same thin binding as the other operators': arguments are checked and passed
on, every computation is a kernel of libseqsum.so.  Streams, given results and
devices are as theirs.  Vectors of tokens are contiguous float32 tensors.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import SeqsumError, lib
from .operators import _call, _gradient, _logits, _new, _no_tangents, _other, _output, _vector

_SCRATCH = 49152           # SEQSUM_POLICY_SCRATCH
_NO_SCRATCH = 65536        # tokens that need none
_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}


class _Policy(ctypes.Structure):
    _fields_ = [("clip_low", ctypes.c_double), ("clip_high", ctypes.c_double), ("max_ratio", ctypes.c_double),
                ("kl_coef", ctypes.c_double), ("entropy_coef", ctypes.c_double), ("temperature", ctypes.c_double),
                ("old_logps", ctypes.c_void_p), ("advantages", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("ref_logps", ctypes.c_void_p)]


class _Preference(ctypes.Structure):
    _fields_ = [("beta", ctypes.c_double), ("margin", ctypes.c_double), ("smoothing", ctypes.c_double),
                ("kind", ctypes.c_int32), ("average", ctypes.c_int32)]


_lib = None


def _entries():
    """The library, with the argument types of the entries that this module calls."""
    global _lib
    if _lib is not None:
        return _lib
    L = lib()
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    policy, preference = ctypes.POINTER(_Policy), ctypes.POINTER(_Preference)
    for name, args in (("policy_loss", [vp, i64, policy, vp, vp, vp, vp, vp]),
                       ("policy_loss_backward", [vp, i64, policy, vp, vp, vp]),
                       ("token_policy_grad", [vp, i32, i64, i64, i64, vp, policy, vp, i64, vp, vp, vp, vp, vp, vp]),
                       ("preference_loss", [vp, vp, vp, i64, vp, i64, preference, vp, vp, vp, vp, vp, vp]),
                       ("preference_backward", [vp, i64, vp, i64, vp, vp, vp, vp])):
        fn = getattr(L, "seqsum_" + name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    _lib = L
    return L


def _tokens(t, name):
    """The number of entries and the device index of a vector of one float32 a token."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is torch.float32 and t.dim() == 1 and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous 1-D CUDA tensor of torch.float32")
    return t.shape[0], t.get_device()


def _constant(**named):
    """Refuses tensors that would get no gradient although they ask for one."""
    for name, t in named.items():
        if t is not None and getattr(t, "requires_grad", False) and torch.is_grad_enabled():
            raise SeqsumError(f"seqsum: there is no gradient into {name} (detach it)")


def _recorded(x, given, stream, what):
    """Whether autograd records a call on x; refuses what it then cannot have."""
    if not (isinstance(x, torch.Tensor) and x.requires_grad and torch.is_grad_enabled()):
        return False
    if any(g is not None for g in given) or (stream is not None and _other(stream, x.device) is not None):
        raise SeqsumError(f"seqsum: {what} that require a gradient go with new results on the current stream (or detach them)")
    return True


def _policy(n, index, old_logps, advantages, weights, ref_logps, settings):
    """The settings and the vectors beside n tokens, as the library takes them."""
    clip_low, clip_high, max_ratio, kl_coef, entropy_coef, temperature = settings
    if not (0 <= clip_low <= 1 and clip_high >= 0 and max_ratio >= 1 and -1e30 <= kl_coef <= 1e30
            and -1e30 <= entropy_coef <= 1e30 and 1e-30 <= temperature <= 1e30):
        raise ValueError("clip_low must be in [0, 1], clip_high at least 0, max_ratio at least 1, kl_coef and entropy_coef "
                         "finite, temperature above 0")
    f = torch.float32
    return _Policy(clip_low, clip_high, max_ratio, kl_coef, entropy_coef, temperature,
                   _vector(old_logps, "old_logps", n, f, index), _vector(advantages, "advantages", n, f, index),
                   _vector(weights, "weights", n, f, index),
                   None if ref_logps is None else _vector(ref_logps, "ref_logps", n, f, index))


def _result(t, name, n, like, index, stream):
    """A given float32 result, checked, or a new one beside `like`: the tensor and its address."""
    if t is None and stream is None:
        t = torch.empty(n, dtype=torch.float32, device=like.device)
        return t, t.data_ptr()
    return _output(t, name, n, torch.float32, index, like, stream)


def _scratch(n, like, stream):
    """Memory for the sums of many tokens, and its address."""
    if n <= _NO_SCRATCH:
        return None, None
    t = _new(_SCRATCH // 8, torch.float64, like, stream)
    return t, t.data_ptr()


def _overlap(names, written, in_place, used):
    """After a refusal: names a result, of the first `written` of the tensors `used`, that lies in the memory of another
    of them, if there is one (out may be the tensor called `in_place`)."""
    spans = []
    for name, t in zip(names, used):
        first = last = 0
        if t is not None and t.numel() > 0:
            first = t.data_ptr()
            last = first + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))
        spans.append((name, first, last))
    for name, first, last in spans[:written]:
        for other, start, end in spans:
            if other != name and first < end and start < last and not (
                    name == "out" and other == in_place and (first, last) == (start, end)):
                raise ValueError(f"{name} and {other} are the same memory, or overlap") from None


def policy_loss(logps, old_logps, advantages, weights, ref_logps=None, clip_low=0.2, clip_high=0.2, max_ratio=math.inf,
                kl_coef=0.0, loss=None, stats=None, stream=None):
    """(loss, stats), float32: the clipped policy loss over tokens from their
    log-probabilities `logps`, those under the policy that drew the tokens
    (`old_logps`), advantages and weights, all of one entry a token.

    With r = exp(logp - old) and A the advantage a token's loss is
    -min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A), at most -max_ratio A
    where A < 0, and kl_coef times exp(ref - logp) - (ref - logp) - 1 where
    ref_logps are given.  `loss` (1 entry) is the sum of the weights times that:
    weights of 1 / tokens give the mean over tokens, 1 / (sequences * the
    sequence's tokens) the mean over sequences; a token of weight 0 is unused
    and nothing beside it is looked at.  `stats` has the sums of the weights times:
    the first term, the KL term, 0, 1 where the ratio is past its bound,
    (r - 1) - (logp - old), 1.

    Where autograd records and logps require a gradient, loss has one.  There is
    none through stats or into the other tensors, and none into given results or
    on another stream than the current one; tensors with a forward-mode tangent
    are refused."""
    settings = (clip_low, clip_high, max_ratio, kl_coef, 0.0, 1.0)
    _no_tangents(logps=logps, old_logps=old_logps, advantages=advantages, weights=weights, ref_logps=ref_logps)
    _constant(old_logps=old_logps, advantages=advantages, weights=weights, ref_logps=ref_logps)
    if _recorded(logps, (loss, stats), stream, "logps"):
        return _PolicyLoss.apply(logps, old_logps, advantages, weights, ref_logps, settings)
    return _policy_loss(logps, old_logps, advantages, weights, ref_logps, settings, None, loss, stats, stream)[1:]


def policy_loss_grad(logps, old_logps, advantages, weights, ref_logps=None, clip_low=0.2, clip_high=0.2,
                     max_ratio=math.inf, kl_coef=0.0, out=None, loss=None, stats=None, stream=None):
    """(dlogps, loss, stats): policy_loss and, from the same read, the gradient
    of the loss with respect to logps.  `out` may be logps.  The results have no
    history."""
    settings = (clip_low, clip_high, max_ratio, kl_coef, 0.0, 1.0)
    return _policy_loss(logps, old_logps, advantages, weights, ref_logps, settings, out, loss, stats, stream, True)


def _policy_loss(logps, old_logps, advantages, weights, ref_logps, settings, out, loss, stats, stream, grad=False):
    n, index = _tokens(logps, "logps")
    p = _policy(n, index, old_logps, advantages, weights, ref_logps, settings)
    dp = None
    if grad:
        out, dp = _result(out, "out", n, logps, index, stream)
    loss, lp = _result(loss, "loss", 1, logps, index, stream)
    stats, sp = _result(stats, "stats", 6, logps, index, stream)
    scratch, tp = _scratch(n, logps, stream)
    used = out, loss, stats, scratch, logps, old_logps, advantages, weights, ref_logps
    try:
        _call(index, stream, used, _entries().seqsum_policy_loss, logps.data_ptr(), n, p, dp, lp, sp, tp)
    except SeqsumError:
        _overlap(("out", "loss", "stats", "scratch", "logps", "old_logps", "advantages", "weights", "ref_logps"), 4, "logps", used)
        raise
    return out, loss, stats


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logps, old_logps, advantages, weights, ref_logps, settings):
        _, loss, stats = _policy_loss(logps, old_logps, advantages, weights, ref_logps, settings, None, None, None, None)
        ctx.save_for_backward(logps, old_logps, advantages, weights, ref_logps)
        ctx.settings = settings
        ctx.mark_non_differentiable(stats)
        ctx.set_materialize_grads(False)
        return loss, stats

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss, _):
        if dloss is None:
            return (None,) * 6
        logps, old_logps, advantages, weights, ref_logps = ctx.saved_tensors
        n, index = _tokens(logps, "logps")
        p = _policy(n, index, old_logps, advantages, weights, ref_logps, ctx.settings)
        dlogps = torch.empty_like(logps)
        dloss = dloss.contiguous()
        _call(index, None, (), _entries().seqsum_policy_loss_backward, logps.data_ptr(), n, p, dloss.data_ptr(),
              dlogps.data_ptr())
        return dlogps, None, None, None, None, None


def token_policy_grad(logits, tokens, old_logps, advantages, weights, ref_logps=None, clip_low=0.2, clip_high=0.2,
                      max_ratio=math.inf, kl_coef=0.0, entropy_coef=0.0, temperature=1.0, out=None, loss=None, stats=None,
                      logps=None, entropies=None, stream=None):
    """(dlogits, loss, stats, logps, entropies): the policy loss of the tokens of
    rows of `logits` (rows x vocab), with an entropy bonus, and its gradient with
    respect to the logits from the same read of them.

    A row's token has its log-probability and the row its entropy under
    softmax(logits / temperature); the loss is policy_loss's minus entropy_coef
    times the entropy, and stats[2] the sum of the weights times the entropies.  A
    row of weight 0, or whose token is outside [0, vocab), is unused: it is not
    read, and its gradient, logp and entropy are 0.  `out` may be the logits, or
    rows of the logits' stride beside them (a padded buffer's, say: rows of another
    alignment are written number by number, at a third of the speed).  The results
    have no history: the gradient is there already, for logits.backward(dlogits) say."""
    rows, vocab, stride, dtype, index = _logits(logits)
    p = _policy(rows, index, old_logps, advantages, weights, ref_logps,
                (clip_low, clip_high, max_ratio, kl_coef, entropy_coef, temperature))
    tp = _vector(tokens, "tokens", rows, torch.int64, index)
    out, ostride = _gradient(out, logits, stream)
    loss, lp = _result(loss, "loss", 1, logits, index, stream)
    stats, sp = _result(stats, "stats", 6, logits, index, stream)
    logps, gp = _result(logps, "logps", rows, logits, index, stream)
    entropies, ep = _result(entropies, "entropies", rows, logits, index, stream)
    scratch, cp = _scratch(rows, logits, stream)
    used = out, loss, stats, logps, entropies, scratch, logits, tokens, old_logps, advantages, weights, ref_logps
    try:
        _call(index, stream, used, _entries().seqsum_token_policy_grad, logits.data_ptr(), dtype, rows, vocab, stride, tp, p,
              out.data_ptr(), ostride, gp, ep, lp, sp, cp)
    except SeqsumError:
        _overlap(("out", "loss", "stats", "logps", "entropies", "scratch", "logits", "tokens", "old_logps", "advantages",
                  "weights", "ref_logps"), 6, "logits", used)
        raise
    return out, loss, stats, logps, entropies


def preference_loss(logps, offsets, ref_logps=None, weights=None, kind="sigmoid", beta=0.1, margin=0.0, smoothing=0.0,
                    average=False, loss=None, scores=None, stream=None):
    """(loss, scores), float32: the loss over pairs of sequences, of which the
    first is preferred, from their tokens' log-probabilities.

    offsets    int64, 2 * pairs + 1 entries in order: sequence i is the tokens
               [offsets[i], offsets[i + 1]); pair p is sequences 2p (chosen) and
               2p + 1 (rejected)
    ref_logps  the tokens' log-probabilities under a reference, or None (0)
    weights    one a token (0: unused, nothing beside it is looked at), or None (1)
    A sequence's score is the sum of weight * (logp - ref) over its tokens, with
    `average` divided by the sum of the weights.  With D the difference of a
    pair's scores and z = beta * D - margin, a pair's loss is
      "sigmoid"  (1 - smoothing) * softplus(-z) + smoothing * softplus(z)
      "hinge"    max(0, 1 - z)
      "ipo"      (D - 1 / (2 * beta)) ** 2
    and `loss` (1 entry) the mean.  Offsets out of order or range make it NaN.

    Where autograd records and logps require a gradient, loss has one.  There is
    none through scores or into the other tensors, and none into given results or
    on another stream than the current one; tensors with a forward-mode tangent
    are refused."""
    settings = _preference(kind, beta, margin, smoothing, average)
    _no_tangents(logps=logps, ref_logps=ref_logps, weights=weights)
    _constant(ref_logps=ref_logps, weights=weights)
    if _recorded(logps, (loss, scores), stream, "logps"):
        return _PreferenceLoss.apply(logps, offsets, ref_logps, weights, settings)
    return _preference_loss(logps, offsets, ref_logps, weights, settings, None, loss, scores, stream)[1:3]


def preference_loss_grad(logps, offsets, ref_logps=None, weights=None, kind="sigmoid", beta=0.1, margin=0.0, smoothing=0.0,
                         average=False, out=None, loss=None, scores=None, stream=None):
    """(dlogps, loss, scores): preference_loss and the gradient of the loss with
    respect to logps, 0 for tokens of no sequence.  `out` may be logps.  The
    results have no history."""
    settings = _preference(kind, beta, margin, smoothing, average)
    return _preference_loss(logps, offsets, ref_logps, weights, settings, out, loss, scores, stream, True)[:3]


def _preference(kind, beta, margin, smoothing, average):
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {', '.join(_KINDS)}")
    if not 1e-30 <= beta <= 1e30:
        raise ValueError("beta must be above 0")
    if not abs(margin) <= 1e30 or (margin != 0 and kind == "ipo"):
        raise ValueError("margin must be finite, and goes with sigmoid and hinge")
    if not 0 <= smoothing <= 1 or (smoothing != 0 and kind != "sigmoid"):
        raise ValueError("smoothing must be in [0, 1], and goes with sigmoid")
    return _Preference(beta, margin, smoothing, _KINDS[kind], bool(average))


def _offsets(offsets, index):
    """The number of pairs, and the address."""
    if not (isinstance(offsets, torch.Tensor) and offsets.dtype is torch.int64 and offsets.get_device() == index
            and offsets.dim() == 1 and offsets.is_contiguous() and offsets.shape[0] % 2 == 1):
        raise TypeError(f"offsets must be a contiguous torch.int64 tensor of 2 * pairs + 1 entries on cuda:{index}")
    return offsets.shape[0] // 2, offsets.data_ptr()


def _preference_loss(logps, offsets, ref_logps, weights, settings, out, loss, scores, stream, grad=False):
    n, index = _tokens(logps, "logps")
    f = torch.float32
    dp = None
    pairs, op = _offsets(offsets, index)
    rp = None if ref_logps is None else _vector(ref_logps, "ref_logps", n, f, index)
    wp = None if weights is None else _vector(weights, "weights", n, f, index)
    if grad:
        out, dp = _result(out, "out", n, logps, index, stream)
    loss, lp = _result(loss, "loss", 1, logps, index, stream)
    scores, sp = _result(scores, "scores", 2 * pairs, logps, index, stream)
    each = _new(3 * pairs, f, logps, stream)    # the sequences' slopes, the pairs' losses
    ep = each.data_ptr()
    used = out, loss, scores, each, logps, offsets, ref_logps, weights
    try:
        _call(index, stream, used, _entries().seqsum_preference_loss, logps.data_ptr(), rp, wp, n, op, pairs, settings, dp, lp,
              sp, ep, ep + 8 * pairs)
    except SeqsumError:
        _overlap(("out", "loss", "scores", "each", "logps", "offsets", "ref_logps", "weights"), 4, "logps", used)
        raise
    return out, loss, scores, each


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logps, offsets, ref_logps, weights, settings):
        _, loss, scores, each = _preference_loss(logps, offsets, ref_logps, weights, settings, None, None, None, None)
        ctx.save_for_backward(offsets, weights, each)
        ctx.n = logps.shape[0]
        ctx.mark_non_differentiable(scores)
        ctx.set_materialize_grads(False)
        return loss, scores

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss, _):
        if dloss is None:
            return (None,) * 5
        offsets, weights, each = ctx.saved_tensors
        index, pairs = each.get_device(), each.shape[0] // 3
        op = _vector(offsets, "offsets", 2 * pairs + 1, torch.int64, index)
        wp = None if weights is None else _vector(weights, "weights", ctx.n, torch.float32, index)
        dlogps = torch.empty(ctx.n, dtype=torch.float32, device=each.device)
        dloss = dloss.contiguous()
        _call(index, None, (), _entries().seqsum_preference_backward, wp, ctx.n, op, pairs, each.data_ptr(),
              dloss.data_ptr(), dlogps.data_ptr())
        return dlogps, None, None, None, None
