"""Sums that decide, on one GB300: tokens drawn from logits, their
log-probabilities and gradients, the norm of many tensors and clipping by it.

The same thin binding as the package's: arguments are checked and passed on,
every computation is a kernel of libseqsum.so.  Work is enqueued on the
current torch stream unless a stream (or its handle) is given; results are
ready once that stream reaches them.  A given stream is the caller's to order
after the work that makes the inputs, and readers of the results after it;
memory of inputs and results stays until the stream is through with it.
"""
from __future__ import annotations

import ctypes

import torch

from . import SeqsumError, _check, lib

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class _Sampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int32), ("top_p", ctypes.c_float),
                ("min_p", ctypes.c_float), ("temperatures", ctypes.c_void_p), ("top_ks", ctypes.c_void_p),
                ("top_ps", ctypes.c_void_p), ("min_ps", ctypes.c_void_p)]


class _Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("count", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


_lib = None


def _entries():
    """The library, with the argument types of the entries that this module calls."""
    global _lib
    if _lib is not None:
        return _lib
    L = lib()
    vp, i64, i32, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    rows = [vp, i32, i64, i64, i64]
    for name, args in (("sample_tokens", rows + [vp, ctypes.POINTER(_Sampling), vp, vp, vp]),
                       ("token_logprob", rows + [vp, vp, vp, vp]),
                       ("token_logprob_grad", rows + [vp, vp, vp, i64, vp, vp, vp]),
                       ("token_logprob_backward", rows + [vp, vp, vp, vp, i64, vp]),
                       ("tensors_create", [ctypes.POINTER(_Tensor), i32, ctypes.POINTER(vp)]),
                       ("tensors_norm", [vp, f, vp, vp]),
                       ("tensors_clip", [vp, f, f, vp, vp])):
        fn = getattr(L, "seqsum_" + name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    L.seqsum_tensors_destroy.argtypes, L.seqsum_tensors_destroy.restype = [vp], None
    _lib = L
    return L


# the current stream's handle without a Stream object around it, where torch has that
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)
# the current device, where CUDA has been initialised (a tensor of it is at hand)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(index, stream, used, fn, *args):
    """Calls an entry on device `index`, its last argument the stream's handle.  Where that is not the current stream,
    the memory of the tensors `used` is kept from others until the stream is through with the call."""
    if stream is None:
        handle = _current_stream(index)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        other = _other(stream, torch.device("cuda", index))
        if other is not None:
            for t in used:
                if isinstance(t, torch.Tensor):
                    t.record_stream(other)
    if index == _current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc:
        _check(rc)


def _other(stream, device):
    """`stream` as torch's, where it is given and not the current one; else None."""
    if stream is None:
        return None
    handle = int(getattr(stream, "cuda_stream", stream))
    if handle == _current_stream(device.index):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


def _new(shape, dtype, like, stream):
    """An output's memory beside `like`.  Another stream than the current one takes it from its own memory: what the
    current stream freed may still be in use there.  The current stream, which will read it, is noted."""
    if stream is not None:
        stream = _other(stream, like.device)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    current = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(current)
    return t


def _logits(x, name="logits"):
    """rows, vocab, row stride, dtype code and device index of a 2-D tensor whose rows are contiguous."""
    dtype = _DTYPES.get(x.dtype) if isinstance(x, torch.Tensor) and x.is_cuda else None
    if dtype is None or x.dim() != 2:
        raise TypeError(f"{name} must be a 2-D CUDA tensor of float32, float16 or bfloat16")
    rows, vocab = x.shape
    stride, unit = x.stride()
    if unit != 1 and vocab > 1:
        raise TypeError(f"{name} must have contiguous rows (stride 1 in the last dimension)")
    return rows, vocab, stride if rows > 1 else vocab, dtype, x.get_device()


def _vector(t, name, n, dtype, index):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.dim() == 1
            and t.shape[0] == n and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous {dtype} tensor of {n} entries on cuda:{index}")
    return t.data_ptr()


def _number(v, name):
    if v != v:
        raise ValueError(f"{name} is NaN")
    return v


# tells autograd that a given tensor is written, so that it finds saved ones that were overwritten
_written = torch.autograd.graph.increment_version


def _output(t, name, n, dtype, index, like, stream):
    """A given output, checked, or a new one: the tensor and its address."""
    if t is None:
        t = _new(n, dtype, like, stream)
        return t, t.data_ptr()
    p = _vector(t, name, n, dtype, index)
    _written(t)
    return t, p


def sample_tokens(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None, logps=None, stream=None):
    """One token a row of `logits` (rows x vocab) from the random numbers `u`
    (float32, one a row, in [0, 1)): (tokens int64, logps float32).

    Each setting is a number for all rows or a tensor of one a row
    (temperature, top_p, min_p float32, top_k int32).  temperature <= 0 is
    greedy; top_k <= 0, top_p >= 1 and min_p <= 0 are off.  The filters apply
    in the order top-k, top-p, min-p.  The sums are integers: a row's token
    does not depend on the batch it is in.  The results have no history
    (token_logprob's have)."""
    rows, vocab, stride, dtype, index = _logits(logits)
    s = _Sampling()
    if isinstance(temperature, torch.Tensor):
        s.temperatures = _vector(temperature, "temperature", rows, torch.float32, index)
    else:
        s.temperature = _number(temperature, "temperature")
    if isinstance(top_k, torch.Tensor):
        s.top_ks = _vector(top_k, "top_k", rows, torch.int32, index)
    elif top_k > 0:
        s.top_k = min(int(top_k), 2 ** 31 - 1)
    if isinstance(top_p, torch.Tensor):
        s.top_ps = _vector(top_p, "top_p", rows, torch.float32, index)
    else:
        s.top_p = _number(top_p, "top_p")
    if isinstance(min_p, torch.Tensor):
        s.min_ps = _vector(min_p, "min_p", rows, torch.float32, index)
    else:
        s.min_p = _number(min_p, "min_p")
    up = _vector(u, "u", rows, torch.float32, index)
    tokens, tp = _output(tokens, "tokens", rows, torch.int64, index, logits, stream)
    logps, lp = _output(logps, "logps", rows, torch.float32, index, logits, stream)
    _call(index, stream, (logits, u, temperature, top_k, top_p, min_p, tokens, logps), _entries().seqsum_sample_tokens,
          logits.data_ptr(), dtype, rows, vocab, stride, up, s, tp, lp)
    return tokens, logps


def token_logprob(logits, tokens, logps=None, lses=None, stream=None):
    """(logps, lses), float32: the log-probability of each row's token and the
    row's log of the sum of exponentials.  A token outside [0, vocab) marks an
    unused row: its logp is 0.

    Where autograd records and the logits require a gradient, logps has one:
    its backward pass is token_logprob_backward.  There is none through lses
    (a backward pass that needs it raises), and none into given results or on
    another stream than the current one."""
    if isinstance(logits, torch.Tensor) and logits.requires_grad and torch.is_grad_enabled():
        if logps is not None or lses is not None or _other(stream, logits.device) is not None:
            raise SeqsumError("seqsum: logits that require a gradient go with new results on the current stream "
                              "(or detach them)")
        return _TokenLogprob.apply(logits, tokens)
    return _token_logprob(logits, tokens, logps, lses, stream)


def _token_logprob(logits, tokens, logps, lses, stream):
    rows, vocab, stride, dtype, index = _logits(logits)
    tp = _vector(tokens, "tokens", rows, torch.int64, index)
    logps, lp = _output(logps, "logps", rows, torch.float32, index, logits, stream)
    lses, sp = _output(lses, "lses", rows, torch.float32, index, logits, stream)
    _call(index, stream, (logits, tokens, logps, lses), _entries().seqsum_token_logprob, logits.data_ptr(), dtype, rows,
          vocab, stride, tp, lp, sp)
    return logps, lses


class _TokenLogprob(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens):
        logps, lses = _token_logprob(logits, tokens, None, None, None)
        ctx.save_for_backward(logits, tokens, lses)
        ctx.set_materialize_grads(False)
        return logps, lses

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dlogps, dlses):
        if dlses is not None:
            raise SeqsumError("seqsum: there is no gradient through the lses of token_logprob")
        if dlogps is None:
            return None, None
        logits, tokens, lses = ctx.saved_tensors
        return token_logprob_backward(logits, tokens, dlogps.contiguous(), lses), None


def _gradient(out, logits, stream):
    """The gradient's tensor and its row stride: apart from the logits, or the logits themselves."""
    if out is None:
        rows, vocab = logits.shape
        return _new((rows, vocab), logits.dtype, logits, stream), vocab
    rows, vocab, stride, _, _ = _logits(out, "out")
    if out.shape != logits.shape or out.dtype != logits.dtype or out.device != logits.device:
        raise TypeError("out must have the logits' shape, type and device")
    if rows > 1 and stride < vocab:
        raise TypeError("out's rows overlap")
    _written(out)
    return out, stride


def token_logprob_grad(logits, tokens, dlogps, out=None, logps=None, lses=None, stream=None):
    """(dlogits, logps, lses): token_logprob and, from the same read of the
    logits, the gradient of (dlogps * logps).sum() with respect to them.
    `out` may be the logits.  The results have no history: the gradient is
    there already, for logits.backward(dlogits) say."""
    rows, vocab, stride, dtype, index = _logits(logits)
    tp = _vector(tokens, "tokens", rows, torch.int64, index)
    gp = _vector(dlogps, "dlogps", rows, torch.float32, index)
    out, ostride = _gradient(out, logits, stream)
    logps, lp = _output(logps, "logps", rows, torch.float32, index, logits, stream)
    lses, sp = _output(lses, "lses", rows, torch.float32, index, logits, stream)
    _call(index, stream, (logits, tokens, dlogps, out, logps, lses), _entries().seqsum_token_logprob_grad,
          logits.data_ptr(), dtype, rows, vocab, stride, tp, gp, out.data_ptr(), ostride, lp, sp)
    return out, logps, lses


def token_logprob_backward(logits, tokens, dlogps, lses, out=None, stream=None):
    """dlogits: the gradient of (dlogps * logps).sum() with respect to the
    logits, from the lses that token_logprob returned.  `out` may be the logits.
    It has no history."""
    rows, vocab, stride, dtype, index = _logits(logits)
    tp = _vector(tokens, "tokens", rows, torch.int64, index)
    gp = _vector(dlogps, "dlogps", rows, torch.float32, index)
    lp = _vector(lses, "lses", rows, torch.float32, index)
    out, ostride = _gradient(out, logits, stream)
    _call(index, stream, (logits, tokens, dlogps, lses, out), _entries().seqsum_token_logprob_backward,
          logits.data_ptr(), dtype, rows, vocab, stride, tp, gp, lp, out.data_ptr(), ostride)
    return out


def _dense(t):
    """Whether the tensor's numbers fill their memory without gaps or overlaps, in some order of its dimensions."""
    if t.is_contiguous():
        return True
    at = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != at:
            return False
        at *= size
    return True


class TensorList:
    """Many tensors as one: their norm, and clipping by it
    (seqsum_tensors_create / _norm / _clip / _destroy).

    tensors  CUDA tensors (float32, float16, bfloat16, mixed as they come) of
             one device, dense in memory (contiguous or permuted)
    outs     where clip() writes: as many tensors, of the same shapes and
             layouts, of their own types; None: the tensors themselves
    The list keeps a table of addresses on the device: make a new one when a
    tensor is replaced by another.  That allocates and waits (50 to 400 us, and
    closing the old one waits for the device), so gradients should stay where
    they are: optimizer.zero_grad(set_to_none=False), or copies into tensors of
    the list's own.  No tensor may be in a list twice where clip() writes to it.
    Calls on one list must be ordered."""

    def __init__(self, tensors, outs=None):
        self._h = None
        tensors = list(tensors)
        outs = [None] * len(tensors) if outs is None else list(outs)
        if len(outs) != len(tensors):
            raise ValueError("outs must be as many as tensors")
        table = (_Tensor * max(len(tensors), 1))()
        device = next((t.device for t in tensors if isinstance(t, torch.Tensor) and t.is_cuda), None)
        if device is None:
            device = torch.device("cuda", torch.cuda.current_device())
        for entry, t, o in zip(table, tensors, outs):
            if not (isinstance(t, torch.Tensor) and t.is_cuda and t.device == device and t.dtype in _DTYPES
                    and _dense(t)):
                raise TypeError("tensors must be dense CUDA tensors of float32, float16 or bfloat16 on one device")
            if o is not None and not (isinstance(o, torch.Tensor) and o.device == device and o.dtype in _DTYPES
                                      and o.shape == t.shape
                                      and (o.stride() == t.stride() or (o.is_contiguous() and t.is_contiguous()))):
                raise TypeError("outs must have their tensors' shapes, layouts and device")
            entry.data, entry.count, entry.dtype = t.data_ptr(), t.numel(), _DTYPES[t.dtype]
            if o is not None:
                entry.out, entry.out_dtype = o.data_ptr(), _DTYPES[o.dtype]
        self._keep = (tensors, outs)
        self._clipped = [t if o is None else o for t, o in zip(tensors, outs)]
        self._device = device
        h = ctypes.c_void_p()
        with torch.cuda.device(device):
            _check(_entries().seqsum_tensors_create(table, len(tensors), ctypes.byref(h)))
        self._h = h

    def _out(self, out, stream):
        if self._h is None:
            raise SeqsumError("seqsum: the list was closed")
        return _output(out, "out", 1, torch.float32, self._device.index, self, stream)

    @property
    def device(self):
        return self._device

    def norm(self, scale: float = 1.0, out=None, stream=None):
        """scale * the 2-norm of all numbers of the list (a 1-element float32 tensor)."""
        out, p = self._out(out, stream)
        _call(self._device.index, stream, (out,), _entries().seqsum_tensors_norm, self._h, scale, p)
        return out

    def clip(self, max_norm: float, scale: float = 1.0, out=None, stream=None):
        """Writes every number times scale * min(1, max_norm / (norm + 1e-6))
        and returns the norm (of the scaled numbers, before clipping)."""
        out, p = self._out(out, stream)
        _written(self._clipped)
        _call(self._device.index, stream, (out,), _entries().seqsum_tensors_clip, self._h, max_norm, scale, p)
        return out

    def close(self):
        if self._h is not None:
            _entries().seqsum_tensors_destroy(self._h)
        self._h = self._keep = self._clipped = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
