"""Refusals of the operators' entries that need no GPU: bad arguments are
refused before any CUDA call."""
import ctypes

import pytest

vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
P = vp(4096)   # never read: the call is refused first
FP32, FP16, BF16 = 0, 1, 2
EINVAL = -1


class Sampling(ctypes.Structure):
    _fields_ = [("temperature", f32), ("top_k", i32), ("top_p", f32), ("min_p", f32), ("temperatures", vp),
                ("top_ks", vp), ("top_ps", vp), ("min_ps", vp)]


class Tensor(ctypes.Structure):
    _fields_ = [("data", vp), ("out", vp), ("count", i64), ("dtype", i32), ("out_dtype", i32)]


@pytest.fixture(scope="module")
def lib():
    from parity_binade_chunked_gb300 import build
    return ctypes.CDLL(build.build())


def rows(logits=P, dtype=BF16, n=4, vocab=100, stride=100):
    return [logits, i32(dtype), i64(n), i64(vocab), i64(stride)]


BAD_ROWS = [dict(n=-1), dict(n=(1 << 27) + 1), dict(vocab=-1), dict(vocab=(1 << 24) + 1), dict(dtype=3), dict(dtype=-1),
            dict(stride=-1), dict(logits=None), dict(logits=vp(4097)), dict(logits=vp(4098), dtype=FP32)]


@pytest.mark.parametrize("bad", BAD_ROWS)
def test_rows_refused(lib, bad):
    s = ctypes.byref(Sampling(1.0, 0, 1.0, 0.0))
    assert lib.seqsum_sample_tokens(*rows(**bad), P, s, P, P, None) == EINVAL
    assert lib.seqsum_token_logprob(*rows(**bad), P, P, P, None) == EINVAL
    assert lib.seqsum_token_logprob_grad(*rows(**bad), P, P, P, i64(100), P, P, None) == EINVAL
    assert lib.seqsum_token_logprob_backward(*rows(**bad), P, P, P, P, i64(100), None) == EINVAL


def test_no_rows_is_no_work(lib):
    s = ctypes.byref(Sampling(1.0, 0, 1.0, 0.0))
    r = rows(n=0, logits=None)
    assert lib.seqsum_sample_tokens(*r, None, s, None, None, None) == 0
    assert lib.seqsum_token_logprob(*r, None, None, None, None) == 0
    assert lib.seqsum_token_logprob_grad(*r, None, None, None, i64(100), None, None, None) == 0
    assert lib.seqsum_token_logprob_backward(*r, None, None, None, None, i64(100), None) == 0


def test_null_vectors_refused(lib):
    s = ctypes.byref(Sampling(1.0, 0, 1.0, 0.0))
    for k in range(4):
        a = [P, s, P, P]
        a[k] = None
        assert lib.seqsum_sample_tokens(*rows(), *a, None) == EINVAL, k
    for k in range(3):
        a = [P, P, P]
        a[k] = None
        assert lib.seqsum_token_logprob(*rows(), *a, None) == EINVAL, k
    for k in range(5):
        a = [P, P, P, P, P]
        a[k] = None
        assert lib.seqsum_token_logprob_grad(*rows(), *a[:3], i64(100), *a[3:], None) == EINVAL, k
    for k in range(4):
        a = [P, P, P, P]
        a[k] = None
        assert lib.seqsum_token_logprob_backward(*rows(), *a, i64(100), None) == EINVAL, k


def test_gradient_rows_must_not_overlap(lib):
    assert lib.seqsum_token_logprob_grad(*rows(), P, P, P, i64(99), P, P, None) == EINVAL
    assert lib.seqsum_token_logprob_backward(*rows(), P, P, P, P, i64(99), None) == EINVAL


@pytest.mark.parametrize("bad", [dict(count=-1), dict(data=None), dict(dtype=3), dict(data=4097), dict(out=4097),
                                 dict(out=4096, out_dtype=7), dict(count=(1 << 46) + 1)])
def test_tensors_refused(lib, bad):
    t = Tensor(**{**dict(data=4096, out=None, count=10, dtype=FP16, out_dtype=FP16), **bad})
    h = vp()
    assert lib.seqsum_tensors_create(ctypes.byref(t), 1, ctypes.byref(h)) == EINVAL
    assert not h.value


def test_lists_refused(lib):
    h = vp()
    assert lib.seqsum_tensors_create(None, 1, ctypes.byref(h)) == EINVAL
    assert lib.seqsum_tensors_create(None, -1, ctypes.byref(h)) == EINVAL
    assert lib.seqsum_tensors_create(None, 0, None) == EINVAL
    assert lib.seqsum_tensors_norm(None, f32(1.0), P, None) == EINVAL
    assert lib.seqsum_tensors_clip(None, f32(1.0), f32(1.0), P, None) == EINVAL
    lib.seqsum_tensors_destroy(None)


def test_binding_refuses_what_is_not_a_cuda_tensor():
    torch = pytest.importorskip("torch")
    import parity_binade_chunked_gb300 as sq
    x, v = torch.zeros(2, 5), torch.zeros(2)
    for call in (lambda: sq.sample_tokens(x, v), lambda: sq.token_logprob(x, v.long()),
                 lambda: sq.token_logprob_grad(x, v.long(), v), lambda: sq.token_logprob_backward(x, v.long(), v, v)):
        with pytest.raises(TypeError):
            call()
