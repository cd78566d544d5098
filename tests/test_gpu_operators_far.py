"""The operators over memory whose offsets pass 31 and 32 bits: rows that far
apart, and one tensor of that many numbers.  The tolerances are those of the
operators' own tests."""
import math

import pytest

import test_gpu_logprob as logprob
import test_gpu_tensors as tensors

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


def spread(x, stride):
    """A copy of x whose rows begin `stride` numbers apart, with 7s right beside them."""
    rows, vocab = x.shape
    m = torch.empty((rows - 1) * stride + vocab + 8, device="cuda", dtype=x.dtype)
    for r in range(rows):
        m[max(0, r * stride - 8):r * stride + vocab + 8] = 7.0
    far = m.as_strided((rows, vocab), (stride, 1))
    far.copy_(x)
    return m, far


# a warp a row, one CTA, a cluster, rows beyond the buffers (16-bit: past 8 * 112 KB)
@pytest.mark.parametrize("vocab", [1001, 9001, 50001, 600001])
@pytest.mark.parametrize("stride", [2 ** 31 + 8, 2 ** 31 + 5])
def test_rows(sq, vocab, stride):
    x, t, a = logprob.make(3, vocab, torch.bfloat16, vocab)
    u = torch.rand(3, device="cuda")
    memory, far = spread(x, stride)
    for settings in (dict(), dict(top_k=50), dict(top_p=0.9, temperature=1.5), dict(temperature=0.0)):
        want, got = sq.sample_tokens(x, u, **settings), sq.sample_tokens(far, u, **settings)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    logps, lses = sq.token_logprob(far, t)
    logprob.check(x, t, a, logps, lses)
    off = 2.0 ** -23 * float(lses.abs().max()) + logprob.SUM_EPS
    logprob.check(x, t, a, dlogits=sq.token_logprob_backward(far, t, a, lses), lse_off=off)
    d, logps, lses = sq.token_logprob_grad(far, t, a, out=far)   # in place, that far apart
    assert d is far
    logprob.check(x, t, a, logps, lses, far)
    far.copy_(x)
    assert sq.token_logprob_backward(far, t, a, lses, out=far) is far
    logprob.check(x, t, a, dlogits=far, lse_off=off)
    for r in range(3):   # nothing beside the rows was written
        end = r * stride + vocab
        assert (memory[end:end + 8] == 7).all() and (r == 0 or (memory[r * stride - 8:r * stride] == 7).all())


@pytest.mark.parametrize("n", [2 ** 31 + 1001, 2 ** 32 + 77])
def test_tensor(sq, n):
    t = torch.zeros(n, device="cuda", dtype=torch.float16)
    places = [slice(0, 9), slice(2 ** 31 - 5, 2 ** 31 + 5), slice(n - 50, n)]
    for i, p in enumerate(places):
        t[p] = tensors.make([(p.stop - p.start,)], torch.float16, i, 1.0)[0]
    before = [t[p].clone() for p in places]
    norm = math.sqrt(math.fsum(float(b.double().square().sum()) for b in before))
    with sq.TensorList([t]) as tl:
        assert tl.norm().item() == pytest.approx(norm, rel=tensors.REL)
        assert tl.clip(1.0).item() == pytest.approx(norm, rel=tensors.REL)
    tensors.check_clip(before, [t[p] for p in places], norm, 1.0, 1.0)
    for p in places:
        t[p] = 0
    assert not any(bool(part.any()) for part in t.split(2 ** 28))
