"""token_logprob where autograd records: its gradient is the backward pass's."""
import pytest

import test_gpu_logprob as logprob

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


@pytest.mark.parametrize("dtype", logprob.DTYPES)
@pytest.mark.parametrize("n,vocab", [(1, 7), (50, 1001), (300, 20011)])
def test_gradient(sq, dtype, n, vocab):
    x, t, a = logprob.make(n, vocab, dtype, 41)
    t[::5] = -100
    want, wl = sq.token_logprob(x, t)
    x.requires_grad_()
    logps, lses = sq.token_logprob(x, t)
    assert logps.requires_grad and torch.equal(logps, want) and torch.equal(lses, wl)
    (a * logps).sum().backward()
    assert x.grad.dtype == dtype
    assert torch.equal(x.grad, sq.token_logprob_backward(x.detach(), t, a, wl))
    logprob.check(x.detach(), t, a, dlogits=x.grad, lse_off=2.0 ** -23 * float(wl.abs().max()) + logprob.SUM_EPS)


def test_through_other_operations(sq):
    """A sum (whose gradient is one number for all rows), a product before, a shared row."""
    g = torch.Generator(device="cuda").manual_seed(42)
    x, t, _ = logprob.make(64, 301, torch.float32, 43, scale=1.0)
    w = torch.randn(301, device="cuda", generator=g, requires_grad=True)
    sq.token_logprob(x * w, t)[0].sum().backward()
    wd = w.detach().double().requires_grad_()
    torch.log_softmax(x.double() * wd, 1).gather(1, t[:, None]).sum().backward()
    # 64 rows' products of numbers below 4, each off by 2e-5 of itself at most
    assert (w.grad.double() - wd.grad).abs().max().item() < 64 * 4 * 2e-5
    row = torch.randn(1, 301, device="cuda", generator=g, requires_grad=True)
    sq.token_logprob(row.expand(64, 301), t)[0].sum().backward()
    d = row.detach().double().requires_grad_()
    torch.log_softmax(d, 1).expand(64, 301).gather(1, t[:, None]).sum().backward()
    assert (row.grad.double() - d.grad).abs().max().item() < 64 * 2e-5


def test_what_is_not_recorded(sq):
    x, t, a = logprob.make(9, 101, torch.float32, 44)
    want = sq.token_logprob(x, t)
    x.requires_grad_()
    with torch.no_grad():
        logps, lses = sq.token_logprob(x, t)
    assert not logps.requires_grad and not lses.requires_grad and torch.equal(logps, want[0])
    assert not sq.token_logprob(x.detach(), t)[0].requires_grad
    d, logps, _ = sq.token_logprob_grad(x, t, a)
    assert not d.requires_grad and not logps.requires_grad
    x.backward(d)   # the gradient as it is
    assert torch.equal(x.grad, d)
    assert not sq.sample_tokens(x, torch.rand(9, device="cuda"))[1].requires_grad


def test_refusals(sq):
    x, t, a = logprob.make(9, 101, torch.float32, 45)
    x.requires_grad_()
    e = torch.empty(9, device="cuda")
    for kw in (dict(logps=e), dict(lses=e), dict(stream=torch.cuda.Stream())):
        with pytest.raises(sq.SeqsumError):
            sq.token_logprob(x, t, **kw)
    with pytest.raises(sq.SeqsumError):   # no gradient through lses, and not in silence
        sq.token_logprob(x, t)[1].sum().backward()
    with pytest.raises(RuntimeError):     # none of the gradient
        logps, _ = sq.token_logprob(x, t)
        d, = torch.autograd.grad(logps.sum(), x, create_graph=True)
        d.sum().backward()
    with pytest.raises(TypeError):
        sq.token_logprob(x.double(), t)
    sq.token_logprob(x, t, stream=torch.cuda.current_stream())[0].sum().backward()
    assert x.grad is not None
