"""Given tensors that the operators write count as written: autograd refuses to
go back over a saved tensor that was overwritten."""
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


def test_overwritten_logits(sq):
    x, t, a = logprob.make(9, 101, torch.float32, 51)
    x.requires_grad_()
    logits = x * 1.0
    logps, lses = sq.token_logprob(logits, t)
    sq.token_logprob_backward(logits.detach(), t, a, lses, out=logits.detach())   # in their place
    with pytest.raises(RuntimeError, match="inplace"):
        logps.sum().backward()


def test_clipped_in_place(sq):
    w = torch.ones(1000, device="cuda", requires_grad=True)
    y = w * 2.0
    z = (y * y).sum()
    with sq.TensorList([y.detach()]) as tl:
        tl.norm()
        z2 = (y * y).sum()
        z2.backward()                       # (the norm writes nothing)
        tl.clip(1.0)
    with pytest.raises(RuntimeError, match="inplace"):
        z.backward()


def test_each_given_tensor(sq):
    x, t, a = logprob.make(9, 101, torch.float32, 52)
    u = torch.rand(9, device="cuda")
    tokens, logps, lses, norm = torch.empty_like(t), torch.empty_like(a), torch.empty_like(a), torch.empty(1, device="cuda")
    d, outs = torch.empty_like(x), [torch.empty_like(x), torch.empty_like(a)]
    tl = sq.TensorList([x, a], outs)

    def grows(call, *written):
        before = [w._version for w in written], [r._version for r in (x, t, a, u)]
        call()
        assert all(w._version > v for w, v in zip(written, before[0]))
        assert [r._version for r in (x, t, a, u)] == before[1]   # what is only read

    grows(lambda: sq.sample_tokens(x, u, tokens=tokens, logps=logps), tokens, logps)
    grows(lambda: sq.token_logprob(x, t, logps=logps, lses=lses), logps, lses)
    grows(lambda: sq.token_logprob_grad(x, t, a, out=d, logps=logps, lses=lses), d, logps, lses)
    grows(lambda: sq.token_logprob_backward(x, t, a, lses, out=d), d)
    grows(lambda: tl.norm(out=norm), norm)
    grows(lambda: tl.clip(1.0, out=norm), norm, *outs)
    with torch.inference_mode():            # tensors without a counter
        i = torch.empty(9, device="cuda")
        sq.token_logprob(x, t, logps=i)
        sq.TensorList([torch.ones(5, device="cuda")]).clip(0.5)
