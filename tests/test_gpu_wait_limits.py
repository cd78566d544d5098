"""Waits of the kernels on rows that give up: a call comes to its end, what it
wrote is right or marked, and the next call is right.  The wait of one warp of
each cluster is taken to have given up; those of the others run out, since that
warp tells them nothing any more."""
import pytest

import test_gpu_logprob as logprob

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LIMIT = 20_000_000   # ns; waits of a call that goes well take microseconds


@pytest.fixture()
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    yield sq
    sq.debug_set_fault(0, 0, 0)


def right_or_nan(got, want):
    return (got == want) | got.isnan()


# one CTA a row, four, eight; rows one after another in each
@pytest.mark.parametrize("n,vocab,dtype,size", [(3000, 20011, torch.bfloat16, 1), (2000, 30001, torch.float32, 4),
                                                (900, 131073, torch.float16, 8)])
@pytest.mark.parametrize("turn,warp", [(0, 0), (0, -1), (1, 3), (2, -1), (2, 0)])
def test_logprob(sq, n, vocab, dtype, size, turn, warp):
    x, t, a = logprob.make(n, vocab, dtype, 21)
    t[::7] = -100
    d, logps, lses = sq.token_logprob_grad(x, t, a)
    warp %= size * 8
    for grad in (False, True):
        for in_place in ((False, True) if grad else (False,)):
            lp, ls = torch.full_like(logps, 7.0), torch.full_like(lses, 7.0)
            y = x.clone()
            out = y if in_place else torch.full_like(x, 7.0)
            sq.debug_set_fault(2, turn * 128 + warp, LIMIT)
            if grad:
                sq.token_logprob_grad(y, t, a, out=out, logps=lp, lses=ls)
            else:
                sq.token_logprob(y, t, logps=lp, lses=ls)
            torch.cuda.synchronize()
            sq.debug_set_fault(0, 0, 0)
            assert right_or_nan(lp, logps).all() and right_or_nan(ls, lses).all()
            assert lp[-1].isnan() and ls[-1].isnan()   # (its turn is a later one)
            if turn == 2:
                assert ls[0] == lses[0] and lp[0] == logps[0]
            if grad:
                assert right_or_nan(out, d).all() and out[-1].isnan().all()
                assert turn < 2 or torch.equal(out[0], d[0])
    again = sq.token_logprob_grad(x, t, a)
    assert torch.equal(again[0], d) and torch.equal(again[1], logps) and torch.equal(again[2], lses)


def test_logprob_with_next_to_no_limit(sq):
    """Waits give up wherever they happen to be long."""
    x, t, a = logprob.make(900, 131073, torch.bfloat16, 22)
    d, logps, lses = sq.token_logprob_grad(x, t, a)
    for wait_ns in (1, 500, 5000):
        out, lp, ls = torch.full_like(x, 7.0), torch.full_like(logps, 7.0), torch.full_like(lses, 7.0)
        sq.debug_set_fault(0, 0, wait_ns)
        sq.token_logprob_grad(x, t, a, out=out, logps=lp, lses=ls)
        torch.cuda.synchronize()
        sq.debug_set_fault(0, 0, 0)
        assert right_or_nan(lp, logps).all() and right_or_nan(ls, lses).all() and right_or_nan(out, d).all()
    assert torch.equal(sq.token_logprob_grad(x, t, a)[0], d)
