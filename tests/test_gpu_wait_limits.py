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


# ------------------------------------------------------------ sampling

def sampling_settings(n):
    i = torch.arange(n, device="cuda")
    each = dict(temperature=torch.where(i % 5 == 0, 0.0, 0.5 + (i % 7) / 6.0).float(),
                top_k=torch.where(i % 3 == 0, i % 100, 0).int(), top_p=torch.where(i % 4 == 1, 0.9, 1.0).float())
    return [dict(), dict(temperature=0.0), dict(top_k=50), dict(top_p=0.9), dict(top_k=3000, top_p=0.8), each]


def sample(sq, x, u, s, mode, arg, wait_ns):
    n = x.shape[0]
    tokens = torch.full((n,), -7, device="cuda", dtype=torch.int64)
    logps = torch.full((n,), 7.0, device="cuda")
    sq.debug_set_fault(mode, arg, wait_ns)
    sq.sample_tokens(x, u, tokens=tokens, logps=logps, **s)
    torch.cuda.synchronize()
    sq.debug_set_fault(0, 0, 0)
    return tokens, logps


def check_sample(got, want):
    (t, lp), (wt, wlp) = got, want
    assert ((t == wt) | (t == -1)).all() and right_or_nan(lp, wlp).all(), (t, wt, lp, wlp)


# one CTA a row; eight of 8 and of 16 warps (75 rows: two turns and four)
@pytest.mark.parametrize("n,vocab,dtype,size,warps", [(3000, 5003, torch.bfloat16, 1, 8), (75, 131001, torch.float16, 8, 8),
                                                      (75, 150001, torch.bfloat16, 8, 16)])
@pytest.mark.parametrize("turn,warp", [(0, 0), (0, -1), (1, 3), (1, -1), (2, 0)])
def test_sampling(sq, n, vocab, dtype, size, warps, turn, warp):
    x, u, _ = logprob.make(n, vocab, dtype, 23)
    u = torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(24))
    x[3] = -float("inf")
    warp %= size * warps
    for s in sampling_settings(n):
        want = sq.sample_tokens(x, u, **s)
        got = sample(sq, x, u, s, 2, turn * 128 + warp, LIMIT)
        check_sample(got, want)
        if turn < 2 or warps == 16 or size == 1:
            assert got[0][-1] == -1 and got[1][-1].isnan()
        if turn == 2:
            assert got[0][0] == want[0][0] and got[1][0] == want[1][0]
        again = sq.sample_tokens(x, u, **s)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_sampling_with_next_to_no_limit(sq):
    x, u, _ = logprob.make(75, 131001, torch.bfloat16, 25)
    u = torch.rand(75, device="cuda", generator=torch.Generator(device="cuda").manual_seed(26))
    for s in sampling_settings(75):
        want = sq.sample_tokens(x, u, **s)
        for wait_ns in (1, 200, 1000, 3000, 10000):
            check_sample(sample(sq, x, u, s, 0, 0, wait_ns), want)
        again = sq.sample_tokens(x, u, **s)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
