"""Results that the caller gives: beside one another and beside the inputs in one
piece of memory, and refused where they lie in what is still read."""
import pytest

import test_gpu_policy_loss as over_tokens
import test_gpu_policy_rows as over_rows
import test_gpu_preference as over_pairs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROWS = dict(kl_coef=0.1, entropy_coef=0.01)


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


def one_piece(*sizes, like=None):
    """Vectors one right after another."""
    memory = torch.full((sum(sizes),), 7.0, device="cuda", dtype=like)
    return memory.split(sizes)


@pytest.mark.parametrize("n", [5, 1003, 70001])
def test_neighbours(sq, n):
    """Places that touch are apart."""
    logps, s = over_tokens.make(n, 1)
    want = sq.policy_loss_grad(logps, **s, kl_coef=0.1)
    out, loss, lp, stats, w = one_piece(n, 1, n, 6, n)
    lp.copy_(logps), w.copy_(s["weights"])
    got = sq.policy_loss_grad(lp, **{**s, "weights": w}, kl_coef=0.1, out=out, loss=loss, stats=stats)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(lp, logps) and torch.equal(w, s["weights"])
    logps, p = over_pairs.make([n // 2, n - n // 2 - 1], 2, after=1)
    want = sq.preference_loss_grad(logps, **p)
    ref, out, scores, loss, lp = one_piece(n, n, 2, 1, n)
    ref.copy_(p["ref_logps"]), lp.copy_(logps)
    got = sq.preference_loss_grad(lp, **{**p, "ref_logps": ref}, out=out, loss=loss, scores=scores)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("n,vocab", [(40, 101), (30, 5001)])
def test_rows_between_rows(sq, n, vocab):
    """The gradient's rows in the gaps between the logits', at their stride and at another; a vector in a gap.  (Against
    the same logits with results apart: a row's last bits go by its address modulo 16.)"""
    x, t, s = over_rows.make(n, vocab, torch.float32, 3, ROWS)
    wide = torch.full((n, 2 * vocab + n + 3), 7.0, device="cuda")
    every = torch.full((2 * n, 3 * vocab), 7.0, device="cuda")
    for view, out, given in (
            (wide[:, :vocab], wide[:, vocab:2 * vocab],
             dict(logps=wide[3, 2 * vocab:2 * vocab + n], entropies=wide[4, 2 * vocab + 3:])),
            (every[::2, :vocab], every[:n, vocab:2 * vocab], {})):   # logits in every second row, gradients in every row
        view.copy_(x)
        want = sq.token_policy_grad(view, t, **s, **ROWS)
        over_rows.check(x, t, s, ROWS, want)
        got = sq.token_policy_grad(view, t, **s, **ROWS, out=out, **given)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(view, x)
    assert (wide[5:, 2 * vocab:] == 7).all() and (every[n:, vocab:] == 7).all() and (every[:n, 2 * vocab:] == 7).all()


def test_refused(sq):
    n, vocab = 33, 101
    x, t, s = over_rows.make(n, vocab, torch.float32, 3, ROWS)
    logps, p = over_pairs.make([10, 12, 5, 6], 2)
    sevens = torch.full((3 * n + 8,), 7.0, device="cuda")
    a = sevens[:n]
    tokens = lambda **kw: sq.policy_loss_grad(a, **s, kl_coef=0.1, **kw)   # noqa: E731
    rows = lambda **kw: sq.token_policy_grad(x, t, **s, **ROWS, **kw)   # noqa: E731
    pairs = lambda **kw: sq.preference_loss_grad(a, **p, **kw)   # noqa: E731
    two = torch.empty(n + 3, device="cuda")
    few = torch.empty(7, device="cuda")
    wide = torch.zeros(n, vocab + 5, device="cuda")
    for call in (lambda: tokens(out=sevens[1:n + 1]), lambda: tokens(out=s["advantages"]), lambda: tokens(loss=a[3:4]),
                 lambda: tokens(stats=s["weights"][:6]), lambda: tokens(loss=few[2:3], stats=few[:6]),
                 lambda: tokens(out=two[:n], loss=two[n - 1:n]),
                 lambda: rows(logps=two[:n], entropies=two[3:]), lambda: rows(loss=s["old_logps"][:1]),
                 lambda: rows(out=x.view(-1)[:n * vocab].view(n, vocab)[:, :], logps=x.view(-1)[5:5 + n]),
                 lambda: rows(entropies=t.view(torch.float32)[:n]), lambda: rows(stats=x[4, 7:13]),
                 lambda: sq.token_policy_grad(wide[:, :vocab], t, **s, **ROWS, out=wide[:, 5:]),
                 lambda: pairs(out=sevens[2:n + 2]), lambda: pairs(loss=a[:1]), lambda: pairs(scores=p["ref_logps"][4:8]),
                 lambda: pairs(scores=p["offsets"].view(torch.float32)[:4]), lambda: pairs(out=p["weights"])):
        with pytest.raises(ValueError, match="overlap"):
            call()
    assert (sevens == 7).all()
    # the very logits and log-probabilities are fine
    want = tokens()[0]
    assert torch.equal(tokens(out=a)[0], want)
    want = rows()[0]
    assert torch.equal(rows(out=x)[0], want)
