"""token_logprob, its fused gradient and its backward pass against 64 bits.

Tolerances: an exponential's argument carries two roundings, relative 2^-23 of
(x - m) * log2(e) together, and ex2 2^-22: an element's weight is off by at
most (2^-23 |d| + 2^-22) of itself, d <= 0 in octaves, so a row's sum by
SUM_EPS = 2e-6 of itself (weights of 2^-30 and less do not reach it), lse by
that and two roundings of its own size; logp by those and one of |x - m|.
A gradient's element: (2^-23 |d| + 2^-22 + SUM_EPS + 3 * 2^-24) of itself, and
the rounding to its type; below 2^-126 it is 0."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
SUM_EPS = 2e-6
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}    # (bf16: half of 2^-7)
TINY = {torch.float32: 2.0 ** -125, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -125}


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


def make(n, vocab, dtype, seed, scale=4.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(n, vocab, device="cuda", generator=g) * scale).to(dtype)
    t = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    a = torch.randn(n, device="cuda", generator=g)
    return x, t, a


def in_64(x, t, a):
    x = x.double()
    n, vocab = x.shape
    lse = torch.logsumexp(x, 1)
    used = (t >= 0) & (t < vocab)
    at = torch.where(used, t, 0)
    r = torch.arange(n, device=x.device)
    logp = torch.where(used, x[r, at] - lse, 0.0)
    a = torch.where(used, a.double(), 0.0)
    p = torch.exp(x - lse[:, None])
    d = -a[:, None] * p
    d[r, at] += a
    return lse, logp, d, p


def check(x, t, a, logps=None, lses=None, dlogits=None, lse_off=0.0):
    lse, logp, d, p = in_64(x, t, a)
    big = x.double().abs().max(1).values
    if lses is not None:
        assert (lses.double() - lse).abs().le(SUM_EPS + 2.0 ** -23 * lse.abs()).all()
        assert (logps.double() - logp).abs().le(SUM_EPS + 2.0 ** -23 * (logp.abs() + big)).all()
    if dlogits is not None:
        assert dlogits.dtype == x.dtype and dlogits.shape == x.shape
        octaves = (x.double() - lse[:, None]).abs() * 1.4427
        rel = 2.0 ** -23 * octaves + 2.0 ** -22 + SUM_EPS + 2.0 ** -22 + lse_off
        tol = rel * p * a.double().abs()[:, None] + (HALF[x.dtype] + 2.0 ** -23) * d.abs() + TINY[x.dtype]
        assert (dlogits.double() - d).abs().le(tol).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 9, 1000, 4099, 32768, 50001, 131077])
@pytest.mark.parametrize("n", [1, 5, 400])
def test_sizes(sq, dtype, vocab, n):
    x, t, a = make(n, vocab, dtype, vocab + n)
    if n > 2:
        t[1], t[2] = -100, vocab
    logps, lses = sq.token_logprob(x, t)
    check(x, t, a, logps, lses)
    d, logps2, lses2 = sq.token_logprob_grad(x, t, a)
    assert torch.equal(logps, logps2) and torch.equal(lses, lses2)
    check(x, t, a, logps2, lses2, d)
    # the lse given to the backward pass has its own rounding, which moves every exponential
    b = sq.token_logprob_backward(x, t, a, lses)
    check(x, t, a, dlogits=b, lse_off=2.0 ** -23 * float(lses.abs().max()) + SUM_EPS)
    if n > 2:
        assert not d[1:3].any() and not b[1:3].any() and logps[1].item() == logps[2].item() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [600001, 1100000])
def test_rows_larger_than_the_chip(sq, dtype, vocab):
    x, t, a = make(3, vocab, dtype, vocab, scale=2.0)
    d, logps, lses = sq.token_logprob_grad(x, t, a)
    check(x, t, a, logps, lses, d)
    check(x, t, a, dlogits=sq.token_logprob_backward(x, t, a, lses), lse_off=2.0 ** -22 * 16 + SUM_EPS)
    y = x.clone()
    d2, _, _ = sq.token_logprob_grad(y, t, a, out=y)
    assert torch.equal(d, d2)


@pytest.mark.parametrize("dtype", DTYPES)
def test_differences(sq, dtype):
    """The gradient along a direction against a central difference of the 64-bit loss: the difference's own error is
    h^2/6 of a third derivative (at most sum |a| * |v|^3 here), the gradient's that of its elements."""
    x, t, a = make(6, 301, dtype, 3, scale=1.5)
    d, _, _ = sq.token_logprob_grad(x, t, a)
    g = torch.Generator(device="cuda").manual_seed(4)
    h = 1e-4
    for _ in range(5):
        v = torch.randn(x.shape, device="cuda", generator=g, dtype=torch.float64)

        def loss(s):
            return (a.double() * in_64(x.double() + s * v, t, a)[1]).sum()
        diff = ((loss(h) - loss(-h)) / (2 * h)).item()
        tol = h * h * float((a.double().abs() * v.abs().max(1).values ** 3).sum()) + 1e-10
        tol += float(((HALF[dtype] + 1e-5) * d.double().abs() * v.abs()).sum()) + TINY[dtype] * float(v.abs().sum())
        assert abs(diff - (d.double() * v).sum().item()) <= tol


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_places(sq, dtype):
    vocab = 3003
    x, t, a = make(9, vocab, dtype, 5)
    low = torch.finfo(dtype).min
    x[0] = -math.inf
    x[1, 1:] = -math.inf
    t[1] = 0
    x[2, 7] = -math.inf
    t[2] = 7
    x[3] = low
    x[4, 10:] = low
    t[4] = 20
    x[5, 3] = math.nan
    x[6, 3] = math.inf
    x[7] = math.nan
    t[7] = -1
    d, logps, lses = sq.token_logprob_grad(x, t, a)
    b = sq.token_logprob_backward(x, t, a, lses)
    lse, logp, want, _ = in_64(x, t, a)
    assert lses[0].item() == logps[0].item() == -math.inf and not d[0].any() and not b[0].any()
    assert logps[1].item() == 0 and lses[1].item() == x[1, 0].item() and d[1, 1:].abs().max() == 0
    assert abs(d[1, 0].item()) <= 1e-6
    assert logps[2].item() == -math.inf and abs(lses[2].item() - lse[2].item()) < 1e-4
    assert d[2, 7].item() == a[2].to(dtype).item() and b[2, 7].item() == a[2].to(dtype).item()
    assert abs(lses[3].item() - lse[3].item()) <= 2.0 ** -23 * abs(low) and abs(logps[3].item() + math.log(vocab)) < 1e-5
    assert logps[4].item() == pytest.approx(logp[4].item(), rel=1e-6)
    for r in (5, 6):
        assert math.isnan(lses[r].item()) and math.isnan(logps[r].item()) and d[r].isnan().all() and b[r].isnan().all()
    assert math.isnan(lses[7].item()) and logps[7].item() == 0 and not d[7].any() and not b[7].any()
    keep = [2, 4, 8]
    np.testing.assert_allclose(d[keep].double().cpu(), want[keep].cpu(), rtol=2 * HALF[dtype] + 1e-5,
                               atol=2 * TINY[dtype] + 1e-7)
    assert (logps[8] - logp[8]).abs().item() < 1e-4


def test_strides_alignments_and_place(sq):
    """Rows of a wider tensor, at odd addresses, gradients written in place and to rows of another alignment; a row's
    numbers do not depend on where it lies or what is beside it."""
    n, vocab = 33, 5001
    x, t, a = make(n, vocab, torch.bfloat16, 7)
    d, logps, lses = sq.token_logprob_grad(x, t, a)
    for shift in (0, 1, 5):
        wide = torch.zeros(n, vocab + 9, device="cuda", dtype=x.dtype)
        view = wide[:, shift:shift + vocab]
        view.copy_(x)
        d2, lp2, ls2 = sq.token_logprob_grad(view, t, a)
        torch.testing.assert_close(lp2, logps, rtol=1e-6, atol=1e-6)
        torch.testing.assert_close(d2.float(), d.float(), rtol=2.0 ** -7, atol=1e-7)
        out = torch.full((n, vocab + 3), 7.0, device="cuda", dtype=x.dtype)
        sq.token_logprob_grad(view, t, a, out=out[:, 2:2 + vocab])
        assert torch.equal(out[:, 2:2 + vocab], d2) and (out[:, :2] == 7).all() and (out[:, 2 + vocab:] == 7).all()
        b = sq.token_logprob_backward(view, t, a, ls2)
        sq.token_logprob_backward(view, t, a, ls2, out=view)
        assert torch.equal(view, b) and not wide[:, :shift].any() and not wide[:, shift + vocab:].any()
    one, lp1, ls1 = sq.token_logprob_grad(x[4:5], t[4:5].clone(), a[4:5].clone())
    assert torch.equal(one[0], d[4]) and lp1.item() == logps[4].item() and ls1.item() == lses[4].item()
    y = x.clone()
    sq.token_logprob_grad(y, t, a, out=y)
    assert torch.equal(y, d)


def test_a_shared_row(sq):
    """One row's memory for many tokens (stride 0): scores of every token of one distribution."""
    vocab = 2003
    x, _, _ = make(1, vocab, torch.float32, 9)
    t = torch.arange(vocab, device="cuda")
    logps, lses = sq.token_logprob(x.expand(vocab, vocab), t)
    want = torch.log_softmax(x[0].double(), 0)
    assert (logps.double() - want).abs().max().item() < 1e-5
    assert (lses == lses[0]).all()


def test_nothing_to_do(sq):
    e = torch.empty(0, 7, device="cuda")
    none = torch.empty(0, device="cuda")
    d, lp, ls = sq.token_logprob_grad(e, none.long(), none)
    assert d.shape == (0, 7) and lp.shape == ls.shape == (0,)
    e = torch.empty(2, 0, device="cuda")
    z = torch.zeros(2, device="cuda")
    lp, ls = sq.token_logprob(e, z.long())
    assert lp.tolist() == [0, 0] and ls.tolist() == [-math.inf] * 2
    assert sq.token_logprob_backward(e, z.long(), z, ls).shape == (2, 0)


def test_graph(sq):
    x, t, a = make(50, 20011, torch.float16, 11)
    d = torch.empty_like(x)
    lp, ls = torch.empty_like(a), torch.empty_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sq.token_logprob_grad(x, t, a, out=d, logps=lp, lses=ls)
    x2, t2, a2 = make(50, 20011, torch.float16, 12)
    for p, q in ((x, x2), (t, t2), (a, a2)):
        p.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    want, wl, _ = sq.token_logprob_grad(x2, t2, a2)
    assert torch.equal(d, want) and torch.equal(lp, wl)


def test_refusals(sq):
    x, t, a = make(4, 100, torch.float32, 13)
    for bad in (lambda: sq.token_logprob(x.double(), t), lambda: sq.token_logprob(x.t(), t),
                lambda: sq.token_logprob(x, t.int()), lambda: sq.token_logprob(x, t[:2]),
                lambda: sq.token_logprob_grad(x, t, a.double()), lambda: sq.token_logprob_grad(x, t, a, out=x.half()),
                lambda: sq.token_logprob_grad(x, t, a, out=torch.empty(1, 100, device="cuda").expand(4, 100)),
                lambda: sq.token_logprob_backward(x, t, a, a[:1]), lambda: sq.token_logprob_backward(x, t, a, a, out=x[:2])):
        with pytest.raises(TypeError):
            bad()
