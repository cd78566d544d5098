"""Sampling (sample_tokens) against its definition in integers, and against
probabilities in 64 bits.

The integer definition is followed entry by entry on the host; its weights'
2^d is torch.exp2 on the GPU, which calls the same exp2f as the kernel, so the
tokens have to be equal.  Against 64 bits: d carries three roundings
(relative 2^-24 each and 2^-25 of the constant), so for |d| <= 32 a weight is
off by at most 32 * 3.5 * 2^-24 * ln 2 < 4.7e-6 of itself, and by 2^-32 (of
the maximum's) from its own rounding: a sum over a row by EPS(vocab)."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def EPS(vocab):
    return 5e-6 + vocab * 2.0 ** -32


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


def rows_of(v, n, dtype):
    return v.cpu().numpy() if isinstance(v, torch.Tensor) else np.full(n, v, dtype)


def by_definition(logits, u, temperature, top_k, top_p, min_p):
    x = logits.float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    n, vocab = x.shape
    t = rows_of(temperature, n, np.float32)
    k = rows_of(top_k, n, np.int64)
    p = rows_of(top_p, n, np.float32)
    q = rows_of(min_p, n, np.float32)
    m = x.max(dim=1, keepdim=True).values if vocab else torch.full((n, 1), -math.inf, device=x.device)
    c = torch.tensor(np.float32(1.4426950408889634) / np.where(t > 0, t, 1).astype(np.float32), device=x.device)[:, None]
    d = torch.where(x == m, 0.0, (x - m) * c)
    w = torch.round(torch.exp2(d) * 2.0 ** 31)
    w = torch.where(torch.isnan(w), 0, w).long().cpu().numpy()
    d, x, m, u = d.cpu().numpy(), x.cpu().numpy(), m.cpu().numpy()[:, 0], u.cpu().numpy()
    tokens, kept_counts = [], []
    for r in range(n):
        if m[r] == -math.inf:
            tokens.append(-1)
            kept_counts.append(0)
            continue
        if not t[r] > 0:
            tokens.append(int(np.flatnonzero(x[r] == m[r])[0]))
            kept_counts.append(1)
            continue
        some = np.flatnonzero(w[r] > 0)   # what weighs nothing decides nothing
        order = some[np.argsort(-d[r][some], kind="stable")]
        if k[r] > 0:
            order = order[:k[r]]
        mass = int(w[r][order].sum())
        if p[r] < 1:
            cut = (int(math.floor(float(p[r]) * 2.0 ** 32)) if p[r] > 0 else 0) * mass >> 32
            before = np.cumsum(w[r][order]) - w[r][order]
            order = order[(before < cut) | (np.arange(len(order)) == 0)]
        least = int(np.round(min(float(q[r]), 1.0) * 2.0 ** 31)) if q[r] > 0 else 0
        kept = np.sort(order[w[r][order] >= least])
        sums = np.cumsum(w[r][kept])
        z = int(sums[-1])
        part = int(min(max(float(u[r]), 0.0), 1.0) * 2.0 ** 32) if u[r] == u[r] else 0
        target = min(part, 2 ** 32 - 1) * z >> 32
        tokens.append(int(kept[np.searchsorted(sums, target, side="right")]))
        kept_counts.append(len(kept))
    return np.array(tokens), kept_counts


def check_64(logits, u, tokens, logps, temperature, top_k, top_p, min_p):
    """Whether each token is one that 64-bit probabilities allow, and its logp."""
    x = logits.double().cpu().numpy()
    x = np.where(np.isnan(x), -np.inf, x)
    n, vocab = x.shape
    eps = EPS(vocab)
    t, k = rows_of(temperature, n, np.float64), rows_of(top_k, n, np.int64)
    p, q = rows_of(top_p, n, np.float64), rows_of(min_p, n, np.float64)
    for r in range(n):
        m = x[r].max()
        tok = tokens[r]
        assert x[r, tok] > -np.inf
        e = np.where(x[r] == m, 1.0, np.exp((x[r] - m) / t[r]))
        order = np.argsort(-e, kind="stable")
        # entries that are surely kept, and those that may be
        rank = np.empty(vocab, int)
        rank[order] = np.arange(vocab)
        sure, may = np.ones(vocab, bool), np.ones(vocab, bool)
        if 0 < k[r] < vocab:
            edge = e[order[k[r] - 1]]
            sure &= e > edge * (1 + eps)
            may &= e >= edge * (1 - eps)
            e_k = np.where(rank < k[r], e, 0)
        else:
            e_k = e
        total = e_k.sum()
        if p[r] < 1:
            s = e_k[order]
            before = np.empty(vocab)
            before[order] = np.cumsum(s) - s
            # equal weights may stand in any order beside each other
            first = np.empty(vocab)
            es = e[order]
            first[order] = before[order][np.searchsorted(-es, -es * (1 + eps), side="left").clip(0, vocab - 1)]
            last = before + e
            sure &= (last < p[r] * total - eps * total) | (e > es[0] * (1 - 1e-15)) & (np.count_nonzero(e >= es[0] * (1 - eps)) == 1)
            may &= (first < p[r] * total + eps * total) | (e >= es[0] * (1 - eps))
        sure &= e >= q[r] * (1 + eps)
        may &= e >= min(q[r], 1) * (1 - eps)
        sure &= may
        assert may[tok], (r, tok)
        z_lo, z_hi = e[sure].sum(), e[may].sum()
        z_lo = max(z_lo, e[tok])
        # the sum before the token must not pass u * z, the sum with it must
        lo_before, hi_upto = e[:tok][sure[:tok]].sum(), e[:tok + 1][may[:tok + 1]].sum()
        assert lo_before <= u[r] * z_hi + 2 * eps * z_hi, (r, tok)
        assert hi_upto >= u[r] * z_lo - 2 * eps * z_hi, (r, tok)
        lp_hi, lp_lo = math.log(e[tok] / z_lo), math.log(e[tok] / z_hi)
        tol = 4 * eps + 1e-6 * (1 + abs(lp_lo))
        assert lp_lo - tol <= logps[r] <= lp_hi + tol, (r, tok, logps[r], lp_lo, lp_hi)


def make(n, vocab, dtype, seed, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(n, vocab, device="cuda", generator=g) * scale).to(dtype)
    return x, torch.rand(n, device="cuda", generator=g)


FILTERS = [dict(), dict(top_k=1), dict(top_k=20), dict(top_p=0.9), dict(top_p=0.3, temperature=0.7), dict(min_p=0.05),
           dict(top_k=500, top_p=0.95, temperature=1.4), dict(top_k=40, top_p=0.8, min_p=0.02), dict(top_p=0.0),
           dict(top_k=7, temperature=50.0), dict(top_p=0.999, temperature=0.01), dict(min_p=2.0)]


def settings(**kw):
    return {**dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), **kw}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 33, 1000, 4099, 50001])
def test_sizes_and_filters(sq, dtype, vocab):
    for i, f in enumerate(FILTERS):
        s = settings(**f)
        n = 9 if vocab < 50001 else 3
        x, u = make(n, vocab, dtype, 1000 + i)
        tokens, logps = sq.sample_tokens(x, u, **s)
        want, _ = by_definition(x, u, **s)
        assert np.array_equal(tokens.cpu().numpy(), want), (f, tokens, want)
        if s["top_p"] > 0:
            check_64(x, u.cpu().numpy().astype(float), want, logps.cpu().numpy().astype(float), **s)


@pytest.mark.parametrize("dtype", DTYPES)
def test_settings_of_each_row(sq, dtype):
    n, vocab = 300, 5003
    x, u = make(n, vocab, dtype, 5)
    g = torch.Generator().manual_seed(6)
    s = dict(temperature=torch.tensor(np.random.RandomState(1).choice([0.0, 0.3, 1.0, 1.7, -1.0], n).astype(np.float32)),
             top_k=torch.randint(-1, 60, (n,), generator=g, dtype=torch.int32),
             top_p=torch.rand(n, generator=g) * 1.2, min_p=torch.rand(n, generator=g) * 0.2 - 0.1)
    s = {k: v.cuda() for k, v in s.items()}
    tokens, logps = sq.sample_tokens(x, u, **s)
    want, _ = by_definition(x, u, **s)
    assert np.array_equal(tokens.cpu().numpy(), want)
    greedy = (s["temperature"] <= 0).cpu().numpy()
    assert np.all(logps.cpu().numpy()[greedy] == 0)
    assert np.all(np.isfinite(logps.cpu().numpy()))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [5, 2049, 40000])
def test_ties(sq, dtype, vocab):
    """All logits equal, or of two values: the lower index goes first, in the filters and in the draw."""
    n = 64
    u = (torch.arange(n, device="cuda") / n).float()
    flat = torch.zeros(n, vocab, device="cuda", dtype=dtype)
    for s in (settings(), settings(top_k=3), settings(top_p=0.5), settings(top_k=1000, top_p=0.4), settings(min_p=1.0)):
        tokens, logps = sq.sample_tokens(flat, u, **s)
        want, kept = by_definition(flat, u, **s)
        assert np.array_equal(tokens.cpu().numpy(), want), s
        np.testing.assert_allclose(logps.cpu().numpy(), -np.log(kept), rtol=1e-6, atol=1e-6)
    two = torch.where(torch.arange(vocab, device="cuda") % 3 == 1, 1.0, 0.5).to(dtype).expand(n, vocab)
    for s in (settings(top_k=2), settings(top_k=vocab // 2), settings(top_p=0.6), settings(top_k=vocab - 1, top_p=0.9)):
        tokens, _ = sq.sample_tokens(two, u, **s)      # one row's memory for all (stride 0)
        assert np.array_equal(tokens.cpu().numpy(), by_definition(two, u, **s)[0]), s


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_places(sq, dtype):
    """-inf, the type's lowest value and NaN in masked places; +inf; rows with nothing left."""
    vocab = 3001
    x, u = make(12, vocab, dtype, 7)
    low = torch.finfo(dtype).min
    x[0] = -math.inf
    x[1] = math.nan
    x[2, :] = low
    x[3, 5:] = -math.inf
    x[4, ::2] = math.nan
    x[5, 17] = math.inf
    x[6, [40, 41]] = math.inf
    x[7, 1:] = low
    x[8, :-1] = -math.inf
    x[9, ::3] = low
    x[10, 100:] = low
    for s in (settings(), settings(top_k=4), settings(top_p=0.7), settings(top_k=900, top_p=0.99, min_p=0.001),
              settings(temperature=0.0), settings(temperature=1e-30), settings(temperature=math.inf),
              settings(temperature=1e-42)):
        tokens, logps = sq.sample_tokens(x, u, **s)
        want, _ = by_definition(x, u, **s)
        assert np.array_equal(tokens.cpu().numpy(), want), (s, tokens, want)
        assert want[0] == want[1] == -1 and want[5] == 17 and want[6] in (40, 41) and want[8] == vocab - 1
        lp = logps.cpu().numpy()
        assert lp[0] == lp[1] == -math.inf and lp[8] == 0 and not np.isnan(lp).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [600001, 1100000])
def test_rows_larger_than_the_chip(sq, dtype, vocab):
    for s in (settings(), settings(top_k=50, top_p=0.9), settings(top_p=0.8)):
        x, u = make(2, vocab, dtype, 9, scale=2.0)
        tokens, logps = sq.sample_tokens(x, u, **s)
        want, _ = by_definition(x, u, **s)
        assert np.array_equal(tokens.cpu().numpy(), want), s
        check_64(x, u.cpu().numpy().astype(float), want, logps.cpu().numpy().astype(float), **s)


@pytest.mark.parametrize("vocab", [1023, 33001])
def test_a_row_alone_and_among_others(sq, vocab):
    """The same row gives the same token and logp in any batch, at any alignment and row stride."""
    x, u = make(400, vocab, torch.bfloat16, 11)
    s = settings(top_k=100, top_p=0.9, temperature=0.9)
    tokens, logps = sq.sample_tokens(x, u, **s)
    wide = torch.zeros(400, vocab + 13, device="cuda", dtype=x.dtype)
    wide[:, 3:3 + vocab] = x
    t2, l2 = sq.sample_tokens(wide[:, 3:3 + vocab], u, **s)
    assert torch.equal(tokens, t2) and torch.equal(logps, l2)
    for r in (0, 1, 7, 399):
        t1, l1 = sq.sample_tokens(x[r:r + 1].clone(), u[r:r + 1].clone(), **s)
        assert t1.item() == tokens[r].item() and l1.item() == logps[r].item()


def test_edges_of_u(sq):
    x, _ = make(6, 4097, torch.float32, 13)
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, math.nan], device="cuda")
    for s in (settings(), settings(top_k=10), settings(top_p=0.5)):
        tokens, _ = sq.sample_tokens(x, u, **s)
        assert np.array_equal(tokens.cpu().numpy(), by_definition(x, u, **s)[0])


def test_frequencies(sq):
    """Tokens of an even grid of u come as often as their probability says, within one of the grid's steps a token."""
    n, vocab = 20000, 11
    x, _ = make(1, vocab, torch.float32, 15, scale=1.0)
    u = (torch.arange(n, device="cuda", dtype=torch.float64) / n).float()
    tokens, _ = sq.sample_tokens(x.expand(n, vocab), u)
    got = np.bincount(tokens.cpu().numpy(), minlength=vocab)
    want = torch.softmax(x[0].double(), 0).cpu().numpy() * n
    assert np.abs(got - want).max() <= 1 + n * 1e-5


def test_nothing_to_do(sq):
    t, p = sq.sample_tokens(torch.empty(0, 10, device="cuda"), torch.empty(0, device="cuda"))
    assert t.shape == p.shape == (0,)
    t, p = sq.sample_tokens(torch.empty(3, 0, device="cuda"), torch.zeros(3, device="cuda"), top_k=3, top_p=0.5)
    assert t.tolist() == [-1] * 3 and p.tolist() == [-math.inf] * 3


def test_other_stream_and_graph(sq):
    x, u = make(20, 30011, torch.bfloat16, 17)
    s = settings(top_k=50, top_p=0.9)
    want, lw = sq.sample_tokens(x, u, **s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t, _ = sq.sample_tokens(x, u, **s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(t, want)
    tokens, logps = torch.empty_like(want), torch.empty_like(lw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sq.sample_tokens(x, u, **s, tokens=tokens, logps=logps)
    x2, u2 = make(20, 30011, torch.bfloat16, 18)
    want2, lw2 = sq.sample_tokens(x2, u2, **s)
    x.copy_(x2)
    u.copy_(u2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(tokens, want2) and torch.equal(logps, lw2)


def test_refusals(sq):
    x, u = make(4, 100, torch.float32, 19)
    for bad in (lambda: sq.sample_tokens(x.double(), u), lambda: sq.sample_tokens(x[0], u),
                lambda: sq.sample_tokens(x.t(), u), lambda: sq.sample_tokens(x, u.double()),
                lambda: sq.sample_tokens(x, u[:3]), lambda: sq.sample_tokens(x, u.cpu()),
                lambda: sq.sample_tokens(x, u, top_k=torch.ones(4, device="cuda")),
                lambda: sq.sample_tokens(x, u, temperature=torch.ones(3, device="cuda")),
                lambda: sq.sample_tokens(x, u, tokens=torch.empty(4, device="cuda"))):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        sq.sample_tokens(x, u, temperature=math.nan)
    with pytest.raises(sq.SeqsumError):
        sq.sample_tokens(torch.empty(1, (1 << 24) + 1, device="cuda", dtype=torch.float16), u[:1])
