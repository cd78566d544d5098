"""token_policy_grad at the ends of its settings' range: rows of nothing but
-inf, masked places and rows of extreme numbers, at every temperature, in every
type and in every kernel.

Tolerances are those of the tests over ordinary rows.  Their 64-bit rows are
taken from the largest number before they are divided by the temperature: x / T
itself keeps nothing of a logarithm beside 1e30."""
import math

import pytest

import test_gpu_policy_rows as over_rows
from test_gpu_logprob import DTYPES, HALF, TINY

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# 8, 16 and 32 lanes a row, one CTA, clusters without and with the next row summed first, rows beyond the chip
VOCABS = [3, 101, 257, 601, 1003, 2900, 9001, 50001, 140001, 600001]


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


def shifted(x):
    """Rows in 64 bits, less their largest number."""
    m = x.double().max(1, keepdim=True).values
    return x.double() - torch.where(m.isfinite(), m, 0.0)


def check(x, t, s, settings, got, rows, loss=True):
    """The given rows' results, and the sums, whose other rows are unused."""
    want = over_rows.in_64(shifted(x), t, s, **settings)
    for name, g in zip(over_rows.NAMES, got):
        w, off = want[name]
        if name in ("dlogits", "logps", "entropies"):
            g, w, off = g[rows], w[rows], off[rows]
        elif not loss:
            continue
        if name == "dlogits":
            off = off + HALF[x.dtype] * (w.abs() + off) + TINY[x.dtype]
        most = torch.finfo(g.dtype).max
        beyond = (w.abs() + off > most) & g.isinf() & (g.sign() == w.sign())
        far = torch.where(beyond, 0.0, (g.double() - w).abs() - off)
        assert far.le(0).all(), (name, far.max(), (g.double() - w).abs().max())


def make(n, vocab, dtype, seed, temperature, weight=1.0, masked=0.0):
    """Rows whose tokens are their largest numbers' and others, as ratios that no bound is near."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(n, vocab, device="cuda", generator=g) * 2).to(dtype)
    mask = torch.rand(n, vocab, device="cuda", generator=g) < masked
    mask[:, 0] = False
    x.masked_fill_(mask, -math.inf)
    t = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    t[::2] = x.float().argmax(1)[::2]
    t = torch.where(x.gather(1, t[:, None])[:, 0].isinf(), 0, t)
    lp = torch.log_softmax(shifted(x) / temperature, 1).gather(1, t[:, None])[:, 0]
    old = torch.where(lp > -30, lp, -30.0) - torch.randn(n, device="cuda", generator=g) * 0.3
    for bound in (math.log(1.2), math.log(0.8)):
        old = torch.where((lp - old - bound).abs() < 1e-3, old - 4e-3, old)
    weights = (torch.rand(n, device="cuda", generator=g) + 0.1) * weight
    return x, t, mask, dict(old_logps=old.float(), advantages=torch.randn(n, device="cuda", generator=g), weights=weights,
                            ref_logps=None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_rows_of_nothing(sq, dtype, vocab):
    """Used rows of nothing but -inf, alone and beside ordinary ones: entropy and gradient 0, whatever -inf is
    brought to beside others."""
    for temperature in (1.0, 1e3, 1e4, 1e30):
        rows_of_nothing(sq, dtype, vocab, temperature)


def rows_of_nothing(sq, dtype, vocab, temperature):
    settings = dict(entropy_coef=0.05, temperature=temperature)
    x, t, _, s = make(9, vocab, dtype, 3, temperature, masked=0.3)
    empty = torch.tensor([0, 4, 8], device="cuda")
    rest = torch.tensor([1, 2, 3, 5, 6, 7], device="cuda")
    x[empty] = -math.inf
    d, loss, stats, logps, h = got = sq.token_policy_grad(x, t, **s, **settings)
    assert (logps[empty] == -math.inf).all() and not h[empty].any() and not d[empty].any()
    others = {**s, "weights": s["weights"].index_fill(0, empty, 0.0)}
    check(x.index_fill(0, empty, 0.0), t, others, settings, got, rest, loss=False)
    want = sq.token_policy_grad(x, t, **others, **settings)
    assert torch.equal(d[rest], want[0][rest]) and torch.equal(h, want[4])
    assert torch.equal(stats[2], want[2][2])
    # a KL term: without end where the reference has the token, and none of it in the gradient
    ref = torch.full_like(s["weights"], -1.0)
    d, loss, stats, _, h = sq.token_policy_grad(x, t, **{**s, "ref_logps": ref}, **settings, kl_coef=0.1)
    assert not d[empty].any() and not h[empty].any() and loss.item() == math.inf
    for r in (0, 8):   # alone
        one = {k: v[r:r + 1].clone() for k, v in s.items() if v is not None}
        d, loss, stats, logps, h = sq.token_policy_grad(x[r:r + 1], t[r:r + 1].clone(), **one, **settings)
        assert logps.item() == -math.inf and h.item() == 0 and stats[2].item() == 0 and not d.any() and loss.isfinite()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("weight,entropy_coef,masked", [(1.0, 0.0, 0.0), (1.0, 0.05, 0.4), (65536.0, 0.05, 0.0),
                                                        (65536.0, 0.01, 0.4)])
def test_low_temperatures(sq, dtype, vocab, weight, entropy_coef, masked):
    """Where the numbers' distances in octaves, and their products with the entropy's factor, pass fp32's range."""
    for temperature in (1e-30, 1e-20, 1e-12, 4e-9, 1e-6, 1e-3):
        low_temperature(sq, dtype, vocab, temperature, weight, entropy_coef, masked)


def low_temperature(sq, dtype, vocab, temperature, weight, entropy_coef, masked):
    settings = dict(entropy_coef=entropy_coef, temperature=temperature)
    x, t, mask, s = make(8, vocab, dtype, 5, temperature, weight, masked)
    x[3] = -math.inf     # used: nothing in it
    x[5] = math.nan      # unused
    s["weights"][5] = 0.0
    d, loss, stats, logps, h = got = sq.token_policy_grad(x, t, **s, **settings)
    assert logps[3].item() == -math.inf and not h[3].any() and not d[3].any()
    assert not logps[5].any() and not h[5].any() and not d[5].any()
    rest = torch.tensor([0, 1, 2, 4, 6, 7], device="cuda")
    assert not d[rest][mask[rest]].any() and h.isfinite().all() and stats[2].isfinite() and not loss.isnan()
    y = torch.where(x[:, :1].isfinite(), x, 0.0)
    check(y, t, {**s, "weights": s["weights"].index_fill(0, torch.tensor([3], device="cuda"), 0.0)}, settings, got, rest, loss=False)
    # the sums, without the row whose logp has no end
    s["weights"][3] = 0.0
    check(y, t, s, settings, sq.token_policy_grad(x, t, **s, **settings), rest)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("entropy_coef", [0.0, 0.1])
def test_extreme_numbers(sq, dtype, vocab, entropy_coef):
    """Rows of one number, of the type's lowest, with its largest, with NaN and +inf, in every kernel and type."""
    for temperature in (1e-30, 1e-3, 1.0, 1e4, 1e30):
        extreme_numbers(sq, dtype, vocab, temperature, entropy_coef)


def extreme_numbers(sq, dtype, vocab, temperature, entropy_coef):
    settings = dict(entropy_coef=entropy_coef, temperature=temperature)
    x, t, _, s = make(9, vocab, dtype, 6, temperature)
    least, most = torch.finfo(dtype).min, torch.finfo(dtype).max
    x[0, 1:] = -math.inf               # one number
    x[1] = least                       # the lowest, all of it
    x[2] = -math.inf
    x[2, ::2] = least                  # and half of it, the rest masked
    x[3, 1:] = least                   # beside an ordinary one
    x[4, 0] = most                     # the largest beside ordinary and masked ones
    x[4, 1::3] = -math.inf
    x[5, 2] = math.nan
    x[6, 2] = math.inf
    x[7, 1], t[7] = -math.inf, 1       # a masked token
    t[:5] = 0
    s["weights"][8] = 0.0
    s["old_logps"][:5] = -0.1
    s["old_logps"][1:3] = -math.log(vocab) + 0.1
    d, loss, stats, logps, h = got = sq.token_policy_grad(x, t, **s, **settings)
    assert loss.isnan() and stats[2].isnan()
    for r in (5, 6):
        assert logps[r].isnan() and h[r].isnan() and d[r].isnan().all()
    assert logps[0].item() == 0 and h[0].item() == 0 and not d[0, 1:].any()
    assert logps[7].item() == -math.inf and d[7, 1].item() == 0 and not d[8].any() and not h[8].any()
    for r in (0, 2, 4, 7):
        assert not d[r][x[r] == -math.inf].any()
    s["weights"][5:7] = 0.0
    finite = x.nan_to_num(nan=0.0, neginf=-math.inf, posinf=0.0)
    rest = torch.tensor([0, 1, 2, 3, 4], device="cuda")
    check(finite, t, s, settings, got, rest, loss=False)
    # nothing beside the bad rows knows of them
    again = sq.token_policy_grad(x, t, **s, **settings)
    keep = torch.tensor([0, 1, 2, 3, 4, 7, 8], device="cuda")
    assert all(torch.equal(again[k][keep], got[k][keep]) for k in (0, 3, 4))
    assert again[2][:4].isfinite().all()   # (of the old policy's KL row 7 has one without end)
