"""Sampling from rows of many shapes against its integer definition (tokens
equal): flat and steep rows, long ties, values sorted along the row, rows whose
every eighth value is unlike the others (a sample of the row misleads), large
k, rows split over one to eight CTAs and kept in small and large buffers."""
import math

import numpy as np
import pytest

from test_gpu_sampling import by_definition, settings

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


def rows(kind, n, vocab, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, vocab, device="cuda", generator=g)
    i = torch.arange(vocab, device="cuda")
    if kind == "flat":
        return x * 0.01
    if kind == "normal":
        return x
    if kind == "steep":
        return x * 8
    if kind == "zipf":
        return torch.empty(n, vocab, device="cuda").exponential_(1.0, generator=g) * 1.3 + x * 0.7
    if kind == "sorted":
        return x.sort(dim=1, descending=True).values * 2
    if kind == "rising":
        return x.sort(dim=1).values * 2
    if kind == "coarse":            # long ties
        return (x * 2).round()
    if kind == "eighths":           # the first of each eight is unlike the rest
        return torch.where(i % 8 == 0, x * 0.1 - 6.0, x)
    if kind == "eighths up":
        return torch.where(i % 8 == 0, x * 0.1 + 6.0, x)
    if kind == "half masked":       # a padded vocabulary
        return torch.where(i > vocab // 2 + 3, -math.inf, x * 3)
    if kind == "few":               # all but some masked
        return torch.where(torch.rand(n, vocab, device="cuda", generator=g) < 0.9995, -math.inf, x)
    raise ValueError(kind)


KINDS = ["flat", "normal", "steep", "zipf", "sorted", "rising", "coarse", "eighths", "eighths up", "half masked", "few"]
FILTERS = [dict(), dict(top_k=50), dict(top_k=2000), dict(top_p=0.9), dict(top_p=0.99, temperature=1.5), dict(top_p=0.3),
           dict(top_k=300, top_p=0.7), dict(top_k=5000, top_p=0.95), dict(min_p=0.1), dict(top_p=0.8, min_p=0.01)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("vocab,dtype", [(9001, torch.float32), (20001, torch.bfloat16), (70001, torch.float16),
                                         (131077, torch.bfloat16), (131072, torch.float32)])
def test_shapes(sq, kind, vocab, dtype):
    n = 5
    x = rows(kind, n, vocab, KINDS.index(kind)).to(dtype)
    x[:, 3] = x[:, 3].clamp(min=-1.0)      # something is left in every row
    u = torch.tensor([0.0, 0.3, 0.7, 0.99, 1.0 - 2.0 ** -24], device="cuda")
    for f in FILTERS:
        s = settings(**f)
        tokens, logps = sq.sample_tokens(x, u, **s)
        want, _ = by_definition(x, u, **s)
        assert np.array_equal(tokens.cpu().numpy(), want), (kind, f, tokens, want)
        assert logps.isfinite().all() and (logps <= 1e-6).all()


@pytest.mark.parametrize("vocab,dtype", [(20001, torch.bfloat16), (140001, torch.float32), (190001, torch.float16)])
def test_more_rows_than_run_at_once(sq, vocab, dtype):
    """Several rows a cluster, of settings in turn, so that buffers and boxes come around."""
    n = 700 if vocab < 30000 else 130
    x = rows("zipf", n, vocab, 3).to(dtype)
    g = torch.Generator(device="cuda").manual_seed(4)
    u = torch.rand(n, device="cuda", generator=g)
    i = torch.arange(n, device="cuda")
    x[i % 17 == 5] = -math.inf
    s = dict(temperature=torch.where(i % 5 == 0, 0.0, 0.5 + (i % 7) / 6.0).float(),
             top_k=torch.where(i % 3 == 0, i % 100, 0).int(),
             top_p=torch.where(i % 4 == 1, 0.9, 1.0).float(), min_p=torch.where(i % 11 == 2, 0.05, 0.0).float())
    tokens, _ = sq.sample_tokens(x, u, **s)
    want, _ = by_definition(x, u, **s)
    assert np.array_equal(tokens.cpu().numpy(), want)
    for f in (dict(), dict(temperature=0.0), dict(min_p=0.02), dict(top_p=0.95)):
        s = settings(**f)
        tokens, _ = sq.sample_tokens(x, u, **s)
        assert np.array_equal(tokens.cpu().numpy(), by_definition(x, u, **s)[0]), f
