"""Sampling where a cluster takes several rows one after another through its
buffers in shared memory: buffers are refilled, barriers and boxes come around,
rows of unlike settings follow each other.  (Calls of many rows of more than 66
steps of 32 vectors read them from L2 instead: these are of fewer steps, or of
fewer rows than half the multiprocessors.)  Tokens against the definition."""
import math

import numpy as np
import pytest

from test_gpu_sampling import by_definition, settings
from test_gpu_sampling_shapes import rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


def of_each_row(n):
    i = torch.arange(n, device="cuda")
    return dict(temperature=torch.where(i % 5 == 0, 0.0, 0.5 + (i % 7) / 6.0).float(),
                top_k=torch.where(i % 3 == 0, i % 100, 0).int(),
                top_p=torch.where(i % 4 == 1, 0.9, 1.0).float(), min_p=torch.where(i % 11 == 2, 0.05, 0.0).float())


# one CTA a row, some ten rows each; then eight CTAs a row, two to four rows each, of one and of two CTAs an SM
@pytest.mark.parametrize("n,vocab,dtype", [(3000, 2001, torch.float32), (3000, 5003, torch.bfloat16),
                                           (75, 150001, torch.bfloat16), (75, 70001, torch.float32),
                                           (75, 131001, torch.float16)])
@pytest.mark.parametrize("kind", ["zipf", "normal"])
def test_several_rows_a_cluster(sq, n, vocab, dtype, kind):
    x = rows(kind, n, vocab, 5).to(dtype)
    i = torch.arange(n, device="cuda")
    x[i % 17 == 5] = -math.inf
    u = torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    for s in (of_each_row(n), settings(), settings(top_k=50), settings(top_p=0.95), settings(top_k=700, top_p=0.8),
              settings(temperature=0.0), settings(min_p=0.02)):
        tokens, logps = sq.sample_tokens(x, u, **s)
        want, _ = by_definition(x, u, **s)
        assert np.array_equal(tokens.cpu().numpy(), want), s
        for _ in range(3):   # and the same whenever the CTAs meet
            again = sq.sample_tokens(x, u, **s)
            assert torch.equal(again[0], tokens) and torch.equal(again[1], logps)
