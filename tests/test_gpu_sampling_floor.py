"""Entries of the least weight: top-p whose cut lies among entries just above 32
octaves below the maximum, each of weight 1 (of 2^31).

With a temperature of float(log2 e) the octaves are the logits' distances
themselves.  top_p = 1 - k 2^-24 leaves 128 k + 1 of the mass out, and u = j 2^-31
draws the j-th unit of mass in index order: the kept entries one by one."""
import math

import numpy as np
import pytest

from test_gpu_sampling import by_definition, settings

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TEMPERATURE = float(np.float32(1.44269504))


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


def row(vocab, upper, lower, seed):
    """The maximum last; `upper` entries 31.9999 octaves below and `lower` 31.999998, each the first of four."""
    x = torch.full((vocab,), -math.inf)
    x[vocab - 1] = 0.0
    at = 4 * torch.from_numpy(np.random.RandomState(seed).permutation(vocab // 4 - 1)[:upper + lower])
    x[at[:upper]] = -31.9999
    x[at[upper:]] = -31.999998
    return x.cuda()


# few rows in shared memory, many read from L2; the cut among a few, at the end of more than 32, and in a long tail
@pytest.mark.parametrize("n", [4, 200])
@pytest.mark.parametrize("vocab", [9000, 131072])
@pytest.mark.parametrize("k,upper,keep", [(8, 20, 10), (8, 20, 1), (8, 40, 40), (23, 40, 25), (23, 500, 500), (8, 20, 30)])
def test_cut_at_the_floor(sq, n, vocab, k, upper, keep):
    left = 128 * k + 1
    lower = left + keep - upper
    if upper + lower >= vocab // 4 - 1:
        pytest.skip("more entries than the row has places for")
    x = row(vocab, upper, lower, 3)
    s = settings(temperature=TEMPERATURE, top_p=1.0 - k * 2.0 ** -24)
    j = np.unique(np.linspace(0, keep + 2, n).round().astype(int))
    j = np.resize(j, n)
    u = torch.tensor(j * 2.0 ** -31, device="cuda", dtype=torch.float32)
    logits = x.expand(n, vocab)
    want, kept = by_definition(logits[:1], u[:1], **s)
    assert kept[0] == keep + 1
    # the kept by index: the upper ones first, then as many of the lower as are left
    up, low = (x == x[x > -31.99995].min()).nonzero()[:, 0], (x == -31.999998).nonzero()[:, 0]
    small = torch.cat([up[:min(upper, keep)], low[:max(0, keep - upper)]]).sort().values.cpu().numpy()
    all_kept = np.append(small, [vocab - 1] * 3)
    for _ in range(5):
        tokens, _ = sq.sample_tokens(logits, u, **s)
        assert np.array_equal(tokens.cpu().numpy(), all_kept[j]), (tokens, all_kept[j])
    assert want[0] == all_kept[0]
