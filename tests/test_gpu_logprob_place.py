"""What the bits of a row's log-probabilities and gradient go by: its numbers
and its address modulo 16, not the other rows, the batch or the stride.  At
another place within 16 bytes they are held to the tolerance of their sums."""
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


def placed(row, n, at, stride, place):
    """`row` as row `at` of n random ones of the given stride, so that it begins `place` numbers past 16 bytes."""
    per = 16 // row.element_size()
    memory = torch.randn(n * stride + 4 * per, device="cuda").to(row.dtype)
    first = (place - at * stride) % per
    rows = memory[first:].as_strided((n, row.shape[0]), (stride, 1))
    rows[at] = row
    assert rows[at].data_ptr() % 16 == place * row.element_size()
    return rows


@pytest.mark.parametrize("dtype", logprob.DTYPES)
@pytest.mark.parametrize("vocab", [33, 1501, 6001, 50001, 131077, 600001])   # a warp, one CTA, several, beyond the buffers
def test_place(sq, dtype, vocab):
    x, t, a = logprob.make(1, vocab, dtype, vocab)
    for place in (0, 1, 3):
        first = None
        for n, at, gap in ((1, 0, 0), (5, 3, 7), (5, 0, 16), (40, 39, 9), (300, 170, 1)):
            if n * vocab > 2 ** 26:
                continue
            rows = placed(x[0], n, at, vocab + gap, place)
            tokens, dlogps = t.expand(n).contiguous(), a.expand(n).contiguous()
            logps, lses = sq.token_logprob(rows, tokens)
            d, logps2, lses2 = sq.token_logprob_grad(rows, tokens, dlogps)
            assert torch.equal(logps, logps2) and torch.equal(lses, lses2)
            got = logps[at:at + 1], lses[at:at + 1], d[at:at + 1].clone()
            if first is None:
                first = got
                logprob.check(x, t, a, *got)
            assert all(torch.equal(p, q) for p, q in zip(got, first)), (place, n, at)
