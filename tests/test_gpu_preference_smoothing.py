"""Label smoothing over its whole range: the loss and its gradient where one label has next to all of the weight.

Tolerances: z is rounded once, 2^-24 |z|, which moves a softplus by that times its
sigmoid; a sigmoid s = e^-|z| / (1 + e^-|z|) or 1 / (1 + e^-|z|) is off by 2^-22 of
itself and by 2^-23 |z| s (1 - s); a softplus by 2^-22; the settings by 2^-24 each, and
three more roundings of each part and of the sum.  One more for the mean, its share and
the gradient."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


# pairs_kernel, and many_pairs_kernel
@pytest.mark.parametrize("pairs", [1, 7, 40, 700])
@pytest.mark.parametrize("smoothing", [0.0, 1e-4, 0.1, 0.5, 0.9, 0.999, 1 - 1e-6, 1.0])
@pytest.mark.parametrize("average", [False, True])
def test_smoothing(sq, pairs, smoothing, average):
    beta = 0.5
    for z in (-60.0, -20.0, -9.3, -2.0, -0.01, 0.0, 0.7, 5.0, 17.0, 40.0):
        between = z / beta
        logps = torch.zeros(2 * pairs, device="cuda")
        logps[0::2] = between
        loss, scores, *_ = sq.preference_loss(logps, torch.arange(2 * pairs + 1, device="cuda"), beta=beta, smoothing=smoothing,
                                              average=average)
        d, loss2, _ = sq.preference_loss_grad(logps, torch.arange(2 * pairs + 1, device="cuda"), beta=beta, smoothing=smoothing,
                                              average=average)
        assert torch.equal(loss, loss2)
        y = beta * logps[0].double().item()
        e = math.exp(-abs(y))
        plus, minus = (1 / (1 + e), e / (1 + e)) if y >= 0 else (e / (1 + e), 1 / (1 + e))   # sigma(y), sigma(-y)
        soft_minus, soft_plus = max(-y, 0.0) + math.log1p(e), max(y, 0.0) + math.log1p(e)
        want = (1 - smoothing) * soft_minus + smoothing * soft_plus
        off = 2.0 ** -20 * want + 2.0 ** -23 * abs(y) * ((1 - smoothing) * minus + smoothing * plus)
        assert abs(loss.item() - want) <= off, (z, loss.item(), want)
        slope = beta * (smoothing * plus - (1 - smoothing) * minus) / pairs
        parts = beta * (smoothing * plus + (1 - smoothing) * minus) / pairs
        off = 2.0 ** -20 * parts + 2.0 ** -22 * abs(y) * beta * plus * minus / pairs
        assert (d[0::2].double() - slope).abs().max().item() <= off, (z, d[0].item(), slope)
        assert (d[1::2].double() + slope).abs().max().item() <= off
