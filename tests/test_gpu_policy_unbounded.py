"""The policy loss without bounds of the ratio, where the ratio passes fp32's range."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

OPEN = dict(clip_low=1.0, clip_high=math.inf)


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


@pytest.mark.parametrize("n", [1, 2, 7, 5003, 70001])
@pytest.mark.parametrize("distance", [50.0, 89.0, 200.0, math.inf])
def test_no_advantage_no_loss(sq, n, distance):
    """0 times any ratio is 0, in the loss and in the gradient; other advantages have a loss without end from e^89 on."""
    logps = torch.full((n,), -1.0, device="cuda")
    old, w = logps - distance, torch.ones(n, device="cuda")
    for zero in (0.0, -0.0):
        a = torch.full((n,), zero, device="cuda")
        d, loss, stats = sq.policy_loss_grad(logps, old, a, w, **OPEN)
        assert loss.item() == 0 and stats[0].item() == 0 and not d.any()
        leaf = logps.clone().requires_grad_()
        sq.policy_loss(leaf, old, a, w, **OPEN)[0].backward()
        assert not leaf.grad.any()
    for sign in (1.0, -1.0):
        a = torch.where(torch.arange(n, device="cuda") == n // 2, sign, 0.0)
        d, loss, _ = sq.policy_loss_grad(logps, old, a, w, **OPEN)
        want = -sign * (math.exp(distance) if distance < 88 else math.inf)
        assert loss.item() == pytest.approx(want, rel=1e-5) and d[n // 2].item() == pytest.approx(want, rel=1e-5)
        d[n // 2] = 0
        assert not d.any()
    nan = torch.full((n,), math.nan, device="cuda")
    assert sq.policy_loss(logps, old, nan, w, **OPEN)[0].isnan() and sq.policy_loss(nan, old, 0 * w, w, **OPEN)[0].isnan()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [101, 5003, 50001])
def test_rows(sq, dtype, vocab):
    x = torch.randn(3, vocab, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dtype)
    t, w = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.ones(3, device="cuda")
    d, loss, stats, logps, _ = sq.token_policy_grad(x, t, torch.full((3,), -200.0, device="cuda"), 0 * w, w, **OPEN)
    assert loss.item() == 0 and stats[0].item() == 0 and not d.any() and logps.isfinite().all()


@pytest.mark.parametrize("clip_high", [1e39, 1e300])
def test_bounds_beyond_fp32(sq, clip_high):
    """Such a bound is none: 0 times it is 0."""
    logps = torch.full((5,), -1.0, device="cuda")
    old, w, a = logps - 800.0, torch.ones(5, device="cuda"), torch.zeros(5, device="cuda")
    d, loss, stats = sq.policy_loss_grad(logps, old, a, w, clip_high=clip_high, max_ratio=clip_high)
    assert loss.item() == 0 and stats[3].item() == 0 and not d.any()
    d, loss, _ = sq.policy_loss_grad(logps, old, a + 1, w, clip_high=clip_high)
    assert loss.item() == -math.inf and (d == -math.inf).all()
