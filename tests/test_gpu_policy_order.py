"""The sums of the policy loss have one order, whatever clusters the GPU has room for."""
import pytest

import test_gpu_policy_loss as over_tokens
import test_gpu_policy_rows as over_rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROWS = dict(kl_coef=0.1, entropy_coef=0.01)


@pytest.fixture()
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    yield sq
    sq.debug_set_fault(0, 0, 0)


def cancelling(n, seed):
    """Weights of both signs and many sizes whose sum is 0: what is left of it is the roundings, which go by the order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    half = torch.randn(n // 2, device="cuda", generator=g) * torch.exp(8 * torch.randn(n // 2, device="cuda", generator=g))
    w = torch.cat([half, -half, torch.zeros(n % 2, device="cuda")])
    return w[torch.randperm(n, device="cuda", generator=g)]


# one group and more of them than any cluster has CTAs; ends inside a chunk; more threads a CTA from 16385 on
@pytest.mark.parametrize("n", [1000, 1025, 5003, 8192, 9001, 16384, 16385, 30001, 65536])
@pytest.mark.parametrize("ctas", [8, 5, 2, 1])
@pytest.mark.parametrize("cancel", [False, True])
def test_smaller_clusters(sq, n, ctas, cancel):
    logps, s = over_tokens.make(n, n, spread=0.5)
    s["weights"][:n // 3] = 0   # whole groups of unused tokens
    if cancel:
        s["weights"] = cancelling(n, n)
    call = dict(kl_coef=0.3, max_ratio=2.0)
    want = sq.policy_loss_grad(logps, **s, **call), sq.policy_loss(logps, **s, **call)
    sq.debug_set_fault(3, ctas)
    got = sq.policy_loss_grad(logps, **s, **call), sq.policy_loss(logps, **s, **call)
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    over_tokens.check(logps, s, call, got[0][1], got[0][2], got[0][0])


@pytest.mark.parametrize("n,vocab", [(3000, 101), (20000, 33), (40, 20011)])
def test_smaller_clusters_behind_rows(sq, n, vocab):
    x, t, s = over_rows.make(n, vocab, torch.bfloat16, 5, ROWS)
    s["weights"] = cancelling(n, n)
    want = sq.token_policy_grad(x, t, **s, **ROWS)
    for ctas in (8, 1):
        sq.debug_set_fault(3, ctas)
        assert all(torch.equal(a, b) for a, b in zip(sq.token_policy_grad(x, t, **s, **ROWS), want))
