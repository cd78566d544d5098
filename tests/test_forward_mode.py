"""Tensors with a forward-mode tangent are refused by the calls that autograd records: it would be lost."""
import pytest

torch = pytest.importorskip("torch")

forward_ad = torch.autograd.forward_ad


def calls(sq, v, t, offsets):
    """The recorded calls by their arguments that may carry a tangent."""
    rest = dict(old_logps=v, advantages=v, weights=v, ref_logps=v)
    yield lambda a: sq.token_logprob(a[:, None].expand(len(v), 5).contiguous(), t), []
    yield lambda a, **kw: sq.policy_loss(a, **{**rest, **kw}), list(rest)
    pairs = dict(ref_logps=v, weights=v)
    yield lambda a, **kw: sq.preference_loss(a, offsets, **{**pairs, **kw}), list(pairs)


@pytest.mark.parametrize("recorded", [False, True])
def test_refused(recorded, device="cpu"):
    import parity_binade_chunked_gb300 as sq
    v = -torch.ones(4, device=device)
    t, offsets = torch.zeros(4, dtype=torch.int64, device=device), torch.tensor([0, 2, 4], device=device)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(v.clone().requires_grad_(recorded), torch.ones_like(v))
        for call, others in calls(sq, v, t, offsets):
            with pytest.raises(sq.SeqsumError, match="forward-mode"):
                call(dual)
            for name in others:
                with pytest.raises(sq.SeqsumError, match=f"forward-mode derivative through {name}"):
                    call(v, **{name: dual})


@pytest.mark.gpu
def test_on_the_gpu():
    """The same there; a tensor without a tangent, and one that was detached, are taken as ever."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    for recorded in (False, True):
        test_refused(recorded, "cuda")
    v = -torch.ones(4, device="cuda")
    t, offsets = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.tensor([0, 2, 4], device="cuda")
    want = [call(v) for call, _ in calls(sq, v, t, offsets)]
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(v.clone(), torch.ones_like(v))
        for (call, _), w in zip(calls(sq, v, t, offsets), want):
            assert all(torch.equal(a, b) for a, b in zip(call(v), w))
            assert all(torch.equal(a, b) for a, b in zip(call(dual.detach()), w))
    # a derivative by functions is refused too
    with pytest.raises(Exception):
        torch.func.jvp(lambda x: sq.preference_loss(x, offsets)[0], (v,), (v,))
