"""The example that runs the operators together: a policy learns which token
each state wants, the same way every time."""
import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_the_policy_learns():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import policy_step
    finally:
        sys.path.pop(0)
    rewards, norms, right = policy_step.train(steps=120, seed=1)
    assert sum(rewards[:5]) / 5 < 0.1 and sum(rewards[-10:]) / 10 > 0.5 and right > 0.6
    assert all(n >= 0 for n in norms) and max(norms) > 0   # (0 where no token of a batch was rewarded)
    again, norms_again, _ = policy_step.train(steps=120, seed=1)
    assert again == rewards and norms_again == norms
