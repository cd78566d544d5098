"""Policy-gradient steps on a small linear policy, with the library's operators
from the logits to the clipped update:

  logits -> sample_tokens -> rewards -> token_logprob_grad -> gradients of the
  parameters -> TensorList.clip -> step

The policy sees one of `states` vectors and is rewarded for one token a state;
after some steps it gives that token.  All randomness is drawn beforehand from
a seed, and every sum of the operators has defined bits.

    python examples/policy_step.py [--steps 60] [--seed 0]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def train(steps=60, seed=0, states=16, hidden=64, vocab=101, batch=512, max_norm=0.03, rate=2.0):
    """Returns the mean reward of each step (a list) and the norms before clipping."""
    import torch

    import parity_binade_chunked_gb300 as sq

    g = torch.Generator(device="cuda").manual_seed(seed)
    features = torch.randn(states, hidden, device="cuda", generator=g) / hidden ** 0.5
    wanted = torch.randint(0, vocab, (states,), device="cuda", generator=g)
    weight = torch.zeros(hidden, vocab, device="cuda")
    bias = torch.zeros(vocab, device="cuda")
    grads = [torch.empty_like(weight), torch.empty_like(bias)]
    rewards, norms = [], []
    with sq.TensorList(grads) as gradients:
        for _ in range(steps):
            state = torch.randint(0, states, (batch,), device="cuda", generator=g)
            x = features[state]
            logits = x @ weight + bias
            u = torch.rand(batch, device="cuda", generator=g)
            tokens, _ = sq.sample_tokens(logits, u, temperature=1.0)
            reward = (tokens == wanted[state]).float()
            advantage = (reward - reward.mean()) / batch
            # the loss is -(advantage * logp).sum(): its gradient with respect to the logits, in their place
            dlogits, _, _ = sq.token_logprob_grad(logits, tokens, -advantage, out=logits)
            torch.matmul(x.t(), dlogits, out=grads[0])
            torch.sum(dlogits, dim=0, out=grads[1])
            norms.append(gradients.clip(max_norm, out=torch.empty(1, device="cuda")))
            weight.sub_(grads[0], alpha=rate * batch ** 0.5)
            bias.sub_(grads[1], alpha=rate)
            rewards.append(reward.mean())
    # greedy answers of the trained policy
    tokens, _ = sq.sample_tokens(features @ weight + bias, torch.zeros(states, device="cuda"), temperature=0.0)
    right = (tokens == wanted).float().mean().item()
    return [r.item() for r in rewards], [n.item() for n in norms], right


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    rewards, norms, right = train(a.steps, a.seed)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  reward {rewards[i]:.3f}  gradient norm {norms[i]:.4f}")
    print(f"mean reward of the last steps {sum(rewards[-5:]) / len(rewards[-5:]):.3f}, greedy answers right {right:.2f}")


if __name__ == "__main__":
    main()
