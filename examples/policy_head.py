"""A policy head trained and sampled with the operators around the language-model head.

The head is a final layer norm and a vocabulary projection. One training step is a policy
gradient over sampled tokens with an entropy bonus:

    h = layer_norm(x),  (logprob, entropy) of the sampled tokens under softmax(h W^T / T)
    loss = -mean(exp(logprob - logprob when sampled) advantage) - beta mean(entropy)

then the gradients are clipped by their global norm and the parameters moved. The [N, V]
logits exist in no training step. Sampling takes one position of each sequence at a time: the
norm of a few rows, and their most likely tokens with their log probabilities straight from
the hidden states, of which one is drawn.

    python examples/policy_head.py [--steps 60] [--tokens 2048] [--vocab 2000] [--hidden 256]

trains it on a task with one right token per context and prints the reward as it goes.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_cross_entropy_flce_gb300 as flce  # noqa: E402


class PolicyHead(torch.nn.Module):
    """Layer norm and vocabulary projection: fp32 parameters, bf16 operands."""

    def __init__(self, hidden: int, vocab: int, temperature: float = 1.0, device="cuda:0"):
        super().__init__()
        self.norm = flce.FusedLayerNorm(hidden, device=device, dtype=torch.float32)
        self.weight = torch.nn.Parameter(torch.randn(vocab, hidden, device=device) * hidden ** -0.5)
        self.temperature = temperature

    def forward(self, x, tokens):
        """(logprob, entropy) of tokens [...] at the positions x [..., hidden], bf16."""
        logprob, entropy, _ = flce.fused_linear_token_logprobs(
            self.norm(x), self.weight.bfloat16(), tokens, temperature=self.temperature)
        return logprob, entropy

    @torch.no_grad()
    def score(self, x, tokens, top_k: int = 0) -> flce.TokenLogprobs:
        """Log probabilities, entropies and top_k alternatives of given tokens, without gradients."""
        h = flce.layer_norm(x, self.norm.weight, self.norm.bias, eps=self.norm.eps).y
        return flce.linear_token_logprobs(h, self.weight.bfloat16(), tokens, top_k=top_k,
                                          temperature=self.temperature)

    @torch.no_grad()
    def sample(self, x, top_k: int = 8, generator=None):
        """Draws a token per row of x among its top_k most likely ones: (tokens int32, their log
        probabilities under the whole distribution)."""
        h = flce.layer_norm(x, self.norm.weight, self.norm.bias, eps=self.norm.eps).y
        r = flce.linear_token_logprobs(h, self.weight.bfloat16(), None, top_k=top_k,
                                       temperature=self.temperature)
        pick = torch.multinomial(r.top_logprob.exp(), 1, generator=generator)
        return r.top_id.gather(1, pick)[:, 0], r.top_logprob.gather(1, pick)[:, 0]


def policy_step(head, x, tokens, sampled_logprob, advantage, *, beta=0.01, max_norm=1.0, lr=0.5):
    """One clipped gradient step; returns (loss, gradient norm) as tensors: nothing waits for
    the GPU."""
    logprob, entropy = head(x, tokens)
    loss = -((logprob - sampled_logprob).exp() * advantage).mean() - beta * entropy.mean()
    head.zero_grad(set_to_none=True)
    loss.backward()
    params = [p for p in head.parameters() if p.grad is not None]
    norm = flce.clip_grads([p.grad for p in params], max_norm)
    with torch.no_grad():
        for p in params:
            p.add_(p.grad, alpha=-lr)
    return loss.detach(), norm


def train(steps=60, tokens=2048, vocab=2000, hidden=256, contexts=32, seed=0, report=None):
    """Rewards per step of the toy task: one right token per context."""
    torch.manual_seed(seed)
    g = torch.Generator(device="cuda:0").manual_seed(seed + 1)   # not the parameters' draws
    head = PolicyHead(hidden, vocab)
    states = torch.randn(contexts, hidden, device="cuda:0", generator=g).bfloat16()
    right = torch.randint(0, vocab, (contexts,), device="cuda:0", generator=g).int()
    with torch.no_grad():   # the right token starts among the likely ones
        head.weight[right.long()] += 0.25 * hidden ** -0.5 * states.float()
    rewards = []
    for step in range(steps):
        c = torch.randint(0, contexts, (tokens,), device="cuda:0", generator=g)
        x = states[c]
        drawn, logprob = head.sample(x, top_k=32, generator=g)
        reward = (drawn == right[c]).float()
        policy_step(head, x, drawn, logprob, reward - reward.mean())
        rewards.append(float(reward.mean()))
        if report and step % 10 == 0:
            report(f"step {step:4d}  reward {rewards[-1]:.3f}")
    return head, states, right, rewards


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, value in (("steps", 60), ("tokens", 2048), ("vocab", 2000), ("hidden", 256)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    head, states, right, _ = train(a.steps, a.tokens, a.vocab, a.hidden, report=print)
    r = head.score(states, right, top_k=3)
    print(f"the right token's mean log probability {float(r.logprob.mean()):.3f}, "
          f"mean entropy {float(r.entropy.mean()):.3f}, "
          f"first in {int((r.top_id[:, 0] == right).sum())} of {len(right)} contexts")
