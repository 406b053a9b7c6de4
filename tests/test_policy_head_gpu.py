"""The policy-head example: its gradients against float64 autograd over the plain formulas, and
that it learns."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
if torch.cuda.is_available():
    import policy_head


def _plain(head, x, tokens, sampled, advantage, beta):
    """Loss and gradients in float64 (weight rounded to bf16 as the head rounds it)."""
    p = {n: (t.bfloat16() if n == "weight" else t).detach().double().requires_grad_()
         for n, t in head.named_parameters()}
    xd = x.double()
    c = xd - xd.mean(1, keepdim=True)
    h = c / (c.square().mean(1, keepdim=True) + head.norm.eps).sqrt() * p["norm.weight"] + p["norm.bias"]
    lp = torch.log_softmax(h @ p["weight"].T / head.temperature, 1)
    logprob = lp.gather(1, tokens.long()[:, None])[:, 0]
    entropy = -(lp.exp() * lp).sum(1)
    loss = -((logprob - sampled.double()).exp() * advantage.double()).mean() - beta * entropy.mean()
    loss.backward()
    size = (h.detach().abs() @ p["weight"].detach().abs().T).max()
    return float(loss.detach()), {n: t.grad for n, t in p.items()}, float(size)


@pytest.mark.parametrize("N,D,V,temperature", [(1, 64, 100, 1.0), (200, 64, 1001, 0.7), (513, 136, 333, 1.5)])
def test_gradients_of_a_step(N, D, V, temperature):
    torch.manual_seed(N)
    head = policy_head.PolicyHead(D, V, temperature)
    x = torch.randn(N, D, device="cuda:0").bfloat16()
    tokens = torch.randint(0, V, (N,), device="cuda:0").int()
    sampled = head.score(x, tokens).logprob + 0.1 * torch.randn(N, device="cuda:0")
    advantage = torch.randn(N, device="cuda:0")
    want_loss, want, size = _plain(head, x, tokens, sampled, advantage, 0.01)
    before = {n: t.detach().clone() for n, t in head.named_parameters()}
    total = torch.stack([g.norm() for g in want.values()]).norm()
    loss, norm = policy_head.policy_step(head, x, tokens, sampled, advantage, max_norm=1e9, lr=1.0)
    # h rounded once (2^-8), which moves a logit by 2^-8 size / T at most, and a probability or
    # its gradient by twice that of itself; dz, dh and dx or dW are rounded once each
    u = 2.0 ** -8
    bound = 4 * u + 3 * u * size / temperature
    assert abs(float(loss) - want_loss) <= bound * float((advantage.abs() * 2).mean() + 0.1)
    assert abs(float(norm) - float(total)) <= bound * float(total)
    for n, t in head.named_parameters():
        g = (before[n] - t.detach()).double()
        assert float((g - want[n]).norm()) <= bound * float(total), n
    # clipped: the same direction, the asked length
    head2 = policy_head.PolicyHead(D, V, temperature)
    head2.load_state_dict(before)
    policy_head.policy_step(head2, x, tokens, sampled, advantage, max_norm=float(norm) / 4, lr=0.0)
    clipped = torch.stack([p.grad.double().norm() for p in head2.parameters()]).norm()
    assert abs(float(clipped) - float(norm) / 4) <= 1e-4 * float(norm)


def test_sampled_log_probabilities_are_those_scored():
    torch.manual_seed(3)
    head = policy_head.PolicyHead(128, 1000)
    x = torch.randn(7, 128, device="cuda:0").bfloat16()
    tokens, logprob = head.sample(x, top_k=5)
    r = head.score(x, tokens, top_k=5)
    # sampling's logits are rounded to bf16 (|z| < 8), scoring's are not
    assert float((r.logprob - logprob).abs().max()) <= 2 * 8 * 2.0 ** -8
    assert bool((r.top_logprob[:, 1:] <= r.top_logprob[:, :-1]).all())


def test_it_learns():
    _, _, _, rewards = policy_head.train(steps=60, tokens=1024, vocab=500, hidden=128)
    first, last = sum(rewards[:5]) / 5, sum(rewards[-5:]) / 5
    assert last > first


def test_a_captured_step_repeats_the_eager_one():
    torch.manual_seed(5)
    N, D, V = 300, 128, 777
    head = policy_head.PolicyHead(D, V)
    x = torch.randn(N, D, device="cuda:0").bfloat16()
    tokens = torch.randint(0, V, (N,), device="cuda:0").int()
    sampled = head.score(x, tokens).logprob
    advantage = torch.randn(N, device="cuda:0")
    start = {n: t.detach().clone() for n, t in head.named_parameters()}
    want = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # no eager graph of the leaves is left when the capture begins
        for _ in range(3):
            loss, norm = policy_head.policy_step(head, x, tokens, sampled, advantage, max_norm=0.1)
            want.append((float(loss), float(norm)))
    torch.cuda.current_stream().wait_stream(side)
    eager = {n: t.detach().clone() for n, t in head.named_parameters()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, norm = policy_head.policy_step(head, x, tokens, sampled, advantage, max_norm=0.1)
    head.load_state_dict(start)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert (float(loss), float(norm)) == want[k]
    assert all(torch.equal(t.detach(), eager[n]) for n, t in head.named_parameters())
