"""A tied table at both ends of a model, trained, and then served in 4 bits.

The table is the embedding and the head:

    x = scale table[tokens],  h = layer_norm(x),  loss = linear cross-entropy(h, table, next tokens)

(the model between them is left out: what stands here are the ends). A training step keeps the
norm's input in 8 bits for its backward pass, and adds the embedding's gradient, by the tokens
that there are, onto the head's dense one, so that no second gradient of the table's size exists.
A server turns the table into 4 bits once; a token then costs its lookup, the norm of one row, and
the product with the 4-bit head, over whose logits the likely tokens and their log
probabilities are taken.

    python examples/tied_head.py [--steps 40] [--tokens 2048] [--vocab 4000] [--hidden 512]

trains it to continue fixed cycles of tokens and prints the loss, and how often the 4-bit head
continues them.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_cross_entropy_flce_gb300 as flce  # noqa: E402


class TiedHead:
    """fp32 parameters: the table [vocab, hidden], and the norm's weight and bias."""

    def __init__(self, vocab: int, hidden: int, device="cuda:0", eps: float = 1e-5):
        self.table = torch.randn(vocab, hidden, device=device) * hidden ** -0.5
        self.weight = torch.ones(hidden, device=device)
        self.bias = torch.zeros(hidden, device=device)
        self.scale, self.eps = hidden ** 0.5, eps

    def gradients(self, tokens, labels):
        """(loss [1], gradients of the table, the norm's weight and its bias) of next tokens `labels`
        (int32 [N], -100: none) after `tokens` (int32 [N], -100: padding)."""
        x = flce.embedding(self.table, tokens, scale=self.scale, dtype=torch.bfloat16)
        r, kept = flce.layer_norm_packed(x, self.weight, self.bias, eps=self.eps)
        head = flce.forward_backward(r.y, self.table.bfloat16(), labels, dw_dtype="float32")
        dx, dweight, dbias = flce.layer_norm_packed_backward(head.dH, kept, self.weight, r)
        flce.embedding_backward(dx, tokens, self.table.shape[0], scale=self.scale, out=head.dW, accumulate=True)
        return head.loss, head.dW, dweight, dbias

    def step(self, tokens, labels, lr: float = 0.5, max_norm: float = 1.0):
        """One clipped gradient step; (loss, gradient norm), on the GPU: nothing waits for it."""
        loss, *grads = self.gradients(tokens, labels)
        norm = flce.clip_grads(grads, max_norm)
        for p, g in zip((self.table, self.weight, self.bias), grads):
            p.add_(g, alpha=-lr)
        return loss, norm

    def server(self, format: str = "nvfp4") -> "Server":
        return Server(self, format)


class Server:
    """The same in 4 bits for the head: next tokens of given ones."""

    def __init__(self, model: TiedHead, format: str):
        self.model, self.format = model, format
        self.head = flce.quantize_fp4(model.table, format=format)

    def next(self, tokens, top_k: int = 4) -> flce.TokenLogprobs:
        """The top_k likeliest tokens after each of `tokens` (int32 [N]), with log probabilities."""
        m = self.model
        x = flce.embedding(m.table, tokens, scale=m.scale, dtype=torch.bfloat16)
        h = flce.layer_norm(x, m.weight, m.bias, eps=m.eps).y
        logits = flce.linear_fp4(flce.quantize_fp4(h, format=self.format), self.head, dtype=torch.float32)
        return flce.token_logprobs(logits, None, top_k=top_k)


def train(steps=40, tokens=2048, vocab=4000, hidden=512, seed=0, report=None):
    """A model taught one successor for each token; (model, successors, losses)."""
    torch.manual_seed(seed)
    model = TiedHead(vocab, hidden)
    successor = torch.randperm(vocab, device="cuda:0").int()
    losses = []
    for step in range(steps):
        t = torch.randint(0, vocab, (tokens,), device="cuda:0").int()
        loss, _ = model.step(t, successor[t.long()].contiguous())
        losses.append(loss.clone())
        if report and step % 10 == 0:
            report(f"step {step:4d}  loss {float(losses[-1]):.3f}")
    return model, successor, losses


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, value in (("steps", 40), ("tokens", 2048), ("vocab", 4000), ("hidden", 512)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    model, successor, losses = train(a.steps, a.tokens, a.vocab, a.hidden, report=print)
    t = torch.arange(min(a.vocab, 256), device="cuda:0").int()
    for fmt in flce.FP4_FORMATS:
        r = model.server(fmt).next(t)
        right = int((r.top_id == successor[t.long()][:, None]).any(1).sum())
        print(f"{fmt}: the successor is among the four likeliest of {right} of {len(t)} tokens")
