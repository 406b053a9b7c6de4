"""The tied-head example: a training step's gradients against float64 from the same 8-bit values, the
4-bit server against float64 over the values that its codes stand for, and that both run captured."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce
    import tied_head


def _tokens(N, V, seed):
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    t = (V ** torch.rand(N, generator=g, device="cuda:0", dtype=torch.float64) - 1).int().clamp_(0, V - 1)
    y = torch.randint(0, V, (N,), generator=g, device="cuda:0").int()
    t[::9] = -100
    y[::9] = -100
    return t, y


def _plain(m, tokens, labels):
    """Loss and gradients in float64: the forward pass as it is defined, the norm's backward pass from
    the values kept in 8 bits."""
    live = tokens != -100
    t = tokens.clamp(min=0).long()
    x = torch.where(live[:, None], (m.table[t] * torch.tensor(m.scale).float()).bfloat16().double(), 0.0)
    mean = x.mean(1, keepdim=True)
    rstd = 1 / (x.var(1, unbiased=False, keepdim=True) + m.eps).sqrt()
    w, W = m.weight.double(), m.table.bfloat16().double()
    h = ((x - mean) * rstd * w + m.bias.double()).bfloat16().double()
    lp = torch.log_softmax(h @ W.T, 1)
    on = labels != -100
    at = labels.clamp(min=0).long()[:, None]
    loss = -(lp.gather(1, at)[:, 0] * on).sum() / on.sum()
    G = lp.exp()
    G.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=torch.float64))
    G = G * on[:, None] / on.sum()
    dW, dy = G.T @ h, (G @ W).bfloat16().double()
    kept = flce.unpack_e4m3(flce.pack_e4m3(x.float()), dtype=torch.float32).double()
    k = (kept - mean) * rstd
    g = dy * w
    dx = (rstd * (g - g.mean(1, keepdim=True) - k * (g * k).mean(1, keepdim=True))).bfloat16().double()
    dW.index_add_(0, t[live], dx[live] * m.scale)
    return loss, dW, (dy * k).sum(0), dy.sum(0)


@pytest.mark.parametrize("N,V,D", [(1, 50, 64), (300, 1000, 128), (1025, 333, 520)])
def test_gradients_of_a_step(N, V, D):
    torch.manual_seed(N)
    m = tied_head.TiedHead(V, D)
    m.weight.normal_(1, 0.1)
    m.bias.normal_(0, 0.1)
    t, y = _tokens(max(N, 2), V, N)
    if N == 1:
        t, y = t[1:].clone(), y[1:].clone()
    loss, *got = m.gradients(t, y)
    want_loss, *want = _plain(m, t, y)
    # G, dH and dx are rounded to bf16, h as well: 2^-8 each of their own; h's other roundings of ties move it by
    # as much again. In norms, of each gradient.
    u = 2.0 ** -8
    assert abs(float(loss) - float(want_loss)) <= 4 * u * (1 + abs(float(want_loss)))
    for a, b in zip(got, want):
        assert float((a.double() - b).norm()) <= 6 * u * float(b.norm())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("N", [1, 40, 300])
def test_server(fmt, N):
    torch.manual_seed(2)
    m = tied_head.TiedHead(2001, 264)
    s = m.server(fmt)
    t = torch.randint(0, 2001, (N,), device="cuda:0").int()
    r = s.next(t, top_k=3)
    x = flce.embedding(m.table, t, scale=m.scale, dtype=torch.bfloat16)
    h = flce.dequantize_fp4(flce.quantize_fp4(flce.layer_norm(x, m.weight, m.bias).y, format=fmt)).double()
    z = h @ flce.dequantize_fp4(s.head).double().T
    lp = torch.log_softmax(z, 1)
    # fp32 sums of at most 264 products in steps of 64, then the log probabilities': 2^-20 of the sums of magnitudes
    size = (h.abs() @ flce.dequantize_fp4(s.head).double().abs().T).amax(1, keepdim=True)
    assert bool(((r.top_logprob.double() - lp.gather(1, r.top_id.long())).abs() <= 2.0 ** -18 * (1 + size)).all())
    assert bool((lp.topk(3, 1).values - r.top_logprob.double() <= 2.0 ** -18 * (1 + size)).all())


def test_a_captured_step_and_a_captured_server():
    torch.manual_seed(4)
    m = tied_head.TiedHead(700, 128)
    t, y = _tokens(400, 700, 4)
    start = [p.clone() for p in (m.table, m.weight, m.bias)]
    want = [(float(loss), float(norm)) for loss, norm in (m.step(t, y) for _ in range(3))]
    after = [p.clone() for p in (m.table, m.weight, m.bias)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, norm = m.step(t, y)
    for p, a in zip((m.table, m.weight, m.bias), start):
        p.copy_(a)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert (float(loss), float(norm)) == want[k]
    assert all(torch.equal(p, a) for p, a in zip((m.table, m.weight, m.bias), after))
    s = m.server()
    token = torch.tensor([5], dtype=torch.int32, device="cuda:0")
    s.next(token)
    serve = torch.cuda.CUDAGraph()
    with torch.cuda.graph(serve):
        r = s.next(token)
    for k in (5, 17, 600):
        token.fill_(k)
        serve.replay()
        torch.cuda.synchronize()
        eager = s.next(torch.tensor([k], dtype=torch.int32, device="cuda:0"))
        assert torch.equal(r.top_id, eager.top_id) and torch.equal(r.top_logprob, eager.top_logprob)


def test_it_runs():
    model, successor, losses = tied_head.train(steps=3, tokens=300, vocab=500, hidden=64)
    assert len(losses) == 3 and all(bool(torch.isfinite(v).all()) for v in losses)
    assert model.server("mxfp4").next(successor[:7].contiguous()).top_id.shape == (7, 4)
