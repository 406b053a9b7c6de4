"""The float64 definitions in oracle/head_ops.py against closed forms and central
differences: uniform and one-hot rows, masked rows, the gradients of log probability,
entropy, log-sum-exp and layer norm."""
import math

import numpy as np
import pytest

from oracle import head_ops as ho


def _rng(seed):
    return np.random.Generator(np.random.Philox(np.random.SeedSequence([seed, 7])))


def test_uniform_and_one_hot_rows():
    z = np.zeros((2, 50))
    z[1, 7] = 800.0
    r = ho.token_logprobs(z, [3, 7], top_k=3)
    assert r["logprob"] == pytest.approx([-math.log(50), 0.0], abs=1e-300)
    assert r["entropy"][0] == pytest.approx(math.log(50), rel=1e-14)
    assert abs(r["entropy"][1]) < 1e-300
    assert r["top_id"].tolist() == [[0, 1, 2], [7, 0, 1]]


def test_masked_rows():
    z = np.full((3, 6), -np.inf)
    z[1, 4] = 1.5
    z[2, [1, 3]] = [0.0, np.nan]
    r = ho.token_logprobs(z, [0, 4, 1], top_k=2)
    assert r["lse"][0] == -np.inf and r["logprob"][0] == -np.inf and r["entropy"][0] == 0
    assert r["lse"][1] == 1.5 and r["logprob"][1] == 0 and r["entropy"][1] == 0
    assert r["top_id"].tolist()[:2] == [[-1, -1], [4, -1]]
    assert np.isnan(r["lse"][2]) and np.isnan(r["top_logprob"][2]).all()
    g = ho.token_logprobs_grad(z[:2], [0, 4], [1.0, 1.0], [1.0, 1.0], [0.0, 0.0])
    assert not g.any()


@pytest.mark.parametrize("temperature", [1.0, 0.6])
def test_gradient_by_differences(temperature):
    g = _rng(1)
    z = g.standard_normal((4, 9)) * 2
    y = np.array([2, -100, 8, 0])
    a, b, c = g.standard_normal((3, 4))
    G = ho.token_logprobs_grad(z, y, a, b, c, temperature=temperature)

    def f(zz):
        r = ho.token_logprobs(zz, y, temperature=temperature)
        return float(a @ r["logprob"] + b @ r["entropy"] + c @ r["lse"])

    h = 1e-5
    for i in range(4):
        for v in range(9):
            up, dn = z.copy(), z.copy()
            up[i, v] += h
            dn[i, v] -= h
            assert (f(up) - f(dn)) / (2 * h) == pytest.approx(G[i, v], abs=1e-8)


def test_layer_norm_gradient_by_differences():
    g = _rng(2)
    x, dy = g.standard_normal((2, 3, 7))
    w, b = g.standard_normal((2, 7))
    dx, dw, db = ho.layer_norm_grad(dy, x, w, 1e-3)

    def f(x, w, b):
        return float((ho.layer_norm(x, w, b, 1e-3)[0] * dy).sum())

    h = 1e-6
    for t, grad in ((x, dx), (w, dw), (b, db)):
        for k in np.ndindex(t.shape):
            keep = t[k]
            t[k] = keep + h
            up = f(x, w, b)
            t[k] = keep - h
            dn = f(x, w, b)
            t[k] = keep
            assert (up - dn) / (2 * h) == pytest.approx(grad[k], abs=1e-7)


def test_layer_norm_of_a_constant_row_and_clip():
    y, mean, rstd = ho.layer_norm(np.full((1, 5), 3.0), None, np.arange(5.0), 1e-4)
    assert y[0].tolist() == [0, 1, 2, 3, 4] and mean[0] == 3 and rstd[0] == pytest.approx(100)
    n = ho.grad_norm([np.array([3.0]), np.array([[0.0], [4.0]])])
    assert n == 5.0
    assert ho.clip_coefficient(n, 10.0) == 1.0
    assert ho.clip_coefficient(n, 1.0) == pytest.approx(0.2, rel=1e-6)
    assert ho.clip_coefficient(math.inf, 1.0) == 0.0 and math.isnan(ho.clip_coefficient(math.nan, 1.0))
