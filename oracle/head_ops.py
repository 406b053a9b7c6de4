"""CPU float64 definitions of the operators around the head: log probabilities of given
tokens with entropy and top alternatives, layer norm, gradient norm and clipping, and
their gradients. Written from the formulas; test infrastructure only."""
from __future__ import annotations

import math

import numpy as np


def token_logprobs(z, tokens, *, top_k=0, temperature=1.0, ignore_index=-100):
    """dict of logprob, entropy, lse [N] and top_logprob, top_id [N, top_k]."""
    z = np.asarray(z, dtype=np.float64)
    N, V = z.shape
    out = {"logprob": np.zeros(N), "entropy": np.zeros(N), "lse": np.zeros(N),
           "top_logprob": np.full((N, top_k), -np.inf), "top_id": np.full((N, top_k), -1, dtype=np.int64)}
    for i in range(N):
        y = ignore_index if tokens is None else int(tokens[i])
        has = y != ignore_index
        x = z[i] / temperature
        if np.isnan(x).any() or np.isposinf(x).any():
            out["lse"][i] = out["entropy"][i] = np.nan
            out["logprob"][i] = np.nan if has else 0.0
            out["top_logprob"][i] = np.nan
            continue
        live = np.nonzero(~np.isneginf(x))[0]
        if live.size == 0:
            out["lse"][i] = -np.inf
            out["logprob"][i] = -np.inf if has else 0.0
            continue
        m = x[live].max()
        e = np.exp(x[live] - m)
        S = e.sum()
        lp = x - m - math.log(S)
        out["lse"][i] = m + math.log(S)
        p = np.exp(lp[live])
        out["entropy"][i] = -np.sum(np.where(p > 0, p * lp[live], 0.0))
        if has:
            others = np.exp(np.delete(x, y) - m).sum() if V > 1 else 0.0
            ey = math.exp(x[y] - m) if np.isfinite(x[y]) else 0.0
            out["logprob"][i] = -math.log1p(others / ey) if ey > 1e-200 else lp[y]
        order = live[np.lexsort((live, -z[i, live]))][:top_k]
        out["top_id"][i, :order.size] = order
        out["top_logprob"][i, :order.size] = lp[order]
    return out


def token_logprobs_grad(z, tokens, a, b, c, *, temperature=1.0, ignore_index=-100):
    """Gradient in z of sum a logprob + b entropy + c lse."""
    z = np.asarray(z, dtype=np.float64)
    r = token_logprobs(z, tokens, temperature=temperature, ignore_index=ignore_index)
    g = np.zeros_like(z)
    for i in range(z.shape[0]):
        y = ignore_index if tokens is None else int(tokens[i])
        has = y != ignore_index
        ai = float(a[i]) if (a is not None and has) else 0.0
        bi = float(b[i]) if b is not None else 0.0
        ci = float(c[i]) if c is not None else 0.0
        if np.isnan(r["lse"][i]):
            g[i] = np.nan
            continue
        if r["lse"][i] < -1e30:
            continue
        lp = z[i] / temperature - r["lse"][i]
        p = np.exp(lp)
        with np.errstate(invalid="ignore"):
            plp = np.where(p > 0, p * lp, 0.0)
        g[i] = p * (ci - ai) - bi * (plp + p * r["entropy"][i])
        if has:
            if np.isneginf(z[i, y]):
                g[i, y] = 0.0
            else:
                lpy = r["logprob"][i]
                py = math.exp(lpy)
                g[i, y] = -math.expm1(lpy) * ai + py * (ci - bi * (lpy + r["entropy"][i]))
    return g / temperature


def layer_norm(x, weight, bias, eps):
    """(y, mean, rstd)."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    h = (x - mean[:, None]) * rstd[:, None]
    w = 1.0 if weight is None else np.asarray(weight, dtype=np.float64)
    b = 0.0 if bias is None else np.asarray(bias, dtype=np.float64)
    return h * w + b, mean, rstd


def layer_norm_grad(dy, x, weight, eps):
    """(dx, dweight, dbias)."""
    dy = np.asarray(dy, dtype=np.float64)
    x = np.asarray(x, dtype=np.float64)
    _, mean, rstd = layer_norm(x, None, None, eps)
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy if weight is None else dy * np.asarray(weight, dtype=np.float64)
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True)
                          - h * (g * h).mean(axis=1, keepdims=True))
    return dx, (dy * h).sum(axis=0), dy.sum(axis=0)


def grad_norm(grads):
    return math.sqrt(math.fsum(float(np.sum(np.asarray(g, dtype=np.float64) ** 2)) for g in grads))


def clip_coefficient(norm, max_norm):
    c = max_norm / (norm + 1e-6)
    return 1.0 if c > 1.0 else c
