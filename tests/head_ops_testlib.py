"""Bounds for the operators around the head, derived from the roundings of their fp32
formulas; shared by the GPU tests.

u = 2^-24 is half a step of fp32. Log probabilities, with x = z / T and X = max |x|:
  * an exponent d = (z - M) log2(e) / T carries three roundings of |d| and the two of its
    factor, 5 u |d|; only terms with |d| < 60 matter, and a term's weight falls as 2^d
    while its error grows as |d|, so the weighted error stays below 5 u * 4. The hardware
    2^d adds 2^-22;
  * a sum of n terms by `chain` additions in a row in a thread, then a tree, adds
    u (chain + 16): EPS below is the relative error of S and of the entropy's sum;
  * lse = M / T + log S: EPS plus two roundings of X and of lse;
  * entropy = log S - ln 2 T' / S: EPS (1 + 2 T' ln2 / S) plus roundings of the two terms,
    each at most log V + 1 or so;
  * logprob = -log1p(S_o / e_y): relative 2 EPS plus the roundings of d_y, log1p and the
    quotient, 8 u; past e_y < 2^-60 a difference of numbers up to X + log V;
  * a gradient entry p (A - B (l + H)): p's relative error is EPS + 4 u (X + |lse|), l and
    H carry the errors of x, lse and the entropy; then one rounding to the output type.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def half_step(dtype) -> float:
    import torch
    return torch.finfo(dtype).eps / 2


def sum_eps(V: int, chain_threads: int = 32) -> float:
    return 20 * U + 2.0 ** -22 + U * (-(-V // chain_threads) + 16)


def extent(z, T):
    """Largest |z| / T of each row over finite logits above -1e30 (0 if there is none)."""
    z = np.asarray(z, dtype=np.float64) / T
    live = np.isfinite(z) & (z > -1e30)
    return np.max(np.where(live, np.abs(z), 0.0), axis=1)


def check_logprobs(res, ref, z, T, *, eps=None, z_err=0.0):
    """res (tensors) against the float64 ref; z the logits that define them. z_err: an
    absolute error of each logit (a product accumulated in fp32)."""
    z = np.asarray(z)
    V = z.shape[1]
    e = (sum_eps(V) if eps is None else eps) + 2 * z_err / T
    X = extent(z, T)
    logv = np.log(V) + 1
    with np.errstate(invalid="ignore"):
        lse_tol = e + 4 * U * (X + logv)
        _close(res.lse, ref["lse"], lse_tol, "lse")
        _close(res.entropy, ref["entropy"], e * (1 + 2 * logv) + 8 * U * logv, "entropy")
        far = np.where(ref["logprob"] < -40, lse_tol + 4 * U * (X + np.abs(ref["logprob"])), 0.0)
        lp_tol = (2 * e + 8 * U) * np.abs(ref["logprob"]) + far + 2 * z_err / T
        _close(res.logprob, ref["logprob"], lp_tol, "logprob")
        if ref["top_id"].shape[1]:
            _close(res.top_logprob, ref["top_logprob"],
                   (e + 8 * U * (X + logv))[:, None] + 4 * U * np.abs(ref["top_logprob"]), "top_logprob")


def _close(t, want, tol, name):
    got = t.double().cpu().numpy()
    want = np.asarray(want, dtype=np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), name
    diff = np.abs(got - np.where(fine, want, 0.0))
    over = fine & ~(diff <= tol)
    assert not over.any(), (name, np.max(np.where(fine, diff / np.maximum(tol, 1e-300), 0)),
                            np.argwhere(over)[:3].tolist())


def grad_bound(z, ref_g, ref, a, b, c, T, dtype, *, eps=None):
    """Element-wise bound of a gradient in the logits (float64 arrays; a, b, c may be None)."""
    z = np.asarray(z, dtype=np.float64)
    N, V = z.shape
    zero = np.zeros(N)
    a, b, c = (np.abs(zero if t is None else np.asarray(t, dtype=np.float64)) for t in (a, b, c))
    e = sum_eps(V) if eps is None else eps
    X = extent(z, T)
    logv = np.log(V) + 1
    lse = np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0.0)
    lse = np.where(lse > 1e30, 0.0, lse)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        l = z / T - np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0)[:, None]
        p = np.where(l > -700, np.exp(np.minimum(l, 0.0)), 0.0)
        absl = np.where(p > 0, np.abs(l), 0.0)
    rel_p = e + 4 * U * (X + lse) + 2.0 ** -22
    err_l = e + 4 * U * (X + lse)
    err_h = e * (1 + 2 * logv) + 8 * U * logv
    size = (a + c)[:, None] + b[:, None] * (absl + ref["entropy"][:, None])
    bound = p * ((rel_p + 8 * U)[:, None] * size + (b * (err_l + err_h))[:, None]) / T
    # the token's own entry: a (1 - p) from its log probability
    return bound + (half_step(dtype) + 8 * U + 4 * e) * np.abs(ref_g) + 2.0 ** -126
