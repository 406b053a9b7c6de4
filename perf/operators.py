"""Performance cases of the operators around the language-model head: log
probabilities of given tokens with entropy and top alternatives (over logits, and
straight from hidden states), layer norm, and the global gradient norm with
clipping.

`run` computes a case either through this package (`own` true) or in its plain
form: elementary torch operations in 32 bits, rounded once at the end. `exact` is
the same from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

IGNORE = -100
EPS = 1e-5
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sequence's next token in a server that returns eight alternatives
        {"name": "logits_step", "op": "logits", "N": 1, "V": 128256, "pad": 0, "dtype": "bf16",
         "top_k": 8, "temperature": 1.0, "banned": 0, "train": False},
        # a decoding batch with fp32 logits, sampled at a temperature, a vocabulary padded to
        # a multiple of 64 whose padding and a few banned ids are masked
        {"name": "logits_batch", "op": "logits", "N": 48, "V": 152064, "pad": 0, "dtype": "f32",
         "top_k": 20, "temperature": 0.7, "banned": 300, "train": False},
        # scoring of prompts whose logits are at hand
        {"name": "logits_score", "op": "logits", "N": 8192, "V": 128256, "pad": 0, "dtype": "bf16",
         "top_k": 5, "temperature": 1.0, "banned": 0, "train": False},
        # policy-gradient step with an entropy bonus over logits of an odd vocabulary: rows
        # that start at any element
        {"name": "logits_train", "op": "logits", "N": 2048, "V": 100003, "pad": 0, "dtype": "bf16",
         "top_k": 0, "temperature": 1.0, "banned": 0, "train": True},
        # one next token straight from its hidden state: the head's weight is read once
        {"name": "linear_step", "op": "linear", "N": 1, "D": 4096, "V": 128256, "top_k": 8,
         "temperature": 1.0, "train": False},
        # scoring of long prompts without their logits in memory (Llama-3-8B-shaped head)
        {"name": "linear_score", "op": "linear", "N": 8192, "D": 4096, "V": 128256, "top_k": 5,
         "temperature": 1.0, "train": False},
        # policy-gradient step of a head (Llama-2-like), gradients of H and W
        {"name": "linear_train", "op": "linear", "N": 4096, "D": 2048, "V": 32000, "top_k": 0,
         "temperature": 1.0, "train": True},
        # the final norm of one token
        {"name": "norm_step", "op": "norm", "N": 1, "D": 4096, "dtype": "bf16", "wdtype": "bf16",
         "train": False},
        # the final norm of a training batch, forward and backward
        {"name": "norm_train", "op": "norm", "N": 8192, "D": 4096, "dtype": "bf16",
         "wdtype": "bf16", "train": True},
        # an odd hidden size in fp32: no row but the first is aligned
        {"name": "norm_odd", "op": "norm", "N": 3001, "D": 1111, "dtype": "f32", "wdtype": "f32",
         "train": True},
        # gradients of a small fine-tune: a norm's vectors and low-rank factors
        {"name": "clip_small", "op": "clip", "tensors": 64, "rows": 16, "D": 2048, "head": 0,
         "dtype": "f32", "max_norm": 1.0},
        # gradients of a model's layers and of its 128256-row head
        {"name": "clip_large", "op": "clip", "tensors": 48, "rows": 4096, "D": 4096,
         "head": 128256, "dtype": "bf16", "max_norm": 1.0},
    ]


# hidden sizes of whole 64s, and ones that are not
_HIDDEN = [512, 640, 768, 896, 1024, 1280, 1536, 1792, 2048, 2560, 3584, 4096]
_HIDDEN_ODD = [520, 600, 1000, 1544, 2056, 2728, 4072]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logits", "logits", "linear", "linear", "norm", "norm", "clip"])
    if op == "logits":
        V = _log_int(rng, 1000, 200000)
        N = _log_int(rng, 1, max(1, min(16384, 8192 * 128256 // (V * 2))))
        train = rng.random() < 0.4
        return {"op": op, "N": N, "V": V, "pad": rng.choice([0, 0, -V % 8, 13]),
                "dtype": rng.choice(["bf16", "f32"]), "top_k": 0 if train else rng.choice([0, 1, 5, 8, 20]),
                "temperature": rng.choice([1.0, 1.0, 0.7]), "banned": rng.choice([0, 0, 300]),
                "train": train}
    if op == "linear":
        D = rng.choice(_HIDDEN + _HIDDEN_ODD)
        V = _log_int(rng, 8000, 152064)
        train = rng.random() < 0.4
        most = (1.2e12 if train else 4.2e12) / (D * V)
        N = _log_int(rng, 1, max(1, min(8192, int(most))))
        return {"op": op, "N": N, "D": D, "V": V, "top_k": 0 if train else rng.choice([0, 1, 5, 8, 20]),
                "temperature": rng.choice([1.0, 1.0, 0.7]), "train": train}
    if op == "norm":
        D = _log_int(rng, 64, 8191) if rng.random() < 0.4 else rng.choice([64, 128, 256] + _HIDDEN + [5120, 8192])
        return {"op": op, "N": _log_int(rng, 1, 16384), "D": D, "dtype": rng.choice(["bf16", "f32"]),
                "wdtype": rng.choice(["bf16", "f32"]), "train": rng.random() < 0.6}
    return {"op": op, "tensors": _log_int(rng, 1, 200), "rows": _log_int(rng, 1, 1024),
            "D": rng.choice([64, 100, 256] + _HIDDEN + _HIDDEN_ODD), "head": rng.choice([0, 0, 32000]),
            "dtype": rng.choice(["bf16", "f32", "mixed"]), "max_norm": rng.choice([0.1, 1.0, 1e9])}


# ---- inputs ----------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _tokens(g, N, V):
    """Token ids that favour the low ones, as frequent words do; one in ten is ignored."""
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    y = (V ** u - 1).to(torch.int32).clamp_(0, V - 1)
    skip = torch.rand(N, generator=g, device="cuda") < 0.1
    return torch.where(skip, torch.full_like(y, IGNORE), y) if N > 1 else y


def _clip_sizes(case):
    """Shapes of a model's gradients: matrices of up to rows x D with vectors of D between."""
    shapes = []
    for i in range(case["tensors"]):
        if i % 4 == 3:
            shapes.append((case["D"],))
        else:
            shapes.append((max(1, case["rows"] // (1 + i % 3) - i % 2), case["D"]))
    if case["head"]:
        shapes.append((case["head"], case["D"]))
    return shapes


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "logits":
        N, V, ld = case["N"], case["V"], case["V"] + case["pad"]
        y = _tokens(g, N, V)
        full = torch.empty(N, ld, dtype=_TYPES[case["dtype"]], device="cuda")
        z = _randn(g, N, V).mul_(2.0)
        # half of the tokens are ones that the model is confident of
        sure = (torch.rand(N, generator=g, device="cuda") < 0.5).float() * 12.0
        z.scatter_add_(1, y.clamp(min=0).long()[:, None], sure[:, None])
        if case["banned"]:
            z[:, -64:] = -math.inf
            ban = torch.randint(0, V, (case["banned"],), generator=g, device="cuda")
            z[:, ban] = -math.inf
            y = torch.where((y >= 0) & torch.isneginf(z.gather(1, y.clamp(min=0).long()[:, None])[:, 0]),
                            torch.full_like(y, IGNORE), y)
        full[:, V:] = 0
        full[:, :V].copy_(z)
        s = {"case": case, "logits": full[:, :V], "tokens": y}
    elif op == "linear":
        N, D, V = case["N"], case["D"], case["V"]
        # Hidden states and weights on grids of 2^-5 and 2^-11 (std 1 and 0.02): every logit is
        # a whole number of 2^-16, exact in fp32 in whatever order it is summed, so which id
        # ranks first does not hang on the order.
        H = (_randn(g, N, D) * 32).round_().clamp_(-255, 255).mul_(2.0 ** -5)
        W = (_randn(g, V, D) * 41).round_().clamp_(-255, 255).mul_(2.0 ** -11)
        s = {"case": case, "H": H.bfloat16(), "W": W.bfloat16(), "tokens": _tokens(g, N, V)}
    elif op == "norm":
        N, D = case["N"], case["D"]
        dt, wt = _TYPES[case["dtype"]], _TYPES[case["wdtype"]]
        # a residual stream: a few channels far larger than the others, a mean that is not 0
        x = _randn(g, N, D) * (1 + 8 * (torch.rand(D, generator=g, device="cuda") < 0.01).float()) + 0.25
        s = {"case": case, "x": x.to(dt), "w": (1 + 0.1 * _randn(g, D)).to(wt),
             "b": (0.1 * _randn(g, D)).to(wt)}
        if case["train"]:
            s["dy"] = (_randn(g, N, D) * 1e-2).to(dt)
        return s
    else:
        grads, outs, total = [], [], 0
        both = case["dtype"] == "mixed"
        shapes = _clip_sizes(case)
        types = [torch.float32 if both and len(sh) == 1 else torch.bfloat16 if both else _TYPES[case["dtype"]]
                 for sh in shapes]
        # the clipped gradients go to one flat buffer for each type, each at a multiple of 64
        flat, at = {}, {t: 0 for t in types}
        places = []
        for sh, t in zip(shapes, types):
            places.append(at[t])
            at[t] += -(-math.prod(sh) // 64) * 64
        for t, n in at.items():
            flat[t] = torch.zeros(n, dtype=t, device="cuda")
        for sh, t, p in zip(shapes, types, places):
            grads.append((_randn(g, *sh) * 3e-3).to(t))
            outs.append(flat[t][p:p + math.prod(sh)].view(sh))
        return {"case": case, "grads": grads, "outs": outs, "places": places,
                "flat": {str(t).replace("torch.", ""): f for t, f in flat.items()}}
    if case["train"]:
        N = case["N"]
        s["dlogprob"] = _randn(g, N) / N      # advantages over the batch
        s["dentropy"] = torch.full((N,), -0.01 / N, device="cuda")
    return s


# ---- plain forms -----------------------------------------------------------------------------


def _rows(z, case, tokens):
    """logprob, entropy, lse, and the log probabilities and probabilities of every id."""
    x = z / case["temperature"]
    m = x.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(1, keepdim=True))
    lp = x - lse
    p = torch.exp(lp)
    ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    valid = tokens != IGNORE
    at = lp.gather(1, tokens.clamp(min=0).long()[:, None])[:, 0]
    return torch.where(valid, at, torch.zeros_like(at)), ent, lse[:, 0], lp, p


def _top(z, lp, k):
    """The k largest logits: their ids (the lowest first where logits are equal) and log
    probabilities. A 64-bit key orders by the logit and then by the id."""
    bits = (z.float() + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    ids = torch.arange(z.shape[1], device=z.device)
    key = order * (1 << 32) + (z.shape[1] - 1 - ids)
    top = torch.topk(key, k, dim=1).values
    idx = z.shape[1] - 1 - (top & 0xFFFFFFFF)
    val = lp.gather(1, idx)
    return val, torch.where(torch.isneginf(val), torch.full_like(idx, -1), idx).int()


def _dlogits(state, case, ent, lp, p):
    a, b = state["dlogprob"].to(p.dtype), state["dentropy"].to(p.dtype)
    tokens = state["tokens"]
    a = torch.where(tokens != IGNORE, a, torch.zeros_like(a))[:, None]
    g = p * (-a - b[:, None] * (torch.where(p > 0, lp, torch.zeros_like(lp)) + ent[:, None]))
    g = g.scatter_add_(1, tokens.clamp(min=0).long()[:, None], a)
    return g / case["temperature"]


def _plain(state):
    """The case in elementary operations, in 32 bits, rounded once at the end."""
    case = state["case"]
    op = case["op"]
    if op in ("logits", "linear"):
        z = state["logits"].float() if op == "logits" else state["H"].float() @ state["W"].float().T
        logprob, ent, lse, lp, p = _rows(z, case, state["tokens"])
        out = {"logprob": logprob, "entropy": ent, "lse": lse}
        if case["top_k"]:
            out["top_logprob"], out["top_id"] = _top(z, lp, case["top_k"])
        if case["train"]:
            g = _dlogits(state, case, ent, lp, p)
            if op == "logits":
                out["dlogits"] = g.to(state["logits"].dtype)
            else:
                out["dH"] = (g @ state["W"].float()).bfloat16()
                out["dW"] = (g.T @ state["H"].float()).bfloat16()
        return out
    if op == "norm":
        x, w = state["x"].float(), state["w"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        r = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
        h = xc * r
        out = {"y": (h * w + state["b"].float()).to(state["x"].dtype)}
        if case["train"]:
            dy = state["dy"].float()
            g = dy * w
            out["dx"] = (r * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))).to(state["x"].dtype)
            out["dw"] = (dy * h).sum(0).to(state["w"].dtype)
            out["db"] = dy.sum(0).to(state["w"].dtype)
        return out
    norm = torch.sqrt(torch.stack([t.float().square().sum() for t in state["grads"]]).sum())
    coef = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    for t, o in zip(state["grads"], state["outs"]):
        o.copy_(t.float() * coef)
    return {"norm": norm.reshape(1), **state["flat"]}


# ---- the package's operators -----------------------------------------------------------------


def _own(state):
    import linear_cross_entropy_flce_gb300 as flce
    case = state["case"]
    op = case["op"]
    if op == "logits":
        r = flce.token_logprobs(state["logits"], state["tokens"], top_k=case["top_k"],
                                temperature=case["temperature"])
        out = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
        if case["top_k"]:
            out["top_logprob"], out["top_id"] = r.top_logprob, r.top_id
        if case["train"]:
            out["dlogits"] = flce.token_logprobs_backward(
                state["logits"], state["tokens"], r, dlogprob=state["dlogprob"],
                dentropy=state["dentropy"], temperature=case["temperature"])
        return out
    if op == "linear":
        r = flce.linear_token_logprobs(state["H"], state["W"], state["tokens"], top_k=case["top_k"],
                                       temperature=case["temperature"])
        out = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
        if case["top_k"]:
            out["top_logprob"], out["top_id"] = r.top_logprob, r.top_id
        if case["train"]:
            out["dH"], out["dW"] = flce.linear_token_logprobs_backward(
                state["H"], state["W"], state["tokens"], r, dlogprob=state["dlogprob"],
                dentropy=state["dentropy"], temperature=case["temperature"], dw_dtype="bfloat16")
        return out
    if op == "norm":
        r = flce.layer_norm(state["x"], state["w"], state["b"], eps=EPS)
        out = {"y": r.y}
        if case["train"]:
            out["dx"], out["dw"], out["db"] = flce.layer_norm_backward(state["dy"], state["x"], state["w"], r)
        return out
    norm = flce.clip_grads(state["grads"], case["max_norm"], out=state["outs"])
    return {"norm": norm, **state["flat"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- definitions in 64 bits ------------------------------------------------------------------


def _exact_rows(z, tokens, tau, k):
    """Per row, from the definition: log softmax at the token, entropy, log-sum-exp, and the
    sorted largest log probabilities."""
    x = z / tau
    lse = torch.logsumexp(x, 1)
    lp = torch.log_softmax(x, 1)
    ent = -torch.xlogy(lp.exp(), lp.exp()).sum(1)
    rows = torch.arange(z.shape[0], device=z.device)
    lp_y = torch.where(tokens == IGNORE, 0.0, lp[rows, tokens.long().clamp(min=0)])
    out = {"logprob": lp_y, "entropy": ent, "lse": lse}
    if k:
        out["top_logprob"], out["top_id"] = torch.topk(lp, k, dim=1).values, None
    return out, lp, rows


def _exact_grad(lp, ent, rows, tokens, a, b, tau):
    """The gradient of sum a logprob + b entropy in the logits: d logprob / dx_v = [v = y] - p_v,
    d entropy / dx_v = -p_v (log p_v + entropy)."""
    p = lp.exp()
    keep = tokens != IGNORE
    a = a.double() * keep
    g = -a[:, None] * p - b.double()[:, None] * (torch.xlogy(p, p) + p * ent[:, None])
    g[rows, tokens.long().clamp(min=0)] += a
    return g / tau


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("logits", "linear"):
        if case["N"] * case["V"] > 1.2e9:
            return None
        if op == "linear" and case["N"] * case["V"] * case["D"] * (3 if case["train"] else 1) > 6e12:
            return None
        z = s["logits"].double() if op == "logits" else s["H"].double() @ s["W"].double().T
        out, lp, rows = _exact_rows(z, s["tokens"], case["temperature"], case["top_k"])
        if case["train"]:
            g = _exact_grad(lp, out["entropy"], rows, s["tokens"], s["dlogprob"], s["dentropy"],
                            case["temperature"])
            if op == "logits":
                out["dlogits"] = g
            else:
                out["dH"], out["dW"] = g @ s["W"].double(), g.T @ s["H"].double()
        return out
    if op == "norm":
        x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
        mu = x.mean(1)
        var = x.var(1, unbiased=False)
        h = (x - mu[:, None]) / (var + EPS).sqrt()[:, None]
        out = {"y": h * w + b}
        if case["train"]:
            D = case["D"]
            dy = s["dy"].double()
            dh = dy * w
            out["dx"] = (D * dh - dh.sum(1)[:, None] - h * (dh * h).sum(1)[:, None]) / (
                D * (var + EPS).sqrt()[:, None])
            out["dw"], out["db"] = (dy * h).sum(0), dy.sum(0)
        return out
    norm = math.sqrt(sum(float((t.double() ** 2).sum()) for t in s["grads"]))
    coef = min(1.0, case["max_norm"] / (norm + 1e-6))
    out = {"norm": torch.tensor([norm], dtype=torch.float64)}
    for name, f in s["flat"].items():
        wide = torch.zeros(f.shape, dtype=torch.float64, device=f.device)
        for t, p in zip(s["grads"], s["places"]):
            if str(t.dtype) == "torch." + name:
                wide[p:p + t.numel()] = t.double().reshape(-1) * coef
        out[name] = wide
    return out


# ---- work ------------------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op in ("logits", "linear"):
        N, V = case["N"], case["V"]
        small = N * (4 + 12 + 8 * case["top_k"] + (8 if case["train"] else 0))
        if op == "logits":
            e = 2 if case["dtype"] == "bf16" else 4
            return {"bytes": N * V * e * (2 if case["train"] else 1) + small,
                    "flops": N * V * (16 if case["train"] else 7)}
        D = case["D"]
        return {"bytes": (N + V) * D * 2 * (2 if case["train"] else 1) + small,
                "flops": 2.0 * N * V * D * (3 if case["train"] else 1)}
    if op == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        N, D = case["N"], case["D"]
        return {"bytes": N * D * e * (4 if case["train"] else 2) + 4 * D * e,
                "flops": N * D * (20 if case["train"] else 7)}
    n = b = 0
    for sh in _clip_sizes(case):
        m = math.prod(sh)
        n += m
        b += m * (4 if case["dtype"] == "f32" or (case["dtype"] == "mixed" and len(sh) == 1) else 2)
    return {"bytes": 2 * b + 4, "flops": 3 * n}
