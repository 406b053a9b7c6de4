"""Performance cases of the operators on either side of the head in fewer bits: embedding lookup
with its gradient by sorted tokens (the head's tied table), activations kept in 8 bits for the
backward pass (alone, and by the layer norm), and block-scaled 4-bit floating point
(quantisation, and the product of a 4-bit head).

`run` computes a case either through this package (`own` true) or in its plain form:
elementary torch operations in 32 bits, rounded once at the end. `exact` is the same from the
definitions in 64 bits. What is held in 8 or 4 bits is returned as the values it stands for.
"""
from __future__ import annotations

import math

import torch

own = False

IGNORE = -100
EPS = 1e-5
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BLOCK = {"nvfp4": 16, "mxfp4": 32}


def listed():
    return [
        # the token that a decoding step feeds back
        {"name": "embed_step", "op": "embed", "N": 1, "D": 4096, "V": 128256, "dtype": "bf16",
         "out": "bf16", "scale": 1.0, "train": False},
        # ragged prompts through an fp32 table of an odd hidden size, scaled by sqrt(D) as tied
        # tables are, to bf16, and the table's gradient
        {"name": "embed_odd", "op": "embed", "N": 3001, "D": 1111, "V": 32000, "dtype": "f32",
         "out": "bf16", "scale": 33.33, "train": True},
        # a training batch: lookup, and the whole gradient of the table by its tokens
        {"name": "embed_train", "op": "embed", "N": 8192, "D": 4096, "V": 128256, "dtype": "bf16",
         "out": "bf16", "scale": 1.0, "train": True},
        # one hidden state put away in 8 bits and taken out again
        {"name": "pack_step", "op": "pack", "N": 1, "D": 4096, "dtype": "bf16"},
        # a layer's activations of a long batch: put away on the way forward, taken out on the
        # way back
        {"name": "pack_large", "op": "pack", "N": 16384, "D": 8192, "dtype": "bf16"},
        # the final norm of a training batch that keeps its input in 8 bits, forward and backward
        {"name": "norm8_train", "op": "norm8", "N": 8192, "D": 4096, "dtype": "bf16",
         "wdtype": "bf16"},
        # the same at an odd hidden size in fp32: no row but the first is aligned, and the last
        # block of each is short
        {"name": "norm8_odd", "op": "norm8", "N": 3001, "D": 1111, "dtype": "f32", "wdtype": "f32"},
        # a 128256-row head turned into 4 bits, and its values for a check
        {"name": "fp4_weights", "op": "fp4", "N": 128256, "D": 4096, "dtype": "bf16",
         "format": "nvfp4"},
        # ragged fp32 activations of an odd size
        {"name": "fp4_odd", "op": "fp4", "N": 3001, "D": 1111, "dtype": "f32", "format": "mxfp4"},
        # one next token through a 4-bit head: the weights are read once
        {"name": "fp4_step", "op": "linear4", "N": 1, "D": 4096, "V": 128256, "dtype": "bf16",
         "out": "f32", "format": "nvfp4"},
        # a decoding batch through a head of an odd vocabulary
        {"name": "fp4_batch", "op": "linear4", "N": 48, "D": 2048, "V": 100003, "dtype": "bf16",
         "out": "bf16", "format": "mxfp4"},
        # logits of long prompts
        {"name": "fp4_score", "op": "linear4", "N": 8192, "D": 4096, "V": 128256, "dtype": "bf16",
         "out": "bf16", "format": "nvfp4"},
    ]


# hidden sizes of whole 64s, and ones that are not
_HIDDEN = [512, 640, 768, 896, 1024, 1280, 1536, 1792, 2048, 2560, 3584, 4096]
_HIDDEN_ODD = [520, 601, 1000, 1111, 1544, 2056, 2731, 4072]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed", "pack", "norm8", "fp4", "linear4", "linear4"])
    dtype = rng.choice(["bf16", "f32"])
    fmt = rng.choice(["nvfp4", "mxfp4"])
    D = rng.choice(_HIDDEN + _HIDDEN_ODD)
    if op == "embed":
        V = _log_int(rng, 1000, 128256 if dtype == "bf16" else 64128)
        return {"op": op, "N": _log_int(rng, 1, 8192), "D": D, "V": V, "dtype": dtype,
                "out": rng.choice(["bf16", "f32"]) if dtype == "f32" else "bf16",
                "scale": rng.choice([1.0, math.sqrt(D)]), "train": rng.random() < 0.6}
    if op == "pack":
        return {"op": op, "N": _log_int(rng, 1, 16384), "D": _log_int(rng, 32, 8192), "dtype": dtype}
    if op == "norm8":
        D = _log_int(rng, 64, 8191) if rng.random() < 0.4 else D
        return {"op": op, "N": _log_int(rng, 1, 16384), "D": D, "dtype": dtype,
                "wdtype": rng.choice(["bf16", "f32"])}
    if op == "fp4":
        most = 128256 * 4096 // (D * (1 if dtype == "bf16" else 2))
        return {"op": op, "N": _log_int(rng, 1, min(152064, most)), "D": D, "dtype": dtype, "format": fmt}
    V, out = _log_int(rng, 1000, 152064), rng.choice(["bf16", "f32"])
    most = min(4.2e12 / (D * V), (1.0e9 if out == "bf16" else 5.0e8) / V)
    return {"op": op, "N": _log_int(rng, 1, max(1, min(8192, int(most)))), "D": D, "V": V, "dtype": "bf16",
            "out": out, "format": fmt}


# ---- inputs ----------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6271 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _tokens(g, N, V):
    """Token ids that favour the low ones, as frequent words do; one in ten is padding."""
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    y = (V ** u - 1).to(torch.int32).clamp_(0, V - 1)
    skip = torch.rand(N, generator=g, device="cuda") < 0.1
    return torch.where(skip, torch.full_like(y, IGNORE), y) if N > 1 else y


def _hidden(g, N, D):
    """A residual stream: a few channels far larger than the others, a mean that is not 0."""
    return _randn(g, N, D) * (1 + 8 * (torch.rand(D, generator=g, device="cuda") < 0.01).float()) + 0.1


def prepare(case, seed):
    g = _gen(seed)
    op, N, D = case["op"], case["N"], case["D"]
    dt = _TYPES[case["dtype"]]
    if op == "embed":
        s = {"case": case, "tokens": _tokens(g, N, case["V"]), "W": (_randn(g, case["V"], D) * 0.02).to(dt)}
        if case["train"]:
            s["dy"] = (_randn(g, N, D) * 1e-2).to(_TYPES[case["out"]])
        return s
    if op == "norm8":
        wt = _TYPES[case["wdtype"]]
        return {"case": case, "x": _hidden(g, N, D).to(dt), "w": (1 + 0.1 * _randn(g, D)).to(wt),
                "b": (0.1 * _randn(g, D)).to(wt), "dy": (_randn(g, N, D) * 1e-2).to(dt)}
    if op != "linear4":
        return {"case": case, "x": (_randn(g, N, D) * 0.02 if N > 16384 else _hidden(g, N, D)).to(dt)}
    s = {"case": case, "x": _hidden(g, N, D).to(dt)}
    W = (_randn(g, case["V"], D) * 0.02).to(torch.bfloat16)
    # the head is turned into 4 bits once, when it is loaded
    if own:
        import linear_cross_entropy_flce_gb300 as flce
        s["W4"] = flce.quantize_fp4(W, format=case["format"])
    else:
        s["W4"] = _fp4(W, case["format"]).bfloat16()   # 6 significant bits: exact
    return s


# ---- plain forms -----------------------------------------------------------------------------


def _blocks(x, size):
    """x [N, D] fp32 as [N, blocks, size], zeros behind the row."""
    N, D = x.shape
    return torch.nn.functional.pad(x, (0, -D % size)).reshape(N, -1, size)


def _two(k):
    """2^k in 32 bits, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64).float()


def _power(amax, most):
    """The exponent of the smallest power of two s with amax <= most s, from -127 on."""
    e = torch.frexp(amax.double() / most)
    return torch.where(e.mantissa == 0.5, e.exponent - 1, e.exponent).clamp(min=-127)


def _round_bits(x, bits, lowest, most):
    """x to the nearest value of `bits` mantissa bits with exponents from `lowest` on (ties to
    the even one), at most `most` in magnitude."""
    e = (torch.frexp(x).exponent - 1).clamp(min=lowest) - bits
    step = _two(e)
    return (torch.round(x / step) * step).clamp(-most, most)


def _e4m3(x):
    """The values of x in E4M3 with a power-of-two scale for each 32 of a row. A block with an
    infinity or a NaN is NaN."""
    b = _blocks(x.float(), 32)
    amax = b.abs().amax(2, keepdim=True)
    scale = _two(_power(torch.where(torch.isfinite(amax) & (amax > 0), amax, torch.ones_like(amax)), 448.0))
    q = _round_bits(b / scale, 3, -6, 448.0)
    v = torch.where(torch.isfinite(amax), q * scale, torch.full_like(q, math.nan))
    return v.reshape(x.shape[0], -1)[:, :x.shape[1]]


def _fp4(x, fmt):
    """The values of x in E2M1. mxfp4: a power-of-two scale for each 32 of a row. nvfp4: an E4M3
    scale for each 16, times a power of two for each row."""
    b = _blocks(x.float(), _BLOCK[fmt])
    amax = b.abs().amax(2, keepdim=True)
    one = torch.ones_like(amax)
    finite = torch.isfinite(amax)
    if fmt == "mxfp4":
        scale = _two(_power(torch.where(finite & (amax > 0), amax, one), 6.0))
    else:
        top = torch.where(torch.isfinite(b), b, torch.zeros_like(b)).abs().amax((1, 2), keepdim=True)
        row = _two(_power(torch.where(top > 0, top, torch.ones_like(top)), 2688.0).clamp(min=-126))
        block = _round_bits(torch.where(finite, amax / 6.0 / row, one), 3, -6, 448.0)
        scale = block * row
    q = torch.where(scale > 0, b / torch.where(scale > 0, scale, torch.ones_like(scale)), torch.zeros_like(scale))
    q = _round_bits(q, 1, 0, 6.0)
    v = torch.where(finite, q * scale, torch.full_like(q, math.nan))
    return v.reshape(x.shape[0], -1)[:, :x.shape[1]]


def _plain(state):
    """The case in elementary operations, in 32 bits, rounded once at the end."""
    case = state["case"]
    op = case["op"]
    if op == "embed":
        tokens, W = state["tokens"], state["W"]
        live = tokens != IGNORE
        at = torch.where(live, tokens, torch.zeros_like(tokens)).long()
        y = W[at].float() * case["scale"]
        out = {"y": torch.where(live[:, None], y, torch.zeros_like(y)).to(_TYPES[case["out"]])}
        if case["train"]:
            dy = torch.where(live[:, None], state["dy"].float(), torch.zeros_like(y))
            dW = torch.zeros(W.shape, dtype=torch.float32, device=W.device).index_add_(0, at, dy)
            out["dW"] = (dW * case["scale"]).to(W.dtype)
        return out
    x = state["x"]
    if op == "pack":
        return {"values": _e4m3(x).to(x.dtype)}
    if op == "fp4":
        return {"values": _fp4(x, case["format"]).to(x.dtype)}
    if op == "linear4":
        y = _fp4(x, case["format"]) @ state["W4"].float().T
        return {"y": y.to(_TYPES[case["out"]])}
    w, dy = state["w"].float(), state["dy"].float()
    xf = x.float()
    mean = xf.mean(1, keepdim=True)
    xc = xf - mean
    r = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    out = {"y": (xc * r * w + state["b"].float()).to(x.dtype)}
    h = (_e4m3(x) - mean) * r
    g = dy * w
    out["dx"] = (r * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))).to(x.dtype)
    out["dw"] = (dy * h).sum(0).to(state["w"].dtype)
    out["db"] = dy.sum(0).to(state["w"].dtype)
    return out


# ---- the package's operators -----------------------------------------------------------------


def _own(state):
    import linear_cross_entropy_flce_gb300 as flce
    case = state["case"]
    op = case["op"]
    if op == "embed":
        W = state["W"]
        out = {"y": flce.embedding(W, state["tokens"], scale=case["scale"], dtype=_TYPES[case["out"]])}
        if case["train"]:
            out["dW"] = flce.embedding_backward(state["dy"], state["tokens"], W.shape[0],
                                                scale=case["scale"], dtype=W.dtype)
        return out
    x = state["x"]
    if op == "pack":
        return {"values": flce.unpack_e4m3(flce.pack_e4m3(x), dtype=x.dtype)}
    if op == "fp4":
        return {"values": flce.dequantize_fp4(flce.quantize_fp4(x, format=case["format"]), dtype=x.dtype)}
    if op == "linear4":
        return {"y": flce.linear_fp4(flce.quantize_fp4(x, format=case["format"]), state["W4"],
                                     dtype=_TYPES[case["out"]])}
    r, packed = flce.layer_norm_packed(x, state["w"], state["b"], eps=EPS)
    out = {"y": r.y}
    out["dx"], out["dw"], out["db"] = flce.layer_norm_packed_backward(state["dy"], packed, state["w"], r)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---- definitions in 64 bits ------------------------------------------------------------------


def _grid(bits, lowest, count):
    """The first `count` non-negative values of a format with `bits` mantissa bits whose
    subnormals have the exponent `lowest`: value k has code k."""
    vals = []
    for k in range(count):
        e, m = divmod(k, 2 ** bits)
        vals.append(math.ldexp(m, lowest - bits) if e == 0 else math.ldexp(2 ** bits + m, lowest + e - 1 - bits))
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _nearest(x, grid):
    """The nearest grid value with x's sign; halfway, the one with the even code."""
    mid = (grid[1:] + grid[:-1]) / 2
    a = x.abs().contiguous()
    lo = torch.searchsorted(mid, a)               # a midpoint itself counts to the code below it
    hi = torch.searchsorted(mid, a, right=True)   # and here to the one above
    return torch.copysign(grid[torch.where(lo % 2 == 0, lo, hi)], x)


def _exact_two(k):
    table = torch.tensor([math.ldexp(1.0, i) for i in range(-200, 201)], dtype=torch.float64, device="cuda")
    return table[(k + 200).long()]


def _exact_power(amax, most):
    k = torch.full_like(amax, -127.0)
    k = torch.maximum(k, torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)) / most)) - 1)
    for _ in range(3):
        k = torch.where(amax > most * _exact_two(k), k + 1, k)
    return torch.where(amax > 0, k, torch.zeros_like(k))


def _exact_values(x, fmt):
    """What x [N, D] stands for in the format, in 64 bits, some rows at a time."""
    size = 32 if fmt == "e4m3" else _BLOCK[fmt]
    e4m3, e2m1 = _grid(3, -6, 127), _grid(1, 0, 8)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    D = x.shape[1]
    step = max(1, (1 << 26) // D)
    for i in range(0, x.shape[0], step):
        part = x[i:i + step].double()
        full = part.new_zeros(part.shape[0], -(-D // size) * size)
        full[:, :D] = part
        b = full.view(part.shape[0], -1, size)
        amax = b.abs().amax(2, keepdim=True)
        if fmt == "e4m3":
            s = _exact_two(_exact_power(amax, 448.0))
            v = _nearest(b / s, e4m3) * s
        elif fmt == "mxfp4":
            s = _exact_two(_exact_power(amax, 6.0))
            v = _nearest(b / s, e2m1) * s
        else:
            row = _exact_two(_exact_power(amax.amax(1, keepdim=True), 2688.0).clamp(min=-126))
            s = _nearest(amax / 6.0 / row, e4m3) * row
            v = torch.where(s > 0, _nearest(b / torch.where(s > 0, s, 1.0), e2m1) * s, 0.0)
        out[i:i + step] = v.view(part.shape[0], -1)[:, :D]
    return out


def exact(case, seed):
    op, N, D = case["op"], case["N"], case["D"]
    if op == "linear4" and (N * case["V"] > 1.2e9 or N * case["V"] * D > 6e12):
        return None
    if op == "linear4":
        g = _gen(seed)
        x = _hidden(g, N, D).to(_TYPES[case["dtype"]])
        W = (_randn(g, case["V"], D) * 0.02).to(torch.bfloat16)
        return {"y": _exact_values(x, case["format"]) @ _exact_values(W, case["format"]).T}
    s = prepare(case, seed)
    if op == "embed":
        W, tokens = s["W"], s["tokens"].long()
        rows = (tokens != IGNORE).nonzero()[:, 0]
        y = torch.zeros(N, D, dtype=torch.float64, device=W.device)
        y[rows] = W.index_select(0, tokens[rows]).double() * case["scale"]
        out = {"y": y}
        if case["train"]:
            dW = torch.zeros(W.shape, dtype=torch.float64, device=W.device)
            dW.index_put_((tokens[rows],), s["dy"][rows].double() * case["scale"], accumulate=True)
            out["dW"] = dW
        return out
    x = s["x"]
    if op == "pack":
        return {"values": _exact_values(x, "e4m3")}
    if op == "fp4":
        return {"values": _exact_values(x, case["format"])}
    xd, w, dy = x.double(), s["w"].double(), s["dy"].double()
    mu, std = xd.mean(1), (xd.var(1, unbiased=False) + EPS).sqrt()
    out = {"y": (xd - mu[:, None]) / std[:, None] * w + s["b"].double()}
    h = (_exact_values(x, "e4m3") - mu[:, None]) / std[:, None]
    dh = dy * w
    out["dx"] = (D * dh - dh.sum(1)[:, None] - h * (dh * h).sum(1)[:, None]) / (D * std[:, None])
    out["dw"], out["db"] = (dy * h).sum(0), dy.sum(0)
    return out


# ---- work ------------------------------------------------------------------------------------


def work(case):
    op, N, D = case["op"], case["N"], case["D"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "embed":
        V, eo = case["V"], 2 if case["out"] == "bf16" else 4
        # a row looked up for each token (fewer where tokens repeat), the table's gradient whole
        b = N * (4 + D * (min(1.0, V / N) * e + eo))
        f = N * D
        if case["train"]:
            b += N * (4 + D * eo) + V * D * e
            f += N * D
        return {"bytes": b, "flops": f}
    eight, four = 1 + 1 / 32, 0.5 + 1 / _BLOCK.get(case.get("format"), 32)
    if op == "pack":
        return {"bytes": N * D * 2 * (e + eight), "flops": 4 * N * D}
    if op == "fp4":
        return {"bytes": N * D * 2 * (e + four), "flops": 5 * N * D}
    if op == "norm8":
        # x read, y and the 8 bits written; the 8 bits and dy read, dx written
        return {"bytes": N * D * (4 * e + 2 * eight) + 4 * D * e, "flops": 25 * N * D}
    V, eo = case["V"], 2 if case["out"] == "bf16" else 4
    return {"bytes": N * D * e + V * D * four + N * V * eo, "flops": 2.0 * N * V * D}
