"""The operators around the head under PyTorch autograd.

    norm = FusedLayerNorm(hidden)
    logprob, entropy, lse = fused_linear_token_logprobs(norm(x), lm_head.weight, tokens)
    loss = -(advantage * logprob).mean() - 0.01 * entropy.mean()
    loss.backward()
    clip_grads([p.grad for p in parameters], max_norm=1.0)

Every arithmetic step runs in libflce.so; this module only marshals tensors. The
gradients are first order only.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _blocks_binding as Q
from . import _embed_binding as E
from . import _ops_binding as B
from ._binding import int32_ids


def _flat_tokens(tokens, ignore_index):
    if tokens is None:
        return None
    t = int32_ids(tokens.reshape(-1), ignore_index)
    return t if t.is_contiguous() else t.contiguous()


def _flat_grad(g):
    return None if g is None else g.detach().reshape(-1).to(torch.float32)


class _Places:
    """Where the rows of a [..., V] view are among the R equally spaced rows that enclose it."""

    def __init__(self, sizes, steps, rows):
        self.sizes, self.steps, self.rows = sizes, steps, rows

    def spread(self, t, fill):
        """t, one value for each row of the view, as a vector of R: `fill` in the other places."""
        e = t.new_full((self.rows,), fill)
        e.as_strided(self.sizes, self.steps).copy_(t.reshape(self.sizes))
        return e

    def pick(self, t):
        """The view's values of a vector of R, in the view's shape."""
        return t.as_strided(self.sizes, self.steps).contiguous()

    def pick_rows(self, t):
        """The view's rows of a [R, V] matrix, as a view of it."""
        ld = t.stride(0)
        return t.as_strided((*self.sizes, t.shape[1]), (*(n * ld for n in self.steps), 1))


def _rows(logits):
    """logits [..., V] as (z [R, V] of unit column stride, places). Without places, z has the
    rows in order. A view that leaves out some rows of an evenly spaced whole, as the shifted
    logits[:, :-1] does, would have to be copied for that; where they are few (an eighth of the
    others at most: a row is read once and a copy writes and reads it as well) z is the whole,
    and the operators run over the rows between too, whose results count nowhere."""
    V = logits.shape[-1]
    sizes, strides = logits.shape[:-1], logits.stride()[:-1]
    dims = [(n, st) for n, st in zip(sizes, strides) if n > 1]
    if len(dims) > 1 and logits.numel() > 0 and (V == 1 or logits.stride(-1) == 1):
        ld = dims[-1][1]
        if ld >= V and all(st % ld == 0 and st >= n * inner
                           for (_, st), (n, inner) in zip(dims, dims[1:])):
            whole = 1 + sum((n - 1) * (st // ld) for n, st in dims)
            rows = logits.numel() // V
            if whole > rows and 8 * whole <= 9 * rows:
                steps = [st // ld if n > 1 else 1 for n, st in zip(sizes, strides)]
                return logits.as_strided((whole, V), (ld, 1)), _Places(sizes, steps, whole)
    z = logits.reshape(-1, V)
    if V > 1 and z.stride(1) != 1 or z.shape[0] > 1 and z.stride(0) < V:
        z = z.contiguous()
    return z, None


class TokenLogprobsFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature: float, ignore_index: int):
        z, places = _rows(logits)
        y = _flat_tokens(tokens, ignore_index)
        rows = logits.shape[:-1]
        if places is not None and y is not None:
            if y.numel() != rows.numel():
                raise ValueError("tokens must have one id for each row of logits")
            y = places.spread(y, ignore_index)
        r = B.token_logprobs(z, y, temperature=temperature, ignore_index=ignore_index)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(z, y, r.logprob, r.entropy, r.lse)
        ctx.shape, ctx.options, ctx.places = logits.shape, (temperature, ignore_index), places
        outputs = r.logprob, r.entropy, r.lse
        return tuple(t.reshape(rows) if places is None else places.pick(t) for t in outputs)

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogprob, dentropy, dlse):
        if dlogprob is None and dentropy is None and dlse is None:
            return None, None, None, None
        z, y, *saved = ctx.saved_tensors
        temperature, ignore_index = ctx.options
        places = ctx.places
        up = [_flat_grad(g) for g in (dlogprob, dentropy, dlse)]
        if places is not None:
            up = [g if g is None else places.spread(g, 0) for g in up]
        dz = B.token_logprobs_backward(z, y, B.TokenLogprobs(*saved), dlogprob=up[0], dentropy=up[1],
                                       dlse=up[2], temperature=temperature, ignore_index=ignore_index)
        return dz.reshape(ctx.shape) if places is None else places.pick_rows(dz), None, None, None


class LinearTokenLogprobsFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden_states, weight, tokens, temperature: float, ignore_index: int):
        H = hidden_states.reshape(-1, hidden_states.shape[-1])
        H = H if H.is_contiguous() else H.contiguous()
        y = _flat_tokens(tokens, ignore_index)
        r = B.linear_token_logprobs(H, weight, y, temperature=temperature,
                                    ignore_index=ignore_index)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(H, weight, y, r.logprob, r.entropy, r.lse)
        ctx.shape, ctx.options = hidden_states.shape, (temperature, ignore_index)
        rows = hidden_states.shape[:-1]
        return r.logprob.reshape(rows), r.entropy.reshape(rows), r.lse.reshape(rows)

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogprob, dentropy, dlse):
        need_dh, need_dw = ctx.needs_input_grad[:2]
        if dlogprob is None and dentropy is None and dlse is None or not (need_dh or need_dw):
            return None, None, None, None, None
        H, weight, y, *saved = ctx.saved_tensors
        temperature, ignore_index = ctx.options
        dH, dW = B.linear_token_logprobs_backward(
            H, weight, y, B.TokenLogprobs(*saved), dlogprob=_flat_grad(dlogprob),
            dentropy=_flat_grad(dentropy), dlse=_flat_grad(dlse), temperature=temperature,
            ignore_index=ignore_index, need_dh=need_dh, need_dw=need_dw, dw_dtype="bfloat16")
        return dH.reshape(ctx.shape) if need_dh else None, dW, None, None, None


class LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps: float):
        r = B.layer_norm(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, weight, r.mean, r.rstd)
        return r.y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = B.layer_norm_backward(
            dy, x, weight, B.LayerNormResult(None, mean, rstd), need_dx=ctx.needs_input_grad[0],
            need_dweight=ctx.needs_input_grad[1], need_dbias=ctx.needs_input_grad[2])
        return dx, dw, db, None


class PackedLayerNormFunction(torch.autograd.Function):
    """LayerNormFunction that keeps its input in 8 bits between the passes."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps: float):
        r, packed = Q.layer_norm_packed(x, weight, bias, eps=eps)
        ctx.save_for_backward(packed.data, weight, r.mean, r.rstd)
        ctx.packed = packed.shape, packed.dtype
        return r.y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        data, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = Q.layer_norm_packed_backward(
            dy, Q.PackedRows(data, *ctx.packed), weight, B.LayerNormResult(None, mean, rstd),
            need_dx=ctx.needs_input_grad[0], need_dweight=ctx.needs_input_grad[1],
            need_dbias=ctx.needs_input_grad[2])
        return dx, dw, db, None


class EmbeddingFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale: float, ignore_index: int, dtype):
        if tokens.dtype.is_floating_point or tokens.dtype.is_complex:
            raise TypeError("tokens must be integers")
        y = int32_ids(tokens, ignore_index)
        y = y if y.is_contiguous() else y.contiguous()
        ctx.save_for_backward(y)
        ctx.table, ctx.options = (weight.shape[0], weight.dtype), (scale, ignore_index)
        return E.embedding(weight, y, scale=scale, ignore_index=ignore_index, dtype=dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        if not ctx.needs_input_grad[1]:
            return None, None, None, None, None
        tokens, = ctx.saved_tensors
        scale, ignore_index = ctx.options
        dW = E.embedding_backward(dy, tokens, ctx.table[0], scale=scale, ignore_index=ignore_index,
                                  dtype=ctx.table[1])
        return None, dW, None, None, None


def fused_token_logprobs(logits, tokens, *, temperature: float = 1.0, ignore_index: int = -100):
    """(logprob, entropy, lse), each of tokens' shape and fp32, of tokens [...] over
    logits [..., V] (fp32 or bf16); differentiable in the logits."""
    return TokenLogprobsFunction.apply(logits, tokens, float(temperature), int(ignore_index))


def fused_linear_token_logprobs(hidden_states, weight, tokens, *, temperature: float = 1.0,
                                ignore_index: int = -100):
    """fused_token_logprobs of the logits hidden_states @ weight.T without forming them:
    hidden_states [..., D] and the head's weight [V, D] are bf16, both differentiable."""
    return LinearTokenLogprobsFunction.apply(hidden_states, weight, tokens, float(temperature),
                                             int(ignore_index))


def fused_layer_norm(x, weight=None, bias=None, eps: float = 1e-5, packed: bool = False):
    """Layer norm over the last dimension of x (fp32 or bf16); differentiable in x,
    weight and bias (of one dtype, fp32 or bf16). `packed`: x is kept in 8 bits for the
    backward pass (1.03 bytes a value), which uses those values in x's place."""
    if bias is not None and weight is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have one dtype")
    if bias is not None and weight is None and bias.dtype != torch.float32 and bias.requires_grad:
        raise TypeError("a bias without a weight must be float32 to have a gradient")
    return (PackedLayerNormFunction if packed else LayerNormFunction).apply(x, weight, bias, float(eps))


class FusedLayerNorm(torch.nn.Module):
    """nn.Module form: FusedLayerNorm(hidden)(x)."""

    def __init__(self, hidden_size: int, eps: float = 1e-5, bias: bool = True, device=None,
                 dtype=None, packed: bool = False):
        super().__init__()
        self.eps = float(eps)
        self.packed = bool(packed)
        self.weight = torch.nn.Parameter(torch.ones(hidden_size, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(hidden_size, device=device, dtype=dtype)) if bias else None

    def forward(self, x):
        return fused_layer_norm(x, self.weight, self.bias, self.eps, self.packed)


def fused_embedding(tokens, weight, *, scale: float = 1.0, ignore_index: int = -100, dtype=None):
    """scale * weight[tokens] of integer tokens [...], as `dtype` (fp32 or bf16; the weight's by
    default); rows of ignore_index are 0, of other ids outside the table NaN. Differentiable in weight [V, D] (fp32 or bf16), whose
    gradient sums each id's tokens in fp32 in a fixed order."""
    return EmbeddingFunction.apply(tokens, weight, float(scale), int(ignore_index), dtype)


class FusedEmbedding(torch.nn.Module):
    """nn.Module form: FusedEmbedding(vocab, hidden)(tokens). A table shared with the head is
    its `weight`."""

    def __init__(self, num_embeddings: int, embedding_dim: int, scale: float = 1.0, ignore_index: int = -100,
                 device=None, dtype=None, out_dtype=None):
        super().__init__()
        self.scale, self.ignore_index, self.out_dtype = float(scale), int(ignore_index), out_dtype
        self.weight = torch.nn.Parameter(torch.randn(num_embeddings, embedding_dim, device=device, dtype=dtype))

    def forward(self, tokens):
        return fused_embedding(tokens, self.weight, scale=self.scale, ignore_index=self.ignore_index,
                               dtype=self.out_dtype)
