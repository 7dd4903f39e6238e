"""The two ends of a training step for PyTorch autograd, around the MXFP4 linear layers.

``embedding`` stands in front of the first layer, ``linear_cross_entropy`` is the output layer and
the loss behind the last one, and ``clip_grad_norm_`` is for the gradients that the backward pass
leaves.  Every step runs in the CUDA library; this file only wires the calls into autograd.
The logits of the output layer are never in memory: what is kept between the two passes is one
fp32 number for each token.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import binding as mx

_REDUCTIONS = {"none": mx.REDUCE_NONE, "sum": mx.REDUCE_SUM, "mean": mx.REDUCE_MEAN}


def _rows(x: torch.Tensor) -> torch.Tensor:
    """x [..., dim] as a matrix whose rows do not overlap (a broadcast gradient's do) and are contiguous."""
    x = x.reshape(math.prod(x.shape[:-1]), x.shape[-1])
    if (x.shape[1] > 1 and x.stride(1) != 1) or (x.shape[0] > 1 and x.stride(0) < x.shape[1]):
        x = x.contiguous()
    return x


class EmbeddingFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, w, scale, padding_id, out_dtype):
        ids = ids.contiguous()
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.w_dtype, ctx.scale, ctx.padding_id = w.shape[0], w.dtype, scale, padding_id
        w = _rows(w) if w.dim() == 2 else w  # the library's own check refuses other shapes
        return mx.embedding(ids, w, scale=scale, out_dtype=None if out_dtype is None else mx._OUT_OF[out_dtype])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (ids,) = ctx.saved_tensors
        dw = mx.embedding_grad(ids.reshape(-1), _rows(dy), ctx.vocab, scale=ctx.scale, padding_id=ctx.padding_id,
                               out_dtype=mx._OUT_OF[ctx.w_dtype])
        return None, dw, None, None, None


def embedding(ids: torch.Tensor, w: torch.Tensor, scale: float = 1.0, padding_id: int = -1,
              out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """scale * w[ids] for a table w [vocab, dim] (fp32 or bf16; one whose rows are not contiguous is copied), in
    out_dtype (default: w's).  Its gradient is dense, in w's type, with each row's sum in fp32 in a fixed order;
    tokens with padding_id give none.  An id outside the vocabulary gives a row of zeros and no gradient, and no error
    here, where nothing is synchronised: binding.device_status() reports it."""
    if out_dtype is not None and out_dtype not in mx._OUT_OF:
        raise ValueError(f"out_dtype must be one of {list(mx._OUT_OF)}, not {out_dtype}")
    return EmbeddingFunction.apply(ids, w, scale, padding_id, out_dtype)


class LinearCrossEntropyFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, targets, ignore_index, reduction):
        h2, w = _rows(h), _rows(w)
        if w.data_ptr() % 16 or (w.shape[0] > 1 and w.stride(0) % 8):
            w = w.clone(memory_format=torch.contiguous_format)  # what the library asks of its rows
        y = targets.reshape(-1).contiguous()
        loss, lse = mx.linear_ce(h2, w, y, ignore_index=ignore_index, reduction=reduction)
        ctx.save_for_backward(h2, w, y, lse)
        ctx.ignore_index, ctx.reduction, ctx.shape = ignore_index, reduction, h.shape
        return loss  # not as a view made here, which torch lets nobody change in place

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        h2, w, y, lse = ctx.saved_tensors
        need_h, need_w = ctx.needs_input_grad[:2]
        dloss = dloss.reshape(-1).float().contiguous()
        dh, dw = mx.linear_ce_grad(h2, w, y, lse, dloss, ignore_index=ctx.ignore_index, reduction=ctx.reduction,
                                   dh_dtype=mx.OUT_BF16 if need_h else None, dw_dtype=mx.OUT_BF16 if need_w else None)
        return None if dh is None else dh.reshape(ctx.shape), dw, None, None, None


def linear_cross_entropy(h: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                         reduction: str = "mean") -> torch.Tensor:
    """Softmax cross entropy of the logits h w^T at `targets`: h [..., dim] and w [vocab, dim] bf16, targets
    [...] int32 or int64 (of h's leading shape, or either of the two flat); dim a multiple of 8.
    `reduction`: "mean" (over the tokens that count; 0 if none does), "sum" or "none".  Tokens whose target is
    ignore_index do not count, and their rows of h may hold anything.  Other targets outside the vocabulary do not count either, and raise no error here, where nothing
    is synchronised: binding.device_status() reports them."""
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(_REDUCTIONS)}")
    if w.dim() != 2:
        raise ValueError(f"w must be a matrix [vocab, dim], not {tuple(w.shape)}")
    # in another shape of as many elements (a batch laid out the other way) targets would be other tokens'
    if targets.shape != h.shape[:-1] and targets.dim() != 1 and h.dim() != 2:
        raise ValueError(f"targets {tuple(targets.shape)} do not fit h {tuple(h.shape)}")
    loss = LinearCrossEntropyFunction.apply(h, w, targets, ignore_index, _REDUCTIONS[reduction])
    shape = targets.shape if reduction == "none" else ()
    return loss if loss.shape == shape else loss.view(shape)


@torch.no_grad()
def clip_grad_norm_(parameters, max_norm: float) -> torch.Tensor:
    """Clips the gradients of `parameters` (one tensor or an iterable; those without a gradient are
    passed over, and one that occurs twice, as a tied weight may, counts once) to a global 2-norm of max_norm,
    in place.  Returns the norm before clipping, a 1-element fp32 CUDA tensor; nothing is synchronised.
    Gradients are fp32 or bf16, on the current device."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in dict.fromkeys(parameters) if p.grad is not None]
    # a gradient with other strides (of a transposed parameter) goes through a contiguous copy
    flat = [g if g.is_contiguous() else g.contiguous() for g in grads]
    norm = mx.clip_grad_norm(flat, max_norm)
    for g, f in zip(grads, flat):
        if f is not g:
            g.copy_(f)
    return norm
