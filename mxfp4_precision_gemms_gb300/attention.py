"""Attention between the query-key-value projection and the output projection of a decoder block, for PyTorch autograd.

``qk_norm_rope`` norms each head of queries and keys and rotates it by position, in one pass; ``attention`` is softmax
attention over packed sequences or a batch of equal lengths.  With the MXFP4 linear layers they make a decoder block:

    q, k, v = (mxfp4_linear(x, w) for w in (wq, wk, wv))         # as [tokens, heads, head_dim]
    q, k = qk_norm_rope(q, k, rope, positions, q_gain, k_gain)
    y = mxfp4_linear(attention(q, k, v, cu_q=edges).flatten(-2), wo)

Every step runs in the CUDA library; this file only wires the calls into autograd.  What attention keeps between the two
passes is its inputs, its output with the rest of its rounding, and one fp32 number for each query and head.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as mx

Rope = mx.Rope


def _rows(x: torch.Tensor, name: str, align: int) -> torch.Tensor:
    """x [tokens, heads, head_dim] or [batch, length, heads, head_dim] as the library takes it: three dimensions, heads that
    do not overlap (a broadcast gradient's do), contiguous and on multiples of `align` bytes; copied where it is not so."""
    if x.dim() not in (3, 4):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] or [batch, length, heads, head_dim], not {tuple(x.shape)}")
    if x.dim() == 4:
        x = x.reshape(x.shape[0] * x.shape[1], *x.shape[2:])
    n, heads, dim = x.shape
    token, head, inner = x.stride()
    size = x.element_size()
    if ((dim > 1 and inner != 1) or (n > 1 and (token < dim or token * size % align))
            or (heads > 1 and (head < dim or head * size % align)) or x.data_ptr() % align):
        x = x.clone(memory_format=torch.contiguous_format)
    return x


def _gain(gain: torch.Tensor | None) -> torch.Tensor | None:
    return None if gain is None else gain.float().contiguous()


class QkNormRopeFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, rope, positions, q_gain, k_gain, eps):
        q3, k3 = _rows(q, "q", q.element_size()), _rows(k, "k", k.element_size())
        gains = _gain(q_gain), _gain(k_gain)
        if positions is not None:  # the axes, if it has them, and the tokens
            lead = positions.shape[:1] if positions.dim() == q.dim() - 1 else ()
            positions = positions.reshape(*lead, q3.shape[0]).contiguous()
        q_out, k_out = mx.qk_norm_rope(q3, k3, rope, positions, *gains, eps=eps)
        ctx.save_for_backward(None if q_gain is None else q3, None if k_gain is None else k3, positions, *gains)
        ctx.rope, ctx.eps, ctx.shapes = rope, eps, (q.shape, k.shape)
        ctx.gains = [None if g is None else (g.dtype, g.shape) for g in (q_gain, k_gain)]
        return q_out, k_out  # not as views made here, which torch lets nobody change in place

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        q, k, positions, q_gain, k_gain = ctx.saved_tensors
        dq, dk = _rows(dq, "dq", dq.element_size()), _rows(dk, "dk", dk.element_size())
        dq, dk, *gains = mx.qk_norm_rope_grad(q, k, dq, dk, ctx.rope, positions, q_gain, k_gain, eps=ctx.eps,
                                              gains=any(ctx.needs_input_grad[4:6]))
        dq_gain, dk_gain = (None if g is None else g.to(kind[0]).view(kind[1]) for g, kind in zip(gains, ctx.gains))
        return dq.reshape(ctx.shapes[0]), dk.reshape(ctx.shapes[1]), None, None, dq_gain, dk_gain, None


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, rope: Rope | None = None, positions: torch.Tensor | None = None,
                 q_gain: torch.Tensor | None = None, k_gain: torch.Tensor | None = None,
                 eps: float = 1e-6) -> tuple[torch.Tensor, torch.Tensor]:
    """Each head of q and k divided by its root mean square and multiplied by its gain ([head_dim]; None: left as it is),
    then rotated.  q and k: [tokens, heads, head_dim] or [batch, length, heads, head_dim], fp32 or bf16 both; head_dim even,
    at most 256; gains of head_dim elements in any shape.  `rope`: Rope(frequencies, axis of each pair, interleaved) or
    None; positions: int32 or int64 of q's leading shape, behind a dimension of rope.axes (which may be left out where
    that is 1).  Gradients of q, k and the gains; sums in fp32, the same bits on every run."""
    if q.dim() != k.dim() or q.shape[:-2] != k.shape[:-2]:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} do not fit together")
    if rope is not None:
        lead = tuple(q.shape[:-2])
        if positions is None or tuple(positions.shape) not in ((rope.axes, *lead), lead if rope.axes == 1 else None):
            raise ValueError(f"positions must be {(rope.axes, *lead) if rope.axes > 1 else lead}")
    q_out, k_out = QkNormRopeFunction.apply(q, k, rope, positions if rope is not None else None, q_gain, k_gain, eps)
    return (q_out, k_out) if q.dim() == 3 else (q_out.view(q.shape), k_out.view(k.shape))


class AttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, scale, cu_q, cu_k, seqs):
        q3, k3, v3 = _rows(q, "q", 16), _rows(k, "k", 16), _rows(v, "v", 16)
        out, lse, rest = mx.attention(q3, k3, v3, causal=causal, scale=scale, cu_q=cu_q, cu_k=cu_k, seqs=seqs, rest=True)
        ctx.save_for_backward(q3, k3, v3, out, lse, rest, cu_q, cu_k)
        ctx.args, ctx.shapes = (causal, scale, seqs), (q.shape, k.shape)
        return out  # not as a view made here, which torch lets nobody change in place

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, rest, cu_q, cu_k = ctx.saved_tensors
        causal, scale, seqs = ctx.args
        dq, dk, dv = mx.attention_grad(q, k, v, out, lse, _rows(dout, "dout", 16), causal=causal, scale=scale, cu_q=cu_q,
                                       cu_k=cu_k, seqs=seqs, rest=rest)
        return (dq.reshape(ctx.shapes[0]), dk.reshape(ctx.shapes[1]), dv.reshape(ctx.shapes[1]), None, None, None, None,
                None)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = True, scale: float | None = None,
              cu_q: torch.Tensor | None = None, cu_k: torch.Tensor | None = None) -> torch.Tensor:
    """Softmax attention: q [batch, length, q_heads, head_dim], k and v [batch, key length, k_heads, head_dim], or without
    the batch dimension one sequence, or several one behind the other: cu_q, cu_k int32 [sequences + 1], where each starts
    (cu_k None: as cu_q).  bf16; q_heads a multiple of k_heads, query head h reads key head h // (q_heads // k_heads);
    head_dim a multiple of 8, at most 128; scale 1 / sqrt(head_dim) by default.
    causal: query i of Lq sees the keys j <= i + Lk - Lq, so that the last one sees all.  A query that sees none gives zeros
    and no gradient, and so do tokens outside of all sequences.  Gradients of q, k and v; the same bits on every run.  They are made from the result, too: where
    they are wanted, change a copy of it, not itself."""
    if q.dim() != k.dim() or k.dim() != v.dim() or q.dim() not in (3, 4):
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not fit together")
    seqs = 1
    if q.dim() == 4:
        if cu_q is not None or cu_k is not None:
            raise ValueError("cu_q and cu_k are for sequences without a batch dimension")
        if not q.shape[0] == k.shape[0] == v.shape[0]:
            raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not fit together")
        seqs = q.shape[0]
    out = AttentionFunction.apply(q, k, v, causal, scale, cu_q, cu_k, seqs)
    return out if q.dim() == 3 else out.view(q.shape)
