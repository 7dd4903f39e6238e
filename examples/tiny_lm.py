"""Trains a small language model whose linear layers run in MXFP4, end to end on one GB300.

    python examples/tiny_lm.py [--steps 60] [--tokens 2048] [--vocab 2000] [--dim 256] [--heads 0]

Tokens come from a fixed random Markov chain (each token has four likely successors), in documents
of random length; the last token of a document has no target.  The model is an embedding, two
MXFP4 feed-forward blocks with residuals, and an output layer:

    embedding -> [x + W2 relu(W1 x)^2] x 2 -> normalise -> cross entropy of the output layer
    backward -> global norm and clipping -> AdamW on the fp32 weights

With --heads above 0 each block has attention in front of it, within the documents: x + Wo attention(q, k, v), q and k
normed and rotated by their place in the document, four query heads (or as many as divide them) to a key head.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from mxfp4_precision_gemms_gb300.attention import Rope, attention, qk_norm_rope  # noqa: E402
from mxfp4_precision_gemms_gb300.linear import mxfp4_linear  # noqa: E402
from mxfp4_precision_gemms_gb300.step import clip_grad_norm_, embedding, linear_cross_entropy  # noqa: E402

IGNORE = -100


def batch(successors: torch.Tensor, tokens: int, g: torch.Generator):
    """A batch of `tokens` ids and targets: documents laid end to end, each a walk of the chain."""
    vocab = successors.shape[0]
    lengths = []
    while sum(lengths) < tokens:
        lengths.append(int(torch.randint(8, 200, (1,), generator=g)))
    lengths[-1] -= sum(lengths) - tokens
    n = len(lengths)
    walk = torch.empty(max(lengths), n, dtype=torch.int64)
    walk[0] = torch.randint(0, vocab, (n,), generator=g)
    pick = torch.randint(0, successors.shape[1], walk.shape, generator=g)
    for i in range(1, walk.shape[0]):
        walk[i] = successors[walk[i - 1], pick[i]]
    ids = torch.cat([walk[:k, d] for d, k in enumerate(lengths)])
    targets = torch.cat([torch.cat([walk[1:k, d], torch.tensor([IGNORE])]) for d, k in enumerate(lengths)])
    return ids.cuda(), targets.cuda()


def key_heads(heads: int) -> int:
    return heads // math.gcd(heads, 4)


def make_model(vocab: int, dim: int, g: torch.Generator, heads: int = 0) -> dict:
    def weight(*shape, std):
        return (std * torch.randn(*shape, generator=g)).cuda().requires_grad_()

    p = {"embed": weight(vocab, dim, std=1.0 / math.sqrt(dim)), "out": weight(vocab, dim, std=0.02)}
    for i in range(2):
        p[f"up{i}"] = weight(4 * dim, dim, std=1.0 / math.sqrt(dim))
        p[f"down{i}"] = weight(dim, 4 * dim, std=0.2 / math.sqrt(4 * dim))
        if heads:
            size = dim // heads
            p[f"qkv{i}"] = weight((heads + 2 * key_heads(heads)) * size, dim, std=1.0 / math.sqrt(dim))
            p[f"o{i}"] = weight(dim, dim, std=0.2 / math.sqrt(dim))
            for side in "qk":
                p[f"{side}_gain{i}"] = torch.ones(size, device="cuda", requires_grad=True)
    return p


def attend(p: dict, i: int, x: torch.Tensor, heads: int, edges: torch.Tensor, places: torch.Tensor) -> torch.Tensor:
    """Block i's attention over documents that start at `edges`, of tokens at `places` in them."""
    size, kv = x.shape[1] // heads, key_heads(heads)
    qkv = mxfp4_linear(x, p[f"qkv{i}"].bfloat16()).view(-1, heads + 2 * kv, size)
    q, k, v = qkv.split([heads, kv, kv], 1)
    rope = Rope([10000.0 ** (-j / (size // 2)) for j in range(size // 2)])
    q, k = qk_norm_rope(q, k, rope, places, p[f"q_gain{i}"], p[f"k_gain{i}"])
    return mxfp4_linear(attention(q, k, v, cu_q=edges).flatten(1), p[f"o{i}"].bfloat16())


def loss_of(p: dict, ids: torch.Tensor, targets: torch.Tensor, heads: int = 0) -> torch.Tensor:
    dim = p["embed"].shape[1]
    x = embedding(ids, p["embed"], scale=math.sqrt(dim), out_dtype=torch.bfloat16)
    if heads:  # a document ends with a token that has no target
        ends = (targets == IGNORE).nonzero()[:, 0] + 1
        edges = torch.cat([ends.new_zeros(1), ends]).int()
        at = torch.arange(len(ids), device="cuda")
        places = at - edges[torch.searchsorted(ends, at, right=True)]
    for i in range(2):
        if heads:
            x = x + attend(p, i, x, heads, edges, places)
        up = torch.relu(mxfp4_linear(x, p[f"up{i}"].bfloat16()))
        x = x + mxfp4_linear(up * up, p[f"down{i}"].bfloat16())
    h = (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).bfloat16()
    return linear_cross_entropy(h, p["out"].bfloat16(), targets, ignore_index=IGNORE)


def train(steps: int = 60, tokens: int = 2048, vocab: int = 2000, dim: int = 256, max_norm: float = 1.0, seed: int = 0,
          say=print, heads: int = 0) -> list[float]:
    g = torch.Generator().manual_seed(seed)
    successors = torch.randint(0, vocab, (vocab, 4), generator=g)
    p = make_model(vocab, dim, g, heads)
    opt = torch.optim.AdamW(p.values(), lr=3e-3, betas=(0.9, 0.95), weight_decay=0.0)
    losses = []
    for step in range(steps):
        ids, targets = batch(successors, tokens, g)
        opt.zero_grad(set_to_none=True)
        loss = loss_of(p, ids, targets, heads)
        loss.backward()
        norm = clip_grad_norm_(p.values(), max_norm)
        opt.step()
        losses.append(loss.item())
        if step % 10 == 0 or step + 1 == steps:
            say(f"step {step:4d}  loss {losses[-1]:.4f}  gradient norm {norm.item():.3f}")
    return losses


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048, help="tokens of a step (a multiple of 32)")
    ap.add_argument("--vocab", type=int, default=2000)
    ap.add_argument("--dim", type=int, default=256, help="a multiple of 32")
    ap.add_argument("--heads", type=int, default=0, help="attention heads of dim / heads elements, a multiple of 32; 0: none")
    a = ap.parse_args()
    losses = train(a.steps, a.tokens, a.vocab, a.dim, heads=a.heads)
    print(f"uniform {math.log(a.vocab):.4f}, chain {math.log(4):.4f}, reached {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
