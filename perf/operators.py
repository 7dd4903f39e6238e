"""Measured cases of the operators at the two ends of a training step: the embedding lookup and its gradient, the
softmax cross entropy of a linear output layer with its gradients, and the global gradient norm with clipping.

`own` selects the side: False computes each operator in its plain form (elementary torch operations in 32 bits, rounded
once at the end), True calls the library's entry points.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}
IGNORE = -100

# The linear layers of one Llama-3.1-8B decoder block and its two norm gains (elements of each gradient).
BLOCK = (4096 * 4096, 1024 * 4096, 1024 * 4096, 4096 * 4096, 14336 * 4096, 14336 * 4096, 4096 * 14336, 4096, 4096)


def listed():
    return [
        # One token's lookup: the smallest call, as in scoring or generating token by token.
        {"name": "embed one token", "op": "embed", "tokens": 1, "vocab": 128256, "dim": 4096, "table": "bf16",
         "out": "bf16", "scale": 1.0},
        # The lookup of a training step of 8192 tokens, scaled by sqrt(dim).
        {"name": "embed step", "op": "embed", "tokens": 8192, "vocab": 128256, "dim": 4096, "table": "bf16",
         "out": "bf16", "scale": 64.0},
        # fp32 master table, odd row length (no 16-byte rows) and an odd number of tokens.
        {"name": "embed odd rows", "op": "embed", "tokens": 5003, "vocab": 32003, "dim": 1001, "table": "f32",
         "out": "bf16", "scale": 0.5},
        # The table's gradient of the same training step, written whole.
        {"name": "embed grad step", "op": "embed_grad", "tokens": 8192, "vocab": 128256, "dim": 4096, "dy": "bf16",
         "out": "bf16", "scale": 64.0, "accumulate": False},
        # Gradient accumulation into an fp32 gradient over a long batch: only the rows that occur are touched.
        {"name": "embed grad accumulate", "op": "embed_grad", "tokens": 32768, "vocab": 32000, "dim": 4096,
         "dy": "bf16", "out": "f32", "scale": 1.0, "accumulate": True},
        # The loss of a few tokens (scoring a short continuation): latency and the read of the output layer's weights.
        {"name": "loss few tokens", "op": "loss", "tokens": 7, "vocab": 32000, "dim": 1024, "ignored": 0.0},
        # Evaluation: the loss alone over 4096 tokens of an 8B model's output layer.
        {"name": "loss evaluation", "op": "loss", "tokens": 4096, "vocab": 128256, "dim": 4096, "ignored": 0.02},
        # Fine-tuning on answers: most tokens are prompt or padding and do not count; odd sizes throughout.
        {"name": "loss and gradients masked", "op": "loss_grad", "tokens": 1531, "vocab": 50021, "dim": 1032,
         "ignored": 0.7},
        # The output layer of a training step of 8192 tokens: loss, hidden-state gradient and weight gradient.
        {"name": "loss and gradients step", "op": "loss_grad", "tokens": 8192, "vocab": 128256, "dim": 4096,
         "ignored": 0.02},
        # Gradients of a small model: many short tensors of both types, an empty one among them.
        {"name": "clip small model", "op": "clip", "sizes": "0,1,333,65536,196608,4097,257,1048576,65536,31,7,196608,"
         "65536,1024,1024,3,262144,262144,1024,99999,12345,512,512,512,131071,2048", "mix": "both", "in_place": False,
         "reach": 0.3},
        # One decoder block's fp32 gradients, clipped into the optimiser's buffers.
        {"name": "clip block f32", "op": "clip", "sizes": ",".join(map(str, BLOCK)), "mix": "f32", "in_place": False,
         "reach": 0.5},
        # Four decoder blocks' bf16 gradients in place, in the ordinary step whose norm is under the limit.
        {"name": "clip under the limit", "op": "clip", "sizes": ",".join(map(str, BLOCK * 4)), "mix": "bf16",
         "in_place": True, "reach": 2.0},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "loss", "loss_grad", "clip"])
    if op == "embed":
        return {"op": op, "tokens": _log_int(rng, 1, 32768), "vocab": _log_int(rng, 1000, 128256),
                "dim": _log_int(rng, 64, 4096), "table": rng.choice(["bf16", "f32"]),
                "out": rng.choice(["bf16", "f32"]), "scale": rng.choice([1.0, 0.5, 11.3])}
    if op == "embed_grad":
        return {"op": op, "tokens": _log_int(rng, 1, 32768), "vocab": _log_int(rng, 1000, 128256),
                "dim": _log_int(rng, 64, 4096), "dy": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"]),
                "scale": rng.choice([1.0, 0.5, 11.3]), "accumulate": rng.random() < 0.4}
    if op in ("loss", "loss_grad"):
        # at most an eighth of the largest listed case's product, so that the plain form stays short
        while True:
            c = {"op": op, "tokens": _log_int(rng, 1, 8192), "vocab": _log_int(rng, 1000, 128256),
                 "dim": 8 * _log_int(rng, 8, 512), "ignored": rng.choice([0.0, 0.02, 0.3, 0.9])}
            if c["tokens"] * c["vocab"] * c["dim"] <= 8192 * 128256 * 512:
                return c
    total, n = _log_int(rng, 1000, 400_000_000), _log_int(rng, 1, 60)
    cuts = [rng.random() ** 3 + 1e-6 for _ in range(n)]
    sizes = [int(total * c / sum(cuts)) for c in cuts]
    sizes[0] += total - sum(sizes)
    in_place = rng.random() < 0.3
    return {"op": op, "sizes": ",".join(map(str, sizes)), "mix": rng.choice(["f32", "bf16", "both"]),
            "in_place": in_place, "reach": 2.0 if in_place else rng.choice([0.1, 0.6, 3.0])}


def _clip_types(case):
    n = len(case["sizes"].split(","))
    if case["mix"] == "both":
        return [BF16 if i % 2 else F32 for i in range(n)]
    return [DTYPES[case["mix"]]] * n


def _ids(tokens, vocab, g):
    """Token ids whose frequency falls with the id, roughly as 1 / (id + 1)."""
    u = torch.rand(tokens, device="cuda", generator=g, dtype=torch.float64)
    return ((vocab + 1.0) ** u - 1.0).long().clamp_(0, vocab - 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=BF16, std=1.0):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        x.normal_(0.0, std, generator=g)
        return x

    s = dict(case)
    op = case["op"]
    if op == "embed":
        s["ids"] = _ids(case["tokens"], case["vocab"], g)
        s["w"] = normal(case["vocab"], case["dim"], dtype=DTYPES[case["table"]], std=0.02)
    elif op == "embed_grad":
        s["ids"] = _ids(case["tokens"], case["vocab"], g)
        s["padding"] = int(s["ids"][0]) if case["tokens"] > 3 else -1
        s["grad"] = normal(case["tokens"], case["dim"], dtype=DTYPES[case["dy"]], std=1e-3)
        if case["accumulate"]:
            s["dw"] = normal(case["vocab"], case["dim"], dtype=DTYPES[case["out"]], std=1e-3)
    elif op in ("loss", "loss_grad"):
        T, V, D = case["tokens"], case["vocab"], case["dim"]
        s["w"] = normal(V, D, std=0.02 * math.sqrt(4096 / D))
        targets = _ids(T, V, g)
        # normalised hidden states that point to their target, from not at all to firmly (target logits up to 12)
        h = normal(T, D, dtype=F32)
        h += (7.3 * torch.rand(T, 1, device="cuda", generator=g) ** 2) * s["w"][targets].float()
        s["h"] = h.to(BF16)
        if case["ignored"]:
            out = torch.rand(T, device="cuda", generator=g) < case["ignored"]
            targets = torch.where(out, torch.full_like(targets, IGNORE), targets)
        s["targets"] = targets
        s["upstream"] = torch.ones(1, device="cuda")
    else:
        sizes = [int(x) for x in case["sizes"].split(",")]
        types = _clip_types(case)
        s["grads"] = [normal(n, dtype=t, std=1e-3) for n, t in zip(sizes, types)]
        # the limit: `reach` times the norm that is expected of these draws
        s["max_norm"] = case["reach"] * 1e-3 * math.sqrt(max(1, sum(sizes)))
        s["outs"] = s["grads"] if case["in_place"] else [torch.empty_like(x) for x in s["grads"]]
    return s


def _run_own(s):
    from mxfp4_precision_gemms_gb300 import binding as mx

    kind = {"bf16": mx.OUT_BF16, "f32": mx.OUT_F32}
    op = s["op"]
    if op == "embed":
        return mx.embedding(s["ids"], s["w"], scale=s["scale"], out_dtype=kind[s["out"]])
    if op == "embed_grad":
        return mx.embedding_grad(s["ids"], s["grad"], s["vocab"], scale=s["scale"], padding_id=s["padding"],
                                 out_dtype=kind[s["out"]], accumulate=s["accumulate"], dw=s.get("dw"))
    if op == "loss":
        loss, lse = mx.linear_ce(s["h"], s["w"], s["targets"], ignore_index=IGNORE, reduction=mx.REDUCE_NONE)
        return {"loss": loss, "lse": lse}
    if op == "loss_grad":
        loss, lse = mx.linear_ce(s["h"], s["w"], s["targets"], ignore_index=IGNORE, reduction=mx.REDUCE_MEAN)
        dh, dw = mx.linear_ce_grad(s["h"], s["w"], s["targets"], lse, s["upstream"], ignore_index=IGNORE,
                                   reduction=mx.REDUCE_MEAN, dh_dtype=mx.OUT_BF16, dw_dtype=mx.OUT_BF16)
        return {"loss": loss, "dh": dh, "dw": dw}
    norm = mx.clip_grad_norm(s["grads"], s["max_norm"], outs=None if s["in_place"] else s["outs"])
    return {"norm": norm, "grads": s["outs"]}


def _run_plain(s):
    op = s["op"]
    if op == "embed":
        return (s["w"][s["ids"]].float() * s["scale"]).to(DTYPES[s["out"]])
    if op == "embed_grad":
        add = s["grad"].float() * s["scale"] * (s["ids"] != s["padding"]).float()[:, None]
        if s["accumulate"] and s["out"] == "f32":
            return s["dw"].index_add_(0, s["ids"], add)
        dw = torch.zeros(s["vocab"], s["dim"], device="cuda") if not s["accumulate"] else s["dw"].float()
        dw.index_add_(0, s["ids"], add)
        return s["dw"].copy_(dw) if s["accumulate"] else dw.to(DTYPES[s["out"]])
    if op in ("loss", "loss_grad"):
        targets = s["targets"]
        counted = targets != IGNORE
        at = torch.where(counted, targets, torch.zeros_like(targets))[:, None]
        h = s["h"].float() * counted.float()[:, None]
        w = s["w"].float()
        z = h @ w.t()
        top = z.amax(1, keepdim=True)
        lse = (z - top).exp_().sum(1).log() + top[:, 0]
        loss = (lse - z.gather(1, at)[:, 0]) * counted.float()
        if op == "loss":
            return {"loss": loss, "lse": lse * counted.float()}
        n = counted.sum().clamp(min=1).float()
        dz = z.sub_(lse[:, None]).exp_()
        dz.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
        dz *= (s["upstream"] * counted.float() / n)[:, None]
        return {"loss": (loss.sum() / n).reshape(1), "dh": (dz @ w).to(BF16), "dw": (dz.t() @ h).to(BF16)}
    norm = torch.stack([x.float().square().sum() for x in s["grads"]]).sum().sqrt()
    by = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": norm.reshape(1), "grads": [o.copy_(x.float() * by) for o, x in zip(s["outs"], s["grads"])]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _distinct(tokens, vocab):
    """How many different ids _ids() is expected to give."""
    p = np.log1p(1.0 / np.arange(1, vocab + 1)) / math.log(vocab + 1.0)
    return float(np.sum(-np.expm1(tokens * np.log1p(-p))))


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "embed":
        T, D = case["tokens"], case["dim"]
        return {"bytes": T * D * (size[case["table"]] + size[case["out"]]) + 8 * T, "flops": T * D}
    if op == "embed_grad":
        T, V, D = case["tokens"], case["vocab"], case["dim"]
        rows = 2 * _distinct(T, V) if case["accumulate"] else V
        return {"bytes": T * D * size[case["dy"]] + 8 * T + rows * D * size[case["out"]], "flops": T * D}
    if op in ("loss", "loss_grad"):
        T, V, D = case["tokens"], case["vocab"], case["dim"]
        n = T * (1.0 - case["ignored"])
        once = 2 * (n + V) * D + 8 * T
        if op == "loss":
            return {"bytes": once + 8 * T, "flops": 2 * n * V * D}
        return {"bytes": once + 2 * (T + V) * D + 4, "flops": 6 * n * V * D}
    sizes = [int(x) for x in case["sizes"].split(",")]
    held = sum(n * (2 if t is BF16 else 4) for n, t in zip(sizes, _clip_types(case)))
    return {"bytes": held if case["in_place"] else 2 * held, "flops": 3 * sum(sizes)}


def exact(case, seed):
    # the gradient products in 64 bits are left out where they would take over about 20 seconds
    whole = 6.0 * case.get("tokens", 0) * case.get("vocab", 0) * case.get("dim", 0) <= 8e12
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        return torch.index_select(s["w"], 0, s["ids"]).double().mul_(case["scale"])
    if op == "embed_grad":
        keep = torch.nonzero(s["ids"] != s["padding"])[:, 0]
        dw = s["dw"].double() if case["accumulate"] else torch.zeros(case["vocab"], case["dim"], dtype=torch.float64,
                                                                      device="cuda")
        return dw.index_put_((s["ids"][keep],), s["grad"][keep].double() * case["scale"], accumulate=True)
    if op in ("loss", "loss_grad"):
        # counted tokens alone, then laid out over all of them
        keep = torch.nonzero(s["targets"] != IGNORE)[:, 0]
        y = s["targets"][keep]
        w, h = s["w"].double(), s["h"][keep].double()
        z = torch.mm(h, w.t())
        lse = torch.logsumexp(z, 1)
        loss = lse - z[torch.arange(len(y), device="cuda"), y]
        full = torch.zeros(2, case["tokens"], dtype=torch.float64, device="cuda")
        full[0, keep], full[1, keep] = loss, lse
        if op == "loss":
            return {"loss": full[0], "lse": full[1]}
        n = max(1, len(y))
        if not whole:
            return {"loss": loss.sum().reshape(1) / n, "dh": None, "dw": None}
        dz = torch.exp(z - lse[:, None])
        dz[torch.arange(len(y), device="cuda"), y] -= 1.0
        dz /= n
        dh = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        dh[keep] = torch.mm(dz, w)
        return {"loss": loss.sum().reshape(1) / n, "dh": dh, "dw": torch.mm(dz.t(), h)}
    norm = math.sqrt(sum(float(torch.sum(x.double() ** 2)) for x in s["grads"]))
    by = min(1.0, s["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=torch.float64), "grads": [x.double() * by for x in s["grads"]]}
