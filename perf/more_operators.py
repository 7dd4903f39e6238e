"""Measured cases of the operators between the query-key-value projection and the output projection of a decoder
block: the norm of each head of queries and keys with the rotation by position, softmax attention over packed
sequences, and the gradients of both.

`own` selects the side: False computes each operator in its plain form (elementary torch operations in 32 bits, angles
in 64, rounded once at the end), True calls the library's entry points.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "f32": F32}
EPS = 1e-6

# Documents of a packed batch of 8192 tokens: most are short, a few long, lengths of every parity.
PACKED = "1,333,2048,17,128,1201,129,777,64,255,1600,1439,200"
# Images of a vision encoder's batch, as patches.
IMAGES = "2500,1369,729,2209"


def listed():
    return [
        # One new token far into its text: the smallest call, latency.
        {"name": "rotate one token", "op": "rope", "tokens": 1, "q_heads": 32, "k_heads": 8, "dim": 128, "pairs": 64,
         "dtype": "bf16", "norm": False, "axes": 1, "interleaved": False, "base": 500000.0, "start": 120000},
        # The queries and keys of an 8B model's training step of 8192 tokens, with their norms.
        {"name": "norm and rotate step", "op": "rope", "tokens": 8192, "q_heads": 32, "k_heads": 8, "dim": 128,
         "pairs": 64, "dtype": "bf16", "norm": True, "axes": 1, "interleaved": False, "base": 500000.0, "start": 0},
        # Video: three axes, neighbouring pairs, a part of the head rotated, odd sizes, fp32.
        {"name": "norm and rotate video f32", "op": "rope", "tokens": 5003, "q_heads": 14, "k_heads": 2, "dim": 72,
         "pairs": 33, "dtype": "f32", "norm": True, "axes": 3, "interleaved": True, "base": 10000.0, "start": 7},
        # The backward pass of the training step.
        {"name": "norm and rotate gradient step", "op": "rope_grad", "tokens": 8192, "q_heads": 32, "k_heads": 8,
         "dim": 128, "pairs": 64, "dtype": "bf16", "norm": True, "axes": 1, "interleaved": False, "base": 500000.0,
         "start": 0},
        # The backward pass of a small batch with several axes and odd sizes.
        {"name": "norm and rotate gradient video", "op": "rope_grad", "tokens": 1777, "q_heads": 9, "k_heads": 3,
         "dim": 80, "pairs": 40, "dtype": "bf16", "norm": True, "axes": 3, "interleaved": False, "base": 10000.0,
         "start": 0},
        # A few tokens that continue a short prompt: latency.
        {"name": "attend few", "op": "attend", "q_lens": "3", "k_lens": "37", "q_heads": 8, "k_heads": 2, "dim": 64,
         "causal": True, "spare": 0},
        # Generating: one to five new tokens for each of four texts, over what was kept of each.
        {"name": "attend new tokens", "op": "attend", "q_lens": "1,1,5,1", "k_lens": "8001,3500,12000,517",
         "q_heads": 32, "k_heads": 8, "dim": 128, "causal": True, "spare": 0},
        # A vision encoder: every patch of an image sees the others; heads of 72.
        {"name": "attend images", "op": "attend", "q_lens": IMAGES, "k_lens": IMAGES, "q_heads": 16, "k_heads": 16,
         "dim": 72, "causal": False, "spare": 0},
        # Evaluation of one text of 8192 tokens, an 8B model's heads.
        {"name": "attend step", "op": "attend", "q_lens": "8192", "k_lens": "8192", "q_heads": 32, "k_heads": 8,
         "dim": 128, "causal": True, "spare": 0},
        # Forward and backward of a small model on one short text.
        {"name": "train small", "op": "train", "q_lens": "333", "k_lens": "333", "q_heads": 8, "k_heads": 8, "dim": 64,
         "causal": True, "spare": 0},
        # Forward and backward of a packed batch with padding behind it.
        {"name": "train packed", "op": "train", "q_lens": PACKED, "k_lens": PACKED, "q_heads": 32, "k_heads": 8,
         "dim": 128, "causal": True, "spare": 0},
        # Forward and backward of one text of 8192 tokens, an 8B model's heads.
        {"name": "train step", "op": "train", "q_lens": "8192", "k_lens": "8192", "q_heads": 32, "k_heads": 8,
         "dim": 128, "causal": True, "spare": 0},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _lens(case):
    return [int(x) for x in case["q_lens"].split(",")], [int(x) for x in case["k_lens"].split(",")]


def _pairs(case):
    """(query, key) pairs that see each other, of all sequences and one head."""
    total = 0
    for a, b in zip(*_lens(case)):
        if not case["causal"]:
            total += a * b
        else:  # query i of a sees the first b - a + i + 1 keys
            first = max(0, a - b)  # queries that see none
            total += (a - first) * (max(b - a, 0) + 1 + b) // 2
    return total


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "attend", "attend", "train", "train"])
    if op in ("rope", "rope_grad"):
        dim = rng.choice([64, 128, 128, 2 * rng.randint(8, 96), 8 * rng.randint(3, 32)])
        pairs = dim // 2 if rng.random() < 0.6 else rng.randint(1, dim // 2)
        k_heads = rng.choice([1, 2, 3, 4, 8])
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "q_heads": k_heads * rng.choice([1, 2, 3, 4]),
                "k_heads": k_heads, "dim": dim, "pairs": pairs, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "norm": rng.random() < 0.7, "axes": rng.choice([1, 1, 3]), "interleaved": rng.random() < 0.4,
                "base": rng.choice([10000.0, 500000.0, 1e6]), "start": rng.choice([0, 5, 100000, 900001])}
    while True:
        k_heads = rng.choice([1, 2, 3, 4, 8])
        c = {"op": op, "q_heads": k_heads * rng.choice([1, 1, 2, 4, 7]), "k_heads": k_heads,
             "dim": rng.choice([64, 128, 128, 8 * rng.randint(2, 16)]), "causal": rng.random() < 0.7,
             "spare": rng.choice([0, 0, 5, 130])}
        n = rng.choice([1, 1, 2, 3, 5, 9])
        longest = _log_int(rng, 1, 8192)
        q = [max(1, int(longest * rng.random() ** 2)) if i else longest for i in range(n)]
        k = q
        if op == "attend" and rng.random() < 0.5:
            k = [_log_int(rng, 1, 16384) for _ in q]
            if rng.random() < 0.5:
                q = [rng.randint(1, 8) for _ in q]
        if rng.random() < 0.2:  # a sequence of nothing
            at = rng.randint(0, n)
            q, k = q[:at] + [0] + q[at:], k[:at] + [0 if k is q else rng.randint(0, 99)] + k[at:]
        c["q_lens"], c["k_lens"] = ",".join(map(str, q)), ",".join(map(str, k))
        # no more than the largest listed case, padded to the longest sequence as the plain form has it
        if len(q) * c["q_heads"] * max(q) * max(k) * c["dim"] <= 32 * 8192 * 8192 * 128 // (1 if op == "train" else 2):
            return c


def _frequencies(case):
    return [case["base"] ** (-i / case["pairs"]) for i in range(case["pairs"])]


def _axis(case):
    """The axis of each pair: a quarter of them turns with time, the others with height and width in equal parts."""
    n = case["pairs"]
    if case["axes"] == 1:
        return [0] * n
    t = n // 4
    h = (n - t) // 2
    return [0] * t + [1] * h + [2] * (n - t - h)


def _positions(case):
    """int64 [axes, tokens]: successive positions of a text, or frames of 24 x 40 patches."""
    i = torch.arange(case["tokens"], device="cuda")
    if case["axes"] == 1:
        return (case["start"] + i)[None]
    return case["start"] + torch.stack([i // 960, i // 40 % 24, i % 40])


def _prepare_rope(case, normal):
    T, D, a, b = case["tokens"], case["dim"], case["q_heads"], case["k_heads"]
    kind = DTYPES[case["dtype"]]
    s = dict(case)
    # queries and keys as they lie in the output of one projection, in front of the values
    qkv = normal(T, (a + 2 * b) * D, dtype=kind, std=0.7).view(T, a + 2 * b, D)
    s["q"], s["k"] = qkv[:, :a], qkv[:, a:a + b]
    s["positions"] = _positions(case)
    s["freq"] = torch.tensor(_frequencies(case), dtype=F64, device="cuda")
    s["axis_of"] = torch.tensor(_axis(case), device="cuda")
    s["q_gain"] = s["k_gain"] = None
    if case["norm"]:
        s["q_gain"] = normal(D, dtype=F32, std=0.2).add_(1.0)
        s["k_gain"] = normal(D, dtype=F32, std=0.2).add_(1.0)
    if case["op"] == "rope_grad":
        s["dq"], s["dk"] = normal(T, a, D, dtype=kind, std=1e-2), normal(T, b, D, dtype=kind, std=1e-2)
    # the plan: frequencies and axes, kept on the host by the program
    s["rope"] = (tuple(_frequencies(case)), tuple(_axis(case)), case["interleaved"])
    return s


def _prepare_attention(case, normal, g):
    D, a, b = case["dim"], case["q_heads"], case["k_heads"]
    q_lens, k_lens = _lens(case)
    Tq, Tk = sum(q_lens) + case["spare"], sum(k_lens) + case["spare"]
    s = dict(case)
    if q_lens == k_lens:  # slices of one projection's output
        qkv = normal(Tq, (a + 2 * b) * D).view(Tq, a + 2 * b, D)
        q, s["k"], s["v"] = qkv[:, :a], qkv[:, a:a + b], qkv[:, a + b:]
    else:
        q, kv = normal(Tq, a, D), normal(Tk, 2 * b, D)
        s["k"], s["v"] = kv[:, :b], kv[:, b:]
    # Queries lean towards one key that they see, from not at all to firmly: scores up to some sqrt(dim).
    edge = lambda lens: torch.tensor([0] + lens, device="cuda").cumsum(0)  # noqa: E731
    cu_q, cu_k = edge(q_lens), edge(k_lens)
    seq = torch.repeat_interleave(torch.arange(len(q_lens), device="cuda"), cu_q[1:] - cu_q[:-1])
    at = torch.arange(len(seq), device="cuda") - cu_q[seq]
    seen = (cu_k[1:] - cu_k[:-1])[seq]
    if case["causal"]:
        seen = (seen - (cu_q[1:] - cu_q[:-1])[seq] + at + 1).clamp(min=0)
    u = torch.rand(len(seq), a, 2, device="cuda", generator=g)
    key = (cu_k[seq][:, None] + (u[..., 0] * seen[:, None]).long()).clamp(max=max(Tk - 1, 0))
    lean = u[..., 1] ** 2 * (seen > 0).float()[:, None]
    if len(seq) and Tk:
        head = torch.arange(a, device="cuda") // (a // b)
        q[:len(seq)] = (q[:len(seq)].float() + lean[..., None] * s["k"][key, head].float()).to(BF16)
    s["q"] = q
    # one sequence that fills its tensors needs no list of lengths
    whole = len(q_lens) == 1 and not case["spare"]
    s["cu_q"], s["cu_k"] = (None, None) if whole else (cu_q.int(), cu_k.int())
    s["edges"], s["longest"] = (cu_q, cu_k), (max(q_lens), max(k_lens))
    if case["op"] == "train":
        s["dout"] = normal(Tq, a, D)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=BF16, std=1.0):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        x.normal_(0.0, std, generator=g)
        return x

    return _prepare_rope(case, normal) if case["op"] in ("rope", "rope_grad") else _prepare_attention(case, normal, g)


def _run_own(s):
    from mxfp4_precision_gemms_gb300 import binding as mx

    op = s["op"]
    if op in ("rope", "rope_grad"):
        if isinstance(s["rope"], tuple):  # laid out once
            s["rope"] = mx.Rope(s["rope"][0], axis=s["rope"][1], interleaved=s["rope"][2])
        if op == "rope":
            q, k = mx.qk_norm_rope(s["q"], s["k"], s["rope"], s["positions"], q_gain=s["q_gain"], k_gain=s["k_gain"],
                                   eps=EPS)
            return {"q": q, "k": k}
        dq, dk, dq_gain, dk_gain = mx.qk_norm_rope_grad(s["q"], s["k"], s["dq"], s["dk"], s["rope"], s["positions"],
                                                        q_gain=s["q_gain"], k_gain=s["k_gain"], eps=EPS)
        return {"dq": dq, "dk": dk, "dq_gain": dq_gain, "dk_gain": dk_gain}
    if op == "attend":
        out, lse = mx.attention(s["q"], s["k"], s["v"], causal=s["causal"], cu_q=s["cu_q"], cu_k=s["cu_k"])
        return {"out": out, "lse": lse}
    out, lse, rest = mx.attention(s["q"], s["k"], s["v"], causal=s["causal"], cu_q=s["cu_q"], cu_k=s["cu_k"], rest=True)
    dq, dk, dv = mx.attention_grad(s["q"], s["k"], s["v"], out, lse, s["dout"], causal=s["causal"], cu_q=s["cu_q"],
                                   cu_k=s["cu_k"], rest=rest)
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def _turn(x, cos, sin, pairs, interleaved):
    """The first 2 * pairs elements of each head of x [tokens, heads, dim] turned; sin negated turns them back."""
    cos, sin = cos[:, None], sin[:, None]
    part, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :pairs], part[..., pairs:])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1), rest], -1)


def _plain_rope(s):
    angle = s["positions"][s["axis_of"]].t().double() * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    kind = DTYPES[s["dtype"]]

    def forward(x, gain):
        x = x.float()
        if gain is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain
        return _turn(x, cos, sin, s["pairs"], s["interleaved"]).to(kind)

    def backward(x, gain, dy):
        dz = _turn(dy.float(), cos, -sin, s["pairs"], s["interleaved"])
        if gain is None:
            return dz.to(kind), None
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        unit = x * r
        dunit = dz * gain
        dx = (dunit - unit * (dunit * unit).mean(-1, keepdim=True)) * r
        return dx.to(kind), (dz * unit).sum((0, 1))

    if s["op"] == "rope":
        return {"q": forward(s["q"], s["q_gain"]), "k": forward(s["k"], s["k_gain"])}
    (dq, dq_gain), (dk, dk_gain) = backward(s["q"], s["q_gain"], s["dq"]), backward(s["k"], s["k_gain"], s["dk"])
    return {"dq": dq, "dk": dk, "dq_gain": dq_gain, "dk_gain": dk_gain}


def _plain_attention(s):
    a, b, D = s["q_heads"], s["k_heads"], s["dim"]
    (cu_q, cu_k), (Lq, Lk) = s["edges"], s["longest"]
    n, scale = len(cu_q) - 1, 1.0 / math.sqrt(D)
    # sequences as a batch padded to the longest
    iq, ik = torch.arange(Lq, device="cuda"), torch.arange(Lk, device="cuda")
    len_q, len_k = (cu_q[1:] - cu_q[:-1])[:, None], (cu_k[1:] - cu_k[:-1])[:, None]
    in_q, in_k = iq < len_q, ik < len_k
    at_q, at_k = (cu_q[:-1, None] + iq) * in_q, (cu_k[:-1, None] + ik) * in_k
    seen = in_q[:, :, None] & in_k[:, None, :]
    if s["causal"]:
        seen = seen & (ik[None, None] <= (iq + len_k - len_q)[:, :, None])
    seen = seen[:, None, None]  # [n, 1, 1, Lq, Lk]

    def pad(x, at, inside):  # -> [n, heads, L, D]
        return (x[at].float() * inside[..., None, None]).transpose(1, 2)

    q = pad(s["q"], at_q, in_q).reshape(n, b, (a // b) * Lq, D)
    k, v = pad(s["k"], at_k, in_k), pad(s["v"], at_k, in_k)
    z = (q @ k.transpose(2, 3)).mul_(scale).view(n, b, a // b, Lq, Lk).masked_fill_(~seen, -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top).masked_fill(total == 0, -math.inf)
    p = p.div_(total.clamp(min=1e-30)).view(n, b, (a // b) * Lq, Lk)
    o = p @ v

    def unpad(x, heads, at, inside, like):  # [n, b, heads / b * L, D] -> like's shape, zeros outside of all sequences
        x = x.view(n, heads, inside.shape[1], D).transpose(1, 2)
        res = torch.zeros(like.shape, device="cuda")
        res[at[inside]] = x[inside]
        return res.to(BF16)

    out = unpad(o, a, at_q, in_q, s["q"])
    if s["op"] == "attend":
        flat = torch.zeros(s["q"].shape[0], a, device="cuda")
        flat[at_q[in_q]] = lse.view(n, a, Lq).transpose(1, 2)[in_q]
        return {"out": out, "lse": flat.t().contiguous()}
    do = pad(s["dout"], at_q, in_q).reshape(n, b, (a // b) * Lq, D)
    dv = p.transpose(2, 3) @ do
    dz = (do @ v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    return {"out": out, "dq": unpad(dz @ k, a, at_q, in_q, s["q"]),
            "dk": unpad(dz.transpose(2, 3) @ q, b, at_k, in_k, s["k"]), "dv": unpad(dv, b, at_k, in_k, s["v"])}


def run(state):
    if own:
        return _run_own(state)
    return _plain_rope(state) if state["op"] in ("rope", "rope_grad") else _plain_attention(state)


def work(case):
    D, a, b = case["dim"], case["q_heads"], case["k_heads"]
    if case["op"] in ("rope", "rope_grad"):
        n = case["tokens"] * (a + b) * D
        size = {"bf16": 2, "f32": 4}[case["dtype"]]
        passes = 3 if case["op"] == "rope_grad" and case["norm"] else 2
        more = 8 * case["tokens"] * case["axes"] + (16 * D if case["norm"] else 0)
        return {"bytes": passes * n * size + more, "flops": n * (12 if case["op"] == "rope_grad" else 6)}
    Tq, Tk = (sum(x) for x in _lens(case))
    product = 2 * _pairs(case) * D * a
    if case["op"] == "attend":
        return {"bytes": 4 * Tq * a * D + 4 * Tk * b * D + 4 * Tq * a, "flops": 2 * product}
    # q, k, v and the output's gradient in; the output and three gradients out; the scores made again
    return {"bytes": 2 * (4 * Tq * a * D + 4 * Tk * b * D), "flops": 7 * product}


def _exact_rope(case, s):
    D, P = case["dim"], case["pairs"]
    even = torch.arange(P, device="cuda") * 2 if case["interleaved"] else torch.arange(P, device="cuda")
    odd = even + 1 if case["interleaved"] else even + P
    turns = torch.stack([s["positions"][x].to(F64) * f for x, f in zip(_axis(case), _frequencies(case))], 1)
    # one complex factor for each token and pair
    by = torch.polar(torch.ones_like(turns), turns)[:, None, :]

    def rotate(x, back):
        c = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * (by.conj() if back else by)
        y = x.clone()
        y[..., even], y[..., odd] = c.real, c.imag
        return y

    def one(name):
        x, gain = s[name].to(F64), s[name + "_gain"]
        length = None
        if gain is not None:
            gain = gain.to(F64)
            length = torch.sqrt(torch.sum(x * x, -1, keepdim=True) / D + EPS)
        if case["op"] == "rope":
            return rotate(x if gain is None else x / length * gain, False), None
        dz = rotate(s["d" + name].to(F64), True)
        if gain is None:
            return dz, None
        # y = x / length * gain: the quotient rule
        along = torch.sum(dz * gain * x, -1, keepdim=True) / (D * length ** 3)
        return dz * gain / length - x * along, torch.sum(dz * x / length, (0, 1))

    (q, dq_gain), (k, dk_gain) = one("q"), one("k")
    if case["op"] == "rope":
        return {"q": q, "k": k}
    return {"dq": q, "dk": k, "dq_gain": dq_gain, "dk_gain": dk_gain}


def _exact_attention(case, s):
    a, b, D = case["q_heads"], case["k_heads"], case["dim"]
    q, k, v = (s[x].to(F64) for x in "qkv")
    out, lse = torch.zeros_like(q), torch.zeros(a, len(q), dtype=F64, device="cuda")
    grads = [torch.zeros_like(x) for x in (q, k, v)]
    q0 = k0 = 0
    for n, m in zip(*_lens(case)):
        hidden = None
        if case["causal"]:
            hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1)
        for h in range(a if n else 0):  # one head at a time
            g = h * b // a
            Q, K, V = q[q0:q0 + n, h], k[k0:k0 + m, g], v[k0:k0 + m, g]
            z = torch.mm(Q, K.t()) / math.sqrt(D)
            if hidden is not None:
                z[hidden] = -math.inf
            l = torch.logsumexp(z, 1) if m else torch.full((n,), -math.inf, dtype=F64, device="cuda")
            lse[h, q0:q0 + n] = l
            p = torch.exp(z - torch.where(torch.isinf(l), torch.zeros_like(l), l)[:, None])
            out[q0:q0 + n, h] = torch.mm(p, V)
            if case["op"] == "train":
                dO = s["dout"][q0:q0 + n, h].to(F64)
                dp = torch.mm(dO, V.t())
                dz = p * (dp - torch.sum(dp * p, 1, keepdim=True)) / math.sqrt(D)
                grads[0][q0:q0 + n, h] = torch.mm(dz, K)
                grads[1][k0:k0 + m, g] += torch.mm(dz.t(), Q)
                grads[2][k0:k0 + m, g] += torch.mm(p.t(), dO)
        q0, k0 = q0 + n, k0 + m
    if case["op"] == "attend":
        return {"out": out, "lse": lse}
    return {"out": out, "dq": grads[0], "dk": grads[1], "dv": grads[2]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "rope_grad"):
        return _exact_rope(case, s)
    whole = sum(n * m for n, m in zip(*_lens(case))) * case["q_heads"] * case["dim"] * (12 if case["op"] == "train"
                                                                                       else 4)
    # left out where 64 bits would take over about 20 seconds
    return _exact_attention(case, s) if whole <= 5e12 else None
