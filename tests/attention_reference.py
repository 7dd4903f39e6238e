"""Plain 64-bit forms of the norm with rotation and of attention with their gradients, and how far the library's
results may be from them: each rounding counted at half a step of its type, each fp32 sum at its length."""
import math

import torch

F64 = torch.float64
U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -24  # half a step relative to the value
TRUNC = 2.0 ** -23                     # a tensor core's step of a sum, which is cut off


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ norm and rotation
def angles(positions, freq, axis):
    """[tokens, pairs] in radians; positions [axes, tokens]."""
    return torch.stack([positions[a].to(F64) * f for a, f in zip(axis, freq)], 1)


def turn(x, angle, interleaved, back=False):
    P = angle.shape[1]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None] * (-1 if back else 1)
    y = x.clone()
    i = torch.arange(P, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + P)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, gain, eps, angle, interleaved):
    x = x.to(F64)
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.to(F64)
    return turn(x, angle, interleaved)


def norm_rope_grad(x, dy, gain, eps, angle, interleaved):
    """(dx, dgain, magnitude of dx's terms, magnitude of dgain's sum)."""
    dz = turn(dy.to(F64), angle, interleaved, back=True)
    if gain is None:
        return dz, None, turn_size(dy, angle, interleaved), None
    x, gain = x.to(F64), gain.to(F64)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u = x * r
    du = dz * gain
    dx = r * (du - u * (du * u).mean(-1, keepdim=True))
    size = turn_size(dy, angle, interleaved) * gain.abs()
    terms = r * (size + u.abs() * (size * u.abs()).mean(-1, keepdim=True))
    big = turn_size(dy, angle, interleaved) * u.abs()
    return dx, (dz * u).sum((0, 1)), terms, big.sum((0, 1))


def turn_size(x, angle, interleaved):
    """|a| + |b| in both places of each pair: what the rounding of a turn is relative to."""
    P = angle.shape[1]
    y = x.to(F64).abs().clone()
    i = torch.arange(P, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + P)
    s = y[..., a] + y[..., b]
    y[..., a], y[..., b] = s, s
    return y


# ------------------------------------------------------------------ attention
def attend(q, k, v, q_lens, k_lens, causal, scale, dout=None, kept=True):
    """Values and tolerances, as dicts of the same keys: out, lse and, with dout, dq, dk, dv; rows outside of all sequences
    hold zeros.  kept: the gradients get the output with the rest of its rounding."""
    a, b, D = q.shape[1], k.shape[1], q.shape[2]
    dev = q.device
    Q, K, V = q.to(F64), k.to(F64), v.to(F64)
    want = {"out": torch.zeros_like(Q), "lse": torch.zeros(a, len(Q), dtype=F64, device=dev)}
    if dout is not None:
        want |= {"dq": torch.zeros_like(Q), "dk": torch.zeros_like(K), "dv": torch.zeros_like(V)}
    tol = {n: torch.zeros_like(x) for n, x in want.items()}
    tol["whole"] = torch.zeros_like(Q)  # of out + rest
    q0 = k0 = 0
    for n, m in zip(q_lens, k_lens):
        rows, cols = slice(q0, q0 + n), slice(k0, k0 + m)
        see = torch.ones(n, m, dtype=torch.bool, device=dev)
        if causal:
            see = torch.arange(m, device=dev)[None] <= torch.arange(n, device=dev)[:, None] + m - n
        for h in range(a):
            g = h // (a // b)
            x, y, w = Q[rows, h], K[cols, g], V[cols, g]
            z = (scale * x @ y.T).masked_fill(~see, -math.inf)
            lse = torch.logsumexp(z, 1) if m else torch.full((n,), -math.inf, dtype=F64, device=dev)
            p = torch.exp(z - lse.clamp(min=-1e300)[:, None])
            o = p @ w
            want["out"][rows, h], want["lse"][h, rows] = o, lse
            # a score: D products summed with a truncation each, then scaled; its exponential feels that in full, and
            # the rounding of the exponent's difference
            dz = scale * (x.abs() @ y.abs().T) * D * TRUNC
            top = torch.where(see, z, torch.zeros_like(z)).abs().amax(1, keepdim=True) if m else z.sum(1, keepdim=True)
            dz = dz + 8 * U_F32 * (top + lse.abs().nan_to_num(posinf=0.0)[:, None] + 8)
            rel = torch.where(see, dz, torch.zeros_like(dz)).amax(1, keepdim=True) if m else dz.sum(1, keepdim=True)
            # p: rounded to bf16, its own error and that of the sum that it is divided by; the sum over the keys
            ep = U_BF16 + 2 * rel + m * TRUNC
            before = ep * (p @ w.abs())  # rounding
            whole = U_BF16 ** 2 * (o.abs() + before) + before
            tol["whole"][rows, h] = whole
            tol["out"][rows, h] = U_BF16 * o.abs() + (1 + U_BF16) * before
            tol["lse"][h, rows] = (rel[:, 0] + m * U_F32 + 8 * U_F32 * (1 + lse.abs())).nan_to_num(posinf=0.0)
            if dout is None:
                continue
            do = dout[rows, h].to(F64)
            delta = (do * o).sum(1, keepdim=True)
            dp = do @ w.T
            ds = p * (dp - delta)
            want["dq"][rows, h] = scale * ds @ y
            want["dk"][cols, g] += scale * ds.T @ x
            want["dv"][cols, g] += p.T @ do
            # dz: rounded to bf16; p's error in it; that of dp and of delta, which the rounded output makes
            edelta = (do.abs() * (whole if kept else tol["out"][rows, h])).sum(1, keepdim=True) + D * U_F32 * (do.abs() * o.abs()).sum(1, keepdim=True)
            eds = (U_BF16 + 2 * rel + m * TRUNC) * ds.abs() + (1 + U_BF16) * p * (
                D * TRUNC * (do.abs() @ w.abs().T) + edelta + 4 * U_F32 * (dp.abs() + delta.abs()))
            tol["dq"][rows, h] = scale * (eds + m * TRUNC * ds.abs()) @ y.abs()
            tol["dk"][cols, g] += scale * (eds + n * a // b * TRUNC * ds.abs()).T @ x.abs()
            tol["dv"][cols, g] += ((U_BF16 + 2 * rel + n * a // b * TRUNC) * p).T @ do.abs()
        q0, k0 = q0 + n, k0 + m
    for n in ("dq", "dk", "dv"):
        if n in want:  # the result's own rounding, after the errors above
            tol[n] = tol[n] * (1 + U_BF16) + U_BF16 * want[n].abs()
    return want, tol


def assert_close(got, want, tol, what=""):
    got = got.to(F64)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    bad = ~same & ~((got - want).abs() <= tol)
    if bad.any():
        at = bad.nonzero()[:4].tolist()
        detail = ", ".join(f"{tuple(i)}: got {got[tuple(i)].item():.6e} want {want[tuple(i)].item():.6e} "
                           f"tolerance {tol[tuple(i)].item():.2e}" for i in at)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; {detail}")
