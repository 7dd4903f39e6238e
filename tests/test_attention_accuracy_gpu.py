"""How near the results come as a whole: the division by the sum of the rounded probabilities, and the rest of the output's
rounding in the gradient.  Element by element the worst case of all roundings is more than either of them gains."""
import pytest

from tests.gpu_util import gpu_ready
from tests.attention_reference import F64, TRUNC, U_BF16, U_F32

pytestmark = pytest.mark.gpu

# One rounding to bf16 is off by 2^-8 / sqrt(3) of the power of two below, in the root of the mean square, and so by 1.66e-3
# of numbers whose mantissas are spread over their logarithm.  dq and dk carry that of dz, that of the result and less than a
# third one from the output and its rest: below sqrt(3) 1.66e-3 = 2.9e-3; dv those of p and of the result, 2.35e-3.
WHOLE = 3.3e-3
# With dp - do . o taken from an output that is off by a rounding of its own, or by that of the largest probability,
# a key that has most of a row's probability keeps that rounding of dp: with scores up to 11 and more 5e-3 to 1e-2.
WITHOUT = 4.4e-3


def _exact(torch, q, k, v, do, causal):
    group = q.shape[1] // k.shape[1]
    Q, K, V, DO = (x.to(F64).transpose(0, 1) for x in (q, k, v, do))
    K, V = K.repeat_interleave(group, 0), V.repeat_interleave(group, 0)
    scale = q.shape[2] ** -0.5
    z = scale * Q @ K.transpose(1, 2)
    if causal:
        z = z.masked_fill(torch.ones_like(z[0], dtype=torch.bool).triu(1 + k.shape[0] - q.shape[0]), -torch.inf)
    p = torch.softmax(z, -1)
    o = p @ V
    dz = p * (DO @ V.transpose(1, 2) - (DO * o).sum(-1, keepdim=True)) * scale
    shared = lambda x: x.unflatten(0, (-1, group)).sum(1).transpose(0, 1)
    return p, o.transpose(0, 1), (dz @ K).transpose(0, 1), shared(dz.transpose(1, 2) @ Q), shared(p.transpose(1, 2) @ DO)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lean", [1.0, 2.0])
@pytest.mark.parametrize("D", [64, 128])
def test_gradients_as_a_whole(D, lean, causal):
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    T, a, b = 2048, 8, 2
    q, k, v, do = rand(T, a, D), rand(T, b, D), rand(T, b, D), rand(T, a, D)
    # each query leans towards a key that it sees, from not at all to firmly
    pick = (torch.rand(T, 1, device="cuda", generator=g) * torch.arange(1, T + 1, device="cuda")[:, None]).long()
    q = q + lean * torch.rand(T, a, 1, device="cuda", generator=g) ** 2 * k[pick, torch.arange(a, device="cuda") // (a // b)]
    q, k, v, do = (x.bfloat16() for x in (q, k, v, do))
    _, o, *want = _exact(torch, q, k, v, do, causal)
    off = lambda x, y: float((x.to(F64) - y).norm() / y.norm())
    out, lse, rest = mx.attention(q, k, v, causal=causal, rest=True)
    assert off(out.to(F64) + rest.to(F64), o) < off(out, o) / 2
    for got, ref, name in zip(mx.attention_grad(q, k, v, out, lse, do, causal=causal, rest=rest), want, ("dq", "dk", "dv")):
        assert off(got, ref) < WHOLE, (name, off(got, ref))
    if D == 128:  # the scores that are that large
        for got, ref, name in zip(mx.attention_grad(q, k, v, out, lse, do, causal=causal)[:2], want, ("dq", "dk")):
            assert off(got, ref) > WITHOUT, (name, off(got, ref))


@pytest.mark.parametrize("lens", [(200, 600), (300, 2100), (4, 5000)], ids=str)
@pytest.mark.parametrize("D", [64, 128])
def test_a_key_that_has_most_of_a_row_gives_its_v(D, lens):
    """out + rest is the mean of the v with weights that are each off by a rounding: by no more than these times what a v is
    off from that mean, however large the weight.  Keys of light tiles, none of which has 1/4 of the sum, are counted in full."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    n, m = lens
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    k, v = rand(m, 2, D).bfloat16(), rand(m, 2, D).bfloat16()
    # behind the first tile of keys, whose largest probability would be rounded without an error
    pick = torch.randint(128, m, (n,), device="cuda", generator=g)
    q = ((128 / D) ** 0.5 * k[pick].repeat_interleave(2, 1).float()).bfloat16()
    out, _, rest = mx.attention(q, k, v, causal=False, rest=True)
    assert (rest.to(F64).abs() <= U_BF16 * out.to(F64).abs()).all()
    p, o, *_ = _exact(torch, q, k, v, torch.zeros_like(q), False)
    heads = torch.arange(4, device="cuda") // 2
    V = v.to(F64)[:, heads].transpose(0, 1)  # [heads, keys, D]
    O = o.transpose(0, 1)
    spread = torch.stack([torch.einsum("hk,hkd->hd", p[:, i], (V - O[:, i, None]).abs()) for i in range(n)])
    most = p.amax(-1).t()[..., None]
    # a score: D products with a truncation each, and its exponential, as in the element-wise bounds
    size = D ** -0.5 * torch.einsum("thd,khd->htk", q.to(F64).abs(), k.to(F64).abs()[:, heads]).amax(-1).t()[..., None]
    rel = 2 * size * D * TRUNC + 16 * U_F32 * (size + 8)
    tol = (U_BF16 * (1 + 2 * U_BF16) + rel) * spread + U_BF16 * (1 - most) * o.abs()
    tol = tol + m * (TRUNC + U_F32) * torch.einsum("htk,hkd->thd", p, V.abs()) + U_BF16 ** 2 * o.abs()
    err = (out.to(F64) + rest.to(F64) - o).abs()
    assert (err <= tol).all(), float((err / tol).max())
    if m < 4000:  # where the sums' own length leaves it so: a rounding of the weight would be seen
        firm = (most > 0.9).expand_as(o)
        assert firm.float().mean() > 0.25 and (tol / o.abs())[firm].median() < U_BF16 / 4
