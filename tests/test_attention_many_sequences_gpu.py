"""Batches of some tens to a million sequences: every one gets what it gets in a batch of a few."""
import itertools

import pytest

from tests.gpu_util import gpu_ready
from tests.test_attention_gpu import _edges, _inputs

pytestmark = pytest.mark.gpu


def _all(torch, q, k, v, do, **kw):
    from mxfp4_precision_gemms_gb300 import binding as mx

    out, lse, rest = mx.attention(q, k, v, rest=True, **kw)
    dq, dk, dv = mx.attention_grad(q, k, v, out, lse, do, rest=rest, **kw)
    return (out, lse.t(), rest, dq), (dk, dv)


@pytest.mark.parametrize("count", [64, 127, 128, 129, 1000, 1025])
@pytest.mark.parametrize("causal", [True, False])
def test_as_in_batches_of_thirty(count, causal):
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    q_lens = [(37 * i) % 151 if i % 7 else (i * 53) % 400 for i in range(count)]
    k_lens = q_lens if causal else [(11 * i) % 190 for i in range(count)]
    q, k, v, do = _inputs(torch, q_lens, k_lens, 4, 2, 64, 21, 1)
    shift = 10  # tokens in front of the first sequence and behind the last
    a, b = _edges(torch, q_lens) + shift, _edges(torch, k_lens) + shift
    got = _all(torch, q, k, v, do, cu_q=a, cu_k=b, causal=causal)
    assert mx.device_status() == 0
    at_q, at_k = [[shift, *(shift + x for x in itertools.accumulate(lens))] for lens in (q_lens, k_lens)]
    for i in range(0, count, 30):
        j = min(i + 30, count)
        sq, sk = slice(at_q[i], at_q[j]), slice(at_k[i], at_k[j])
        want = _all(torch, q[sq], k[sk], v[sk], do[sq], cu_q=a[i:j + 1] - a[i], cu_k=b[i:j + 1] - b[i], causal=causal)
        for rows, gs, ws in zip((sq, sk), got, want):
            assert all(torch.equal(g[rows], w) for g, w in zip(gs, ws)), i
    for rows, gs in zip((at_q, at_k), got):  # outside
        assert not any(g[:rows[0]].any() or g[rows[-1]:].any() for g in gs)


@pytest.mark.parametrize("count", [5000, 40000, 1_000_000])
def test_very_many_short_sequences(count):
    """Sequences of up to three tokens, whose few numbers torch finds at once."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    g = torch.Generator(device="cuda").manual_seed(2)
    lens = torch.randint(0, 4, (count,), device="cuda", generator=g)
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).int()
    T = int(cu[-1])
    q, k, v, do = (torch.randn(T, h, 32, device="cuda", generator=g).bfloat16() for h in (2, 1, 1, 2))
    out, lse, rest = mx.attention(q, k, v, cu_q=cu, rest=True)
    dq, dk, dv = mx.attention_grad(q, k, v, out, lse, do, cu_q=cu, rest=rest)
    assert mx.device_status() == 0
    # a token sees itself and up to two before it, in its own sequence
    x = [t.double().requires_grad_() for t in (q, k, v)]
    seq = torch.repeat_interleave(torch.arange(count, device="cuda"), lens)
    at = torch.arange(T, device="cuda")
    back = at[:, None] - torch.arange(3, device="cuda")
    seen = (back >= 0) & (seq[back.clamp(min=0)] == seq[:, None])
    keys, values = (t[back.clamp(min=0), 0] for t in x[1:])
    z = torch.einsum("thd,tsd->ths", x[0], keys) * 32 ** -0.5
    p = torch.softmax(z.masked_fill(~seen[:, None], -torch.inf), -1)
    want = torch.einsum("ths,tsd->thd", p, values)
    (want * do.double()).sum().backward()
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    # probabilities, dz and the results are rounded to bf16: three half steps of the largest element's size at most
    assert rel(out, want.detach()) < 3 * 2.0 ** -8
    for name, got, ref in zip("qkv", (dq, dk, dv), x):
        assert rel(got, ref.grad) < 3 * 2.0 ** -8, name


@pytest.mark.parametrize("at", [1, 33, 512, 998, 1000])
def test_a_list_that_falls_among_many_is_reported(at):
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    q, k, v, do = _inputs(torch, [3000], [3000], 2, 1, 64, 0, 3)
    good = torch.arange(1001, dtype=torch.int32, device="cuda") * 3
    for value in (-1, 3001, 7 if at == 1 else 2):  # below 0, past the tensors, a fall
        bad = good.clone()
        bad[at] = value
        for a, b in ((bad, good), (good, bad)):
            out, lse = mx.attention(q, k, v, cu_q=a, cu_k=b)
            assert mx.device_status() == 1, value
            mx.attention_grad(q, k, v, out, lse, do, cu_q=a, cu_k=b)
            assert mx.device_status() == 1, value
    mx.attention(q, k, v, cu_q=good)
    assert mx.device_status() == 0
