"""Global gradient norm and clipping (mxfp4_clip_grad_norm) against the formula in 64 bits.
Tolerances: the sum of squares is one of fp32 additions, none of whose chains is longer here than 64 squares of
a chunk in a thread (two sums of 32), 8 chunks, and trees of 8 levels over a CTA and 8 + 8 over the CTAs: it
is off by less than 58 * 2^-24 of itself, and the norm by half of that, plus its rounding to fp32; the
coefficient adds three roundings, and each output one more (2^-9 of its binade in bf16)."""
import math

import pytest

from tests.gpu_util import gpu_ready

pytestmark = pytest.mark.gpu

REL = 30 * 2.0 ** -24


def _setup():
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    return torch, mx


def _grads(torch, sizes, kinds, seed=0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = torch.bfloat16 if kinds == "bf16" or (kinds == "both" and i % 2) else torch.float32
        base = torch.randn(n + offset, device="cuda", generator=g).to(dt)
        out.append(base[offset:])
    return out


def _check(torch, mx, grads, max_norm, in_place):
    want_n = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    c = min(1.0, max_norm / (want_n + 1e-6))
    want = [g.double() * c for g in grads]
    kept = [g.clone() for g in grads]
    outs = None if in_place else [torch.full_like(g, 7.0) for g in grads]
    norm = mx.clip_grad_norm(grads, max_norm, outs=outs)
    assert mx.device_status() == 0
    assert norm.shape == (1,) and abs(float(norm) - want_n) <= REL * want_n
    for g, k, o, w in zip(grads, kept, outs or grads, want):
        tol = (2 * REL + (2.0 ** -8 if o.dtype == torch.bfloat16 else 0.0)) * w.abs() + 2.0 ** -140
        assert bool(((o.double() - w).abs() <= tol).all())
        if not in_place:
            assert torch.equal(g, k)
        elif c == 1.0:
            assert torch.equal(g, k)


@pytest.mark.parametrize("kinds", ["f32", "bf16", "both"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("sizes", [[1], [0], [0, 0, 5, 0], [2047, 2048, 2049, 0, 1, 16385], [1000003],
                                   [333] * 65, [7] * 1100, [3_000_001, 5, 4_000_000]])
def test_norm_and_clip(kinds, in_place, sizes):
    torch, mx = _setup()
    total = sum(sizes)
    for reach in (0.3, 3.0):
        _check(torch, mx, _grads(torch, sizes, kinds), reach * math.sqrt(max(1, total)), in_place)


@pytest.mark.parametrize("offset", [1, 2, 5])
def test_unaligned_tensors(offset):
    torch, mx = _setup()
    for kinds in ("f32", "bf16"):
        _check(torch, mx, _grads(torch, [1000, 4097, 3], kinds, offset=offset), 10.0, False)
        _check(torch, mx, _grads(torch, [1000, 4097, 3], kinds, offset=offset), 10.0, True)


def test_no_gradients_and_zeros():
    torch, mx = _setup()
    assert float(mx.clip_grad_norm([], 1.0)) == 0.0
    z = torch.zeros(5000, device="cuda")
    assert float(mx.clip_grad_norm([z], 1.0)) == 0.0 and not z.any()
    x = torch.ones(100, device="cuda")
    assert float(mx.clip_grad_norm([x], 0.0)) == 10.0 and not x.any()


def test_infinite_and_nan_norms():
    """c = max_norm / inf = 0 (infinities become NaN, the rest 0); a NaN anywhere makes everything NaN."""
    torch, mx = _setup()
    for dt in (torch.float32, torch.bfloat16):
        a = torch.ones(3000, device="cuda", dtype=dt)
        b = torch.ones(10, device="cuda", dtype=dt)
        a[2999] = float("inf")
        assert math.isinf(float(mx.clip_grad_norm([a, b], 1.0)))
        assert bool(a[2999].isnan()) and not a[:2999].any() and not b.any()
        a.fill_(1.0), b.fill_(1.0)
        b[3] = float("nan")
        assert math.isnan(float(mx.clip_grad_norm([a, b], 1.0)))
        assert bool(a.isnan().all()) and bool(b.isnan().all())


def test_same_bits_other_stream_and_graph():
    torch, mx = _setup()
    grads = _grads(torch, [123457, 8, 999999], "both", seed=3)
    outs = [torch.empty_like(g) for g in grads]
    n0 = mx.clip_grad_norm(grads, 2.0, outs=outs).clone()
    o0 = [o.clone() for o in outs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n1 = mx.clip_grad_norm(grads, 2.0, outs=outs, stream=side)
    side.synchronize()
    assert torch.equal(n0, n1) and all(torch.equal(a, b) for a, b in zip(o0, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n2 = mx.clip_grad_norm(grads, 2.0, outs=outs)
    for g in grads:
        g.mul_(0.5)
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    # halving is exact, and so is its effect on every square and sum
    assert torch.equal(n2, n0 * 0.5)
    assert all(((a.double() - b.double()).abs() <= 2.0 ** -7 * a.double().abs()).all() for a, b in zip(o0, outs))


def test_tensor_past_2_31_elements():
    """2.2e9 equal bf16 gradients of 2^-10: fp32 sums of up to 2^24 of their squares (2^-20 each) are exact, which the
    CTAs' sums are; the additions over the CTAs (8 and 8 levels) and of the one other square round."""
    torch, mx = _setup()
    n = 2_200_000_000
    g = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    g[-1] = 4.0
    want = math.sqrt((n - 1) * 2.0 ** -20 + 16.0)
    norm = mx.clip_grad_norm([g], want / 2)
    assert abs(float(norm) - want) <= 12 * 2.0 ** -24 * want
    assert bool((g[:-1] == 2.0 ** -11).all()) and float(g[-1]) == 2.0
