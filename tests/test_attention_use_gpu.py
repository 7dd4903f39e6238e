"""Rotation and attention as a program uses them: strides, what may not be touched and what may not reach a sequence,
streams and graphs, long offsets, refusals, and the autograd forms in a run together."""
import itertools
import math

import pytest

from tests.gpu_util import gpu_ready
from tests.test_attention_gpu import _check, _edges, _inputs

pytestmark = pytest.mark.gpu


def _all(torch, q, k, v, do, cu, **kw):
    from mxfp4_precision_gemms_gb300 import binding as mx

    out, lse, rest = mx.attention(q, k, v, cu_q=cu, rest=True, **kw)
    return (out, lse, rest, *mx.attention_grad(q, k, v, out, lse, do, cu_q=cu, rest=rest, **kw))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads", [(4, 2), (7, 1)])
def test_other_sequences_reach_nothing(heads, value):
    """What sequences beside it and tokens outside of all hold changes no bit of a sequence's results."""
    torch = gpu_ready()
    lens = [130, 77, 200, 5]
    for D in (64, 72, 128):
        q, k, v, do = _inputs(torch, lens, lens, *heads, D, 40, 1)
        cu = _edges(torch, lens)
        for causal in (True, False):
            want = _all(torch, q, k, v, do, cu, causal=causal)
            dirty = [x.clone() for x in (q, k, v, do)]
            for x in dirty:  # the second sequence, the last one, and what is behind it
                x[130:207] = value
                x[407:] = value
            got = _all(torch, *dirty, cu, causal=causal)
            for w, g in zip(want, got):
                w, g = (w.t()[..., None], g.t()[..., None]) if w.dim() == 2 else (w, g)
                assert torch.equal(w[:130], g[:130]) and torch.equal(w[207:407], g[207:407])
                assert torch.equal(g[412:], torch.zeros_like(g[412:]))


def test_rows_outside_of_all_sequences_are_left():
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    lens, spare = [33, 150], 30
    q, k, v, do = _inputs(torch, lens, lens, 4, 2, 64, spare, 2)
    cu = _edges(torch, lens) + 7  # tokens in front of the first, too
    out, lse = torch.full_like(q, 3.0), torch.full((4, len(q)), 5.0, device="cuda")
    mx.attention(q, k, v, cu_q=cu, out=out, lse=lse)
    # gradients as slices of one buffer
    buf = torch.full((len(q), 8, 64), 9.0, device="cuda").bfloat16()
    dq, dk, dv = mx.attention_grad(q, k, v, out, lse, do, cu_q=cu, dq=buf[:, :4], dk=buf[:, 4:6], dv=buf[:, 6:])
    assert dq.data_ptr() == buf.data_ptr()
    outside = [*range(7), *range(190, len(q))]
    assert (out[outside] == 3).all() and (lse[:, outside] == 5).all() and (buf[outside] == 9).all()
    inside = slice(7, 190)
    _, _, _, *want = _all(torch, q[inside], k[inside], v[inside], do[inside], _edges(torch, lens))
    got = mx.attention_grad(q[inside], k[inside], v[inside], out[inside], lse[:, inside].contiguous(), do[inside],
                            cu_q=_edges(torch, lens))
    assert all(torch.equal(a, b[inside]) for a, b in zip(got, (dq, dk, dv)))
    for a, b in zip(got, want):  # the rest of the output's rounding makes no more of a difference than that rounding
        assert float((a.float() - b.float()).norm() / b.float().norm()) < 2.0 ** -6


@pytest.mark.parametrize("few", [True, False])
def test_rows_outside_become_zeros(few):
    """New outputs hold zeros there, whatever was in their memory, and given ones beside new ones are left."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    q_lens, k_lens = ([2, 1], [3000, 1100]) if few else ([300, 4, 90], [300, 4, 90])
    q, k, v, do = _inputs(torch, q_lens, k_lens, 6, 2, 72, 50, 14)
    for shift, drop in ((0, 0), (11, 0), (50, 0), (0, 1), (20, len(q_lens))):  # drop: sequences left out at the end
        a, b = (_edges(torch, x)[:len(x) + 1 - drop] + shift for x in (q_lens, k_lens))
        junk = [torch.full_like(q, math.nan) for _ in range(6)] + [torch.full_like(k, math.nan) for _ in range(4)]
        del junk  # what new tensors are made of
        out, lse, rest = mx.attention(q, k, v, cu_q=a, cu_k=b, rest=True)
        dq, dk, dv = mx.attention_grad(q, k, v, out, lse, do, cu_q=a, cu_k=b, rest=rest)
        for x, edges in ((out, a), (rest, a), (lse.t(), a), (dq, a), (dk, b), (dv, b)):
            assert not x[:edges[0]].any() and not x[edges[-1]:].any()
            assert torch.isfinite(x[edges[0]:edges[-1]].float()).all()
        mine = torch.full_like(q, 2.0)
        _, other = mx.attention(q, k, v, cu_q=a, cu_k=b, out=mine)
        assert torch.equal(other, lse) and (mine[a[-1]:] == 2).all() and torch.equal(mine[a[0]:a[-1]], out[a[0]:a[-1]])
        mine = torch.full_like(k, 2.0)
        got = mx.attention_grad(q, k, v, out, lse, do, cu_q=a, cu_k=b, rest=rest, dv=mine)
        assert torch.equal(got[0], dq) and torch.equal(got[1], dk) and (mine[b[-1]:] == 2).all()
    assert mx.device_status() == 0


def test_many_sequences():
    """More than a warp has lanes, in an order of lengths that goes up and down."""
    torch = gpu_ready()
    lens = [(37 * i) % 151 for i in range(90)]
    q, k, v, do = _inputs(torch, lens, lens, 2, 2, 64, 0, 15)
    _check(torch, q, k, v, do, lens, lens, True)
    for n in (31, 32, 33):
        T = sum(lens[:n])
        _check(torch, q[:T], k[:T], v[:T], do[:T], lens[:n], lens[:n], True)
        _check(torch, q[:T], k[:T], v[:T], do[:T], lens[:n], lens[:n], False)


def test_layouts():
    """Heads of tokens, slices of a projection's output, a tensor with gaps: the same bits."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    lens = [150, 90]
    q, k, v, do = _inputs(torch, lens, lens, 6, 2, 80, 0, 3)
    cu = _edges(torch, lens)
    want = _all(torch, q, k, v, do, cu)
    heads_first = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)
    wide = lambda x: torch.randn(x.shape[0], x.shape[1] + 3, x.shape[2] + 16, device="cuda").bfloat16()[:, 1:-2, 8:-8].copy_(x)
    for lay in (heads_first, wide):
        got = _all(torch, *(lay(x) for x in (q, k, v, do)), cu)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        out = lay(torch.zeros_like(q))
        mx.attention(q, k, v, cu_q=cu, out=out)
        assert torch.equal(out, want[0])
        dq, dk, dv = (lay(torch.zeros_like(x)) for x in (q, k, k))
        mx.attention_grad(q, k, v, want[0], want[1], do, cu_q=cu, dq=dq, dk=dk, dv=dv, rest=want[2])
        assert all(torch.equal(a, b) for a, b in zip(want[3:], (dq, dk, dv)))


def test_offsets_above_32_bits():
    """Rows more than 2^31 elements, and 2^32 bytes, apart."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    q, k, v, do = _inputs(torch, [5, 300], [5, 300], 2, 1, 64, 0, 4)
    buf = torch.empty(305 * 8_000_000, dtype=torch.bfloat16, device="cuda")
    far = lambda x, at: buf.as_strided(x.shape, (8_000_000, 1_000_000, 1), at)
    spread = [far(x, 64 * i).copy_(x) for i, x in enumerate((q, k, v, do))]
    cu = _edges(torch, [5, 300])
    want = _all(torch, q, k, v, do, cu)
    got = _all(torch, *spread, cu)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    outs = [far(x, 64 * (i + 4)) for i, x in enumerate((q, q, k, k))]
    mx.attention(q, k, v, cu_q=cu, out=outs[0])
    mx.attention_grad(q, k, v, want[0], want[1], do, cu_q=cu, dq=outs[1], dk=outs[2], dv=outs[3], rest=want[2])
    assert all(torch.equal(a, b) for a, b in zip((want[0], *want[3:]), outs))
    rope = mx.Rope([1.0 / (i + 1) for i in range(32)])
    pos = torch.arange(305, device="cuda")
    g = torch.rand(64, device="cuda")
    a = mx.qk_norm_rope(q, k, rope, pos, g, g)
    b = mx.qk_norm_rope(spread[0], spread[1], rope, pos, g, g, q_out=outs[0], k_out=outs[2])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_long_text():
    torch = gpu_ready()
    q, k, v, do = _inputs(torch, [3], [70001], 2, 1, 64, 0, 5, lean=2.0)
    _check(torch, q, k, v, do, [3], [70001], True)


@pytest.mark.parametrize("n,m", [(0, 0), (0, 9), (9, 0)])
def test_nothing(n, m):
    torch = gpu_ready()
    q, k, v, do = _inputs(torch, [n], [m], 4, 2, 64, 0, 6)
    for listed in (True, False):
        out, lse, dq, dk, dv = _check(torch, q, k, v, do, [n], [m], True, listed=listed)
        assert not out.any() and not dq.any() and not dk.any() and not dv.any() and (lse == -math.inf).all()


def test_lists_that_point_outside_are_reported():
    """Sequences are cut to the tensors, and the status says so."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    q, k, v, do = _inputs(torch, [200], [200], 4, 2, 64, 0, 7)
    for bad in ([0, 50, 20, 200], [-5, 100, 150, 200], [0, 100, 150, 4000], [0, 300, 400, 500], [7, 5, 3, 1]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for a, b in ((cu, cu), (_edges(torch, [50, 50, 100]), cu), (cu, _edges(torch, [50, 50, 100]))):
            out, lse = mx.attention(q, k, v, cu_q=a, cu_k=b)
            assert mx.device_status() == 1
            mx.attention_grad(q, k, v, out, lse, do, cu_q=a, cu_k=b)
            assert mx.device_status() == 1
    _all(torch, q, k, v, do, _edges(torch, [50, 50, 100]))
    assert mx.device_status() == 0


def test_lists_that_fall_where_keys_are_shared_out():
    """A list that names more keys than there are has more parts than places: it is reported, and reads nothing else."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    q, k, v, do = _inputs(torch, [1, 1, 1], [2000, 2500, 1500], 4, 2, 64, 0, 8)
    cu_q = _edges(torch, [1, 1, 1])
    for bad in ([0, 6000, 0, 6000], [6000, 0, 6000, 0], [0, 6000, 6000, 0]):
        mx.attention(q, k, v, cu_q=cu_q, cu_k=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert mx.device_status() == 1
    cu_k = _edges(torch, [2000, 2500, 1500])
    first = mx.attention(q, k, v, cu_q=cu_q, cu_k=cu_k)
    assert all(torch.equal(x, y) for x, y in zip(first, mx.attention(q, k, v, cu_q=cu_q, cu_k=cu_k)))
    assert mx.device_status() == 0


def test_streams_and_graphs():
    """Two calls at once on two streams, and a captured pass replayed on new numbers beside an eager one, give what calls one
    by one give."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    lens = [700, 1, 333]
    sets = [_inputs(torch, lens, lens, 8, 2, 128, 0, s) for s in (8, 9)]
    few = [_inputs(torch, [2], [5000], 8, 2, 128, 0, s) for s in (8, 9)]
    cu = _edges(torch, lens)
    rope = mx.Rope([0.5 ** i for i in range(64)])
    pos = torch.arange(sum(lens), device="cuda")
    gain = torch.rand(128, device="cuda")

    def run(x, y):
        q, k, v, do = x
        a, b = mx.qk_norm_rope(q, k, rope, pos, gain, gain)
        res = _all(torch, a, b, v, do, cu)
        back = mx.qk_norm_rope_grad(q, k, res[3], res[4], rope, pos, gain, gain)
        return [a, b, *res, *back, *mx.attention(*y[:3])]

    want = [run(x, y) for x, y in zip(sets, few)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(5):
        for s, x, y in zip(streams, sets, few):
            with torch.cuda.stream(s):
                got.append(run(x, y))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(want[i % 2], g))
    # a stream given to the call
    out, lse = mx.attention(*few[0][:3], stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(out, want[0][-2]) and torch.equal(lse, want[0][-1])
    place = [x.clone() for x in sets[0]], [x.clone() for x in few[0]]
    graphs, results = [], []
    for _ in range(2):  # two graphs of the same call
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(run(*place))
        graphs.append(graph)
    for i in (1, 0, 1):
        for to, x in zip(place[0] + place[1], sets[i] + few[i]):
            to.copy_(x)
        for graph, res in zip(graphs, results):
            graph.replay()
            eager = run(sets[i], few[i])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(res, want[i]))
            assert all(torch.equal(a, b) for a, b in zip(eager, want[i]))
    assert mx.device_status() == 0


def test_in_place_and_one_side():
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    for dtype, D, inter in ((torch.bfloat16, 128, False), (torch.float32, 66, True), (torch.bfloat16, 24, False)):
        q, k = torch.randn(300, 6, D, device="cuda").to(dtype), torch.randn(300, 2, D, device="cuda").to(dtype)
        dq, dk = torch.randn_like(q), torch.randn_like(k)
        rope = mx.Rope([0.9 ** i for i in range(D // 2)], interleaved=inter)
        pos = torch.arange(300, device="cuda", dtype=torch.int32)
        g = torch.rand(D, device="cuda")
        want = mx.qk_norm_rope(q, k, rope, pos, g, None)
        a, b = q.clone(), k.clone()
        got = mx.qk_norm_rope(a, b, rope, pos, g, None, q_out=a, k_out=b)
        assert got[0] is a and torch.equal(a, want[0]) and torch.equal(b, want[1])
        alone, none = mx.qk_norm_rope(q, None, rope, pos, g)
        assert none is None and torch.equal(alone, want[0])
        want = mx.qk_norm_rope_grad(q, None, dq, dk, rope, pos, g, None)
        a, b = dq.clone(), dk.clone()
        got = mx.qk_norm_rope_grad(q, None, a, b, rope, pos, g, None, dq_in=a, dk_in=b)
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(got[2], want[2]) and got[3] is None
        a = q.clone()  # over the forward pass's input
        mx.qk_norm_rope_grad(a, None, dq, None, rope, pos, g, dq_in=a, gains=False)
        assert torch.equal(a, want[0])


def test_angles_far_away():
    """Positions to 2^31 and beyond 2^40 turn by the exact angle, in both integer types."""
    torch = gpu_ready()
    from fractions import Fraction

    from mxfp4_precision_gemms_gb300 import binding as mx

    freq = [1.0, 0.1, 3.7e-3, 1e-6, -0.25, 1234.5]
    pos = [0, 1, -1, 8191, 1_000_003, 2**31 - 1, -(2**31)] + [2**33 + 5, 10**12]
    q = torch.zeros(len(pos), 1, 12, device="cuda")
    q[..., 0::2] = 1.0
    rope = mx.Rope(freq, interleaved=True)
    got = mx.qk_norm_rope(q, None, rope, torch.tensor(pos, device="cuda"))[0].cpu().double()
    # pi to 60 digits
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10**60)
    for i, t in enumerate(pos):
        for j, f in enumerate(freq):
            turns = Fraction(f) * t / (2 * pi)
            a = float(turns - round(turns)) * 2 * math.pi
            # the frequency's own place in 64-bit fixed point, the angle in fp32, two units of a cosine
            tol = abs(t) * 2.0 ** -64 * 2 * math.pi + 2.0 ** -24 * math.pi + 4 * 2.0 ** -24
            assert abs(got[i, 0, 2 * j].item() - math.cos(a)) <= tol, (t, f)
            assert abs(got[i, 0, 2 * j + 1].item() - math.sin(a)) <= tol, (t, f)
    p32 = torch.tensor(pos[:7], device="cuda", dtype=torch.int32)
    assert torch.equal(mx.qk_norm_rope(q[:7], None, rope, p32)[0].cpu().double(), got[:7])


def test_each_tensor_of_a_call_is_looked_at(monkeypatch):
    """A tensor on the host or of another type or shape among the others is refused, whichever it is, and so are all on
    another device than the current one (here: another index is made out to be the current one)."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import attention as att
    from mxfp4_precision_gemms_gb300 import binding as mx

    q, k, v, do = _inputs(torch, [40], [40], 4, 2, 64, 0, 10)
    cu = _edges(torch, [40])
    out, lse, rest = mx.attention(q, k, v, rest=True)
    rope = mx.Rope([1.0] * 32)
    pos, g = torch.arange(40, device="cuda"), torch.ones(64, device="cuda")
    calls = [(lambda q, k, v, cu: mx.attention(q, k, v, cu_q=cu), (q, k, v, cu)),
             (lambda *a: mx.attention_grad(*a[:6], cu_q=a[6], rest=a[7]), (q, k, v, out, lse, do, cu, rest)),
             (lambda q, k, pos, g: mx.qk_norm_rope(q, k, rope, pos, g, g), (q, k, pos, g)),
             (lambda q, k, dq, dk, pos, g: mx.qk_norm_rope_grad(q, k, dq, dk, rope, pos, g, g), (q, k, do, k, pos, g)),
             (lambda q, k, v, cu: att.attention(q, k, v, cu_q=cu), (q, k, v, cu)),
             (lambda q, k, pos, g: att.qk_norm_rope(q, k, rope, pos, g, g), (q, k, pos, g))]
    for call, args in calls:
        call(*args)
        for i, x in enumerate(args):
            for bad in (x.cpu(), x.double() if x.is_floating_point() else x.short(), x[:-1]):
                if x.dim() == 1 and x is cu and bad.shape != x.shape:
                    continue  # another list
                if call in (calls[5][0],) and x is g and bad.dtype == torch.float64:
                    continue  # the autograd form converts gains
                with pytest.raises((ValueError, RuntimeError)):
                    call(*(bad if j == i else y for j, y in enumerate(args)))
    for call in (lambda: mx.attention(q, k, v, out=out.cpu()), lambda: mx.attention(q, k, v, out=out[:, :2]),
                 lambda: mx.attention(q, k, v, lse=lse.t()), lambda: mx.attention_grad(q, k, v, out, lse, do, dk=q),
                 lambda: mx.attention(q, k, v, seqs=3), lambda: mx.attention(q, k, v, scale=-1.0),
                 lambda: mx.attention(q, k, v, cu_k=cu), lambda: mx.attention(q[:30], k, v, cu_q=cu),
                 lambda: mx.attention(q.transpose(1, 2), k, v), lambda: mx.attention(q[..., :60], k[..., :60], v[..., :60]),
                 lambda: mx.qk_norm_rope(q, k, rope), lambda: mx.qk_norm_rope(q, k, rope, pos[None].expand(2, 40)),
                 lambda: mx.qk_norm_rope_grad(q, k, do, None, rope, pos, g, g)):
        with pytest.raises((ValueError, mx.Mxfp4Error)):
            call()
    torch.cuda.synchronize()
    monkeypatch.setattr(mx, "_current_device", lambda: 1)
    for call, args in calls:
        with pytest.raises(ValueError, match="current CUDA device"):
            call(*args)


# ------------------------------------------------------------------ autograd
def _plain_block(torch, q, k, v, q_gain, k_gain, positions, freq, eps, causal):
    """Norm, rotation and attention of one sequence with elementary operations in 64 bits."""
    angle = positions[:, None].double() * torch.tensor(freq, device="cuda", dtype=torch.float64)

    def turned(x, gain):
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain
        a, b = x.chunk(2, -1)
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q, k = turned(q, q_gain), turned(k, k_gain)
    group = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    z = torch.einsum("ihd,jhd->hij", q, k) * q.shape[-1] ** -0.5
    if causal:
        z = z.masked_fill(torch.ones_like(z[0], dtype=torch.bool).triu(1), -math.inf)
    return torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), v)


@pytest.mark.parametrize("batched", [True, False])
def test_norm_rotation_and_attention_together(batched):
    """The autograd forms behind one projection's output, over a batch and over packed sequences, against torch's autograd
    in 64 bits.  q and k are rounded to bf16 after the rotation (2^-8 of each element, which scores of size up to some four
    feel), p and dz once, each result once: 2^-5 in all, in the 2-norm."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx
    from mxfp4_precision_gemms_gb300.attention import Rope, attention, qk_norm_rope

    g = torch.Generator(device="cuda").manual_seed(0)
    a, b, D, lens = 6, 2, 64, ([150, 150, 150] if batched else [150, 31, 200])
    T = sum(lens)
    qkv = torch.randn(T, (a + 2 * b) * D, device="cuda", generator=g).bfloat16().requires_grad_()
    gains = [(1 + 0.2 * torch.randn(D, device="cuda", generator=g)).requires_grad_() for _ in range(2)]
    weight = torch.randn(T, a, D, device="cuda", generator=g)
    freq = [100.0 ** (-i / 32) for i in range(32)]
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    lead = (3, 150) if batched else (T,)
    q, k, v = qkv.view(*lead, a + 2 * b, D).split([a, b, b], -2)
    q, k = qk_norm_rope(q, k, Rope(freq), pos.view(lead), *gains, eps=1e-5)
    out = attention(q, k, v) if batched else attention(q, k, v, cu_q=_edges(torch, lens))
    assert out.shape == (*lead, a, D)
    (out.reshape(T, a, D).float() * weight).sum().backward()
    assert mx.device_status() == 0

    x64 = qkv.detach().double().requires_grad_()
    g64 = [x.detach().double().requires_grad_() for x in gains]
    want = []
    at = 0
    for n in lens:
        q, k, v = x64[at:at + n].view(n, a + 2 * b, D).split([a, b, b], 1)
        want.append(_plain_block(torch, q, k, v, *g64, pos[at:at + n], freq, 1e-5, True))
        at += n
    want = torch.cat(want)
    (want * weight).sum().backward()
    rel = lambda x, y: float((x.double() - y).norm() / y.norm())
    assert rel(out.detach().reshape(T, a, D), want.detach()) < 2.0 ** -5
    assert rel(qkv.grad, x64.grad) < 2.0 ** -5
    assert all(x.grad.dtype == torch.float32 and rel(x.grad, y.grad) < 2.0 ** -5 for x, y in zip(gains, g64))


def test_gradients_against_differences():
    """Of the rotation in fp32 against differences of itself; of attention against differences of the formula in 64 bits."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx
    from tests.attention_reference import attend

    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    q, k, gq, gk = rand(9, 3, 24), rand(9, 1, 24), 1 + 0.2 * rand(24), 1 + 0.2 * rand(24)
    wq, wk = rand(9, 3, 24), rand(9, 1, 24)
    rope, pos = mx.Rope([0.3 ** i for i in range(8)]), torch.arange(9, device="cuda") * 1000

    def f(q, k, gq, gk):
        a, b = mx.qk_norm_rope(q, k, rope, pos, gq, gk)
        return ((a.double() * wq).sum() + (b.double() * wk).sum()).item()

    grads = mx.qk_norm_rope_grad(q, k, wq, wk, rope, pos, gq, gk)
    for i in range(4):
        args, d, h = [q, k, gq, gk], rand(*(q, k, gq, gk)[i].shape), 2.0 ** -7
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - h * d, args[i] + h * d
        diff = (f(*hi) - f(*lo)) / (2 * h)
        want = (grads[i].double() * d).sum().item()
        # h^2 of the third derivative (some tens times the size here), and fp32 results' noise over 2 h
        size = float((grads[i].abs() * d.abs()).sum())
        assert abs(diff - want) < 30 * h * h * size + 2.0 ** -22 * 300 / h, (i, diff, want)

    q, k, v, do = _inputs(torch, [7], [9], 2, 1, 16, 0, 11)
    out, lse, rest = mx.attention(q, k, v, rest=True)
    grads = mx.attention_grad(q, k, v, out, lse, do, rest=rest)
    _, tol = attend(q, k, v, [7], [9], True, 0.25, do)
    for i, name in enumerate(("dq", "dk", "dv")):
        d = rand(*(q, k, v)[i].shape).double()

        def along(h):
            x = [y.double() for y in (q, k, v)]
            x[i] = x[i] + h * d
            return (attend(*x, [7], [9], True, 0.25)[0]["out"] * do.double()).sum().item()

        h = 1e-4
        diff = (along(h) - along(-h)) / (2 * h)
        assert abs(diff - (grads[i].double() * d).sum().item()) <= float((tol[name] * d.abs()).sum()) + 1e-5, name


def test_autograd_takes_any_layout():
    """Transposed tensors and broadcast gradients give what contiguous ones give; misaligned ones too, but for the order in
    which a row's squares are added (fp32, 2^-18 of the sum of 64), which now and then rounds an element of q or k to
    the neighbouring bf16 number (2^-7 of it) and so moves results by less than that in the 2-norm."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.attention import Rope, attention, qk_norm_rope

    q, k, v, _ = _inputs(torch, [60], [60], 4, 4, 64, 0, 12)
    rope, pos = Rope([0.7 ** i for i in range(32)]), torch.arange(60, device="cuda")
    gain = torch.rand(64, device="cuda").bfloat16().requires_grad_()

    def run(lay, grad):
        leaves = [lay(x).detach().requires_grad_() for x in (q, k, v)]
        gain.grad = None
        a, b = qk_norm_rope(leaves[0], leaves[1], rope, pos, gain, gain)
        y = attention(a, b, leaves[2])
        y.backward(grad)
        return [y, *(x.grad for x in leaves), gain.grad]

    ones = torch.ones(1, device="cuda").bfloat16().expand(60, 4, 64)  # a sum's gradient
    want = run(lambda x: x, ones.contiguous())
    for lay in (lambda x: x.transpose(0, 1).contiguous().transpose(0, 1), lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)):
        assert all(torch.equal(a, b) for a, b in zip(want, run(lay, ones)))
    odd = lambda x: torch.cat([x.reshape(-1)[:1], x.reshape(-1)])[1:].view(60, 4, 64)
    assert odd(q).data_ptr() % 4 == 2
    for a, b in zip(want, run(odd, ones)):
        assert (a.detach().double() - b.detach().double()).norm().item() < 2.0 ** -7 * a.detach().double().norm().item()
    # one key head broadcast over all: its gradient is the sum
    one = k[:, :1].detach().requires_grad_()
    y = attention(q, one.expand(60, 4, 64), v)
    y.sum().backward()
    assert one.grad.shape == (60, 1, 64) and torch.isfinite(one.grad.float()).all()


def test_only_what_is_asked_for():
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.attention import attention, qk_norm_rope

    q, k, v, _ = _inputs(torch, [20], [20], 2, 2, 64, 0, 13)
    vg = v.clone().requires_grad_()
    attention(q, k, vg).sum().backward()
    assert vg.grad is not None
    qg = q.clone().requires_grad_()
    a, b = qk_norm_rope(qg, k)
    a.sum().backward()  # nothing comes back through b
    assert torch.equal(qg.grad, torch.ones_like(q))
    with torch.no_grad():
        assert not attention(q, k, v).requires_grad


@pytest.mark.parametrize("heads", [2, 4])
def test_the_example_with_attention(heads):
    """A language model with attention in its blocks trains, and every weight gets a gradient."""
    import importlib.util
    import os

    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tiny_lm.py")
    spec = importlib.util.spec_from_file_location("tiny_lm", path)
    lm = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(lm)
    losses = lm.train(steps=4, tokens=1024, vocab=500, dim=128, say=lambda *_: None, heads=heads)
    assert mx.device_status() == 0 and all(math.isfinite(x) for x in losses)
    g = torch.Generator().manual_seed(0)
    p = lm.make_model(500, 128, g, heads)
    ids, targets = lm.batch(torch.randint(0, 500, (500, 4), generator=g), 512, g)
    lm.loss_of(p, ids, targets, heads).backward()
    assert all(w.grad is not None and torch.isfinite(w.grad).all() and w.grad.any() for w in p.values())
