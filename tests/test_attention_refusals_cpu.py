"""Refusals of rotation and attention that need no GPU: every argument is checked on the host before the device is
touched."""
import ctypes

import pytest

import __graft_entry__
from mxfp4_precision_gemms_gb300 import binding as mx

P = ctypes.c_void_p
INVALID, SHAPE, MISALIGNED, WORKSPACE = 1, 2, 3, 4
PASSED = 5  # with no GPU a call that gets past its checks fails at the first CUDA call


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return mx.lib()


def _table(*heads):
    """(data, token stride, head stride, heads, dtype) each, None for NULL."""
    import array

    table = array.array("q", [x for h in heads for x in ((0, 0, 0, 0) if h is None else (*h[:3], h[3] | h[4] << 32))])
    at = table.buffer_info()[0]
    return table, [None if h is None else P(at + 32 * i) for i, h in enumerate(heads)]


BF16_Q, BF16_K = (0x10000, 1536, 128, 8, 1), (0x10800, 1536, 128, 2, 1)


def _rope(L, **kw):
    a = dict(q=BF16_Q, k=BF16_K, n=4, dim=128, qg=0x2000, kg=None, eps=1e-6, freq=(1.0, 0.5), axis=None, pairs=None, inter=0,
             rope=True, pos=0x3000, it=1, axes=1, qo=(0x40000, 1024, 128, 8, 1), ko=(0x50000, 256, 128, 2, 1))
    a.update(kw)
    freq = (ctypes.c_double * max(1, len(a["freq"])))(*a["freq"])
    axis = None if a["axis"] is None else (ctypes.c_int32 * len(a["axis"]))(*a["axis"])
    c = mx.RopeC(ctypes.addressof(freq) if a["freq"] else None, None if axis is None else ctypes.addressof(axis),
                 len(a["freq"]) if a["pairs"] is None else a["pairs"], a["inter"])
    table, (q, k, qo, ko) = _table(a["q"], a["k"], a["qo"], a["ko"])
    return L.mxfp4_qk_norm_rope(q, k, a["n"], a["dim"], P(a["qg"]), P(a["kg"]), a["eps"],
                                ctypes.byref(c) if a["rope"] else None, P(a["pos"]), a["it"], a["axes"], qo, ko, None)


ROPE = [
    (dict(n=-1), INVALID), (dict(dim=-2), INVALID), (dict(dim=127), SHAPE), (dict(dim=258), SHAPE), (dict(dim=0), SHAPE),
    (dict(n=1 << 31), SHAPE), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(it=2), INVALID),
    (dict(pairs=65, freq=(1.0,) * 65), SHAPE), (dict(pairs=-1), SHAPE), (dict(inter=2), INVALID), (dict(axes=0), INVALID),
    (dict(axes=256), INVALID), (dict(freq=(float("inf"),)), INVALID), (dict(freq=(2e6,)), INVALID),
    (dict(axis=(0, 1)), INVALID), (dict(axis=(-1, 0)), INVALID), (dict(pos=None), INVALID), (dict(pos=0x3004), MISALIGNED),
    (dict(qg=0x2002), MISALIGNED), (dict(q=None), INVALID), (dict(q=(0, 1536, 128, 8, 1)), INVALID),
    (dict(q=(0x10001, 1536, 128, 8, 1)), MISALIGNED), (dict(q=(0x10000, 1536, 128, 8, 2)), INVALID),
    (dict(q=(0x10000, 100, 128, 8, 1)), INVALID), (dict(q=(0x10000, 1536, 100, 8, 1)), INVALID),
    (dict(q=(0x10000, -1536, 128, 8, 1)), INVALID), (dict(q=(0x10000, 1536, 128, 0, 1)), SHAPE),
    (dict(q=(0x10000, 1 << 39, 128, 8, 1)), INVALID), (dict(k=(0x10800, 1536, 128, 2, 0)), INVALID),
    (dict(qo=(0x40000, 1024, 128, 7, 1)), INVALID), (dict(qo=(0x40000, 1024, 128, 8, 0)), INVALID), (dict(qo=None), INVALID),
    (dict(ko=None), INVALID), (dict(qo=(0x40000, 512, 128, 8, 1)), INVALID),  # rows that overlap
    (dict(n=0), 0), (dict(n=0, q=(0, 0, 128, 8, 1), pos=None), 0)]


@pytest.mark.parametrize("change,want", ROPE)
def test_rotation_refuses(L, change, want):
    assert _rope(L, **change) == want
    assert (L.mxfp4_last_error() == b"") == (want == 0)


@pytest.mark.parametrize("change", [{}, dict(k=None, ko=None), dict(rope=False, pos=None), dict(axis=(2, 0), axes=3),
                                    dict(q=(0x10002, 1537, 129, 8, 1)), dict(qo=(0x40000, 128, 512, 8, 1)),
                                    dict(qo=BF16_Q, ko=BF16_K)])
def test_rotation_takes(L, change):
    import torch

    if torch.cuda.is_available():
        pytest.skip("pointers of this test are not device memory")
    assert _rope(L, **change) == PASSED


def _rope_grad(L, **kw):
    a = dict(q=BF16_Q, k=BF16_K, dq=(0x60000, 1024, 128, 8, 1), dk=(0x70000, 256, 128, 2, 1), n=4, dim=128, qg=0x2000, kg=None,
             rope=False, dqi=(0x40000, 1024, 128, 8, 1), dki=(0x50000, 256, 128, 2, 1), dqg=0x2400, dkg=None, ws=0x100000,
             wsb=None)
    a.update(kw)
    table, (q, k, dq, dk, dqi, dki) = _table(*(a[x] for x in ("q", "k", "dq", "dk", "dqi", "dki")))
    need = L.mxfp4_qk_norm_rope_grad_workspace_bytes(a["n"], a["dim"]) if a["wsb"] is None else a["wsb"]
    return L.mxfp4_qk_norm_rope_grad(q, k, dq, dk, a["n"], a["dim"], P(a["qg"]), P(a["kg"]), 1e-6, None, None, 0, 0, dqi, dki,
                                     P(a["dqg"]), P(a["dkg"]), P(a["ws"]), need, None)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), INVALID), (dict(dq=None), INVALID), (dict(dqi=None), INVALID), (dict(dki=None), INVALID),
    (dict(dkg=0x2800), INVALID),  # of a gain that is not there
    (dict(dk=None, kg=0x2800), PASSED), (dict(q=(0x10000, 1536, 128, 4, 1)), INVALID),
    (dict(dk=(0x70000, 256, 128, 2, 0)), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=64), WORKSPACE),
    (dict(ws=0x100010), MISALIGNED), (dict(dqg=0x2402), MISALIGNED), (dict(n=0, dqg=None), 0)])
def test_rotation_gradient_refuses(L, change, want):
    import torch

    if want == PASSED and torch.cuda.is_available():
        pytest.skip("pointers of this test are not device memory")
    assert _rope_grad(L, **change) == want


def _attention(L, grad=False, **kw):
    a = dict(q=(0x10000, 1536, 128, 8, 1), k=(0x20000, 1536, 128, 2, 1), v=(0x30000, 1536, 128, 2, 1), n=6, m=9, dim=128,
             cq=0x1000, ck=0x2000, seqs=2, causal=1, scale=0.1, zero=0, out=(0x40000, 1024, 128, 8, 1), rest=None, lse=0x5000,
             dout=(0x60000, 1024, 128, 8, 1), dq=(0x70000, 1024, 128, 8, 1), dk=(0x80000, 256, 128, 2, 1),
             dv=(0x90000, 256, 128, 2, 1), ws=0x100000, wsb=1 << 40)
    a.update(kw)
    table, (q, k, v, out, rest, dout, dq, dk, dv) = _table(*(a[x] for x in ("q", "k", "v", "out", "rest", "dout", "dq", "dk",
                                                                           "dv")))
    tail = (a["n"], a["m"], a["dim"], P(a["cq"]), P(a["ck"]), a["seqs"], a["causal"], a["scale"], a["zero"])
    if grad:
        return L.mxfp4_attention_grad(q, k, v, out, rest, P(a["lse"]), dout, *tail, dq, dk, dv, P(a["ws"]), a["wsb"], None)
    return L.mxfp4_attention(q, k, v, *tail, out, rest, P(a["lse"]), P(a["ws"]), a["wsb"], None)


ATTENTION = [
    (dict(n=-1), INVALID), (dict(m=-1), INVALID), (dict(seqs=-1), INVALID), (dict(n=1 << 30), SHAPE), (dict(m=1 << 30), SHAPE),
    (dict(seqs=1 << 24), SHAPE), (dict(dim=4), SHAPE), (dict(dim=136), SHAPE), (dict(dim=100), SHAPE),
    (dict(causal=2), INVALID), (dict(zero=2), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=3e38), INVALID), (dict(q=None), INVALID), (dict(v=None), INVALID),
    (dict(q=(0x10000, 1536, 128, 8, 0)), INVALID), (dict(k=(0x20000, 1536, 128, 3, 1)), SHAPE),
    (dict(v=(0x30000, 1536, 128, 1, 1)), SHAPE), (dict(q=(0x10008, 1536, 128, 8, 1)), MISALIGNED),
    (dict(q=(0x10000, 1540, 128, 8, 1)), MISALIGNED), (dict(k=(0x20000, 1536, 132, 2, 1)), MISALIGNED),
    (dict(cq=None), INVALID), (dict(ck=None), INVALID), (dict(cq=0x1002), MISALIGNED), (dict(cq=None, ck=None, seqs=4), SHAPE),
    (dict(cq=None, ck=None, seqs=0), SHAPE), (dict(out=None), INVALID), (dict(out=(0x40000, 1024, 128, 4, 1)), INVALID),
    (dict(rest=(0x40000, 1024, 128, 4, 1)), INVALID), (dict(lse=None), INVALID),
    (dict(lse=0x5002), MISALIGNED), (dict(seqs=0), 0)]


@pytest.mark.parametrize("change,want", ATTENTION + [(dict(n=0), 0), (dict(out=(0x40000, 512, 128, 8, 1)), INVALID),  # rows that overlap
                                                     (dict(m=4000, n=2, ws=None), WORKSPACE),
                                                     (dict(m=4000, n=2, wsb=100), WORKSPACE),
                                                     (dict(m=4000, n=2, ws=0x100010), MISALIGNED)])
def test_attention_refuses(L, change, want):
    assert _attention(L, **change) == want
    assert (L.mxfp4_last_error() == b"") == (want == 0)


@pytest.mark.parametrize("change,want", ATTENTION + [
    (dict(dout=None), INVALID), (dict(dout=(0x60000, 1024, 128, 4, 1)), INVALID), (dict(dq=(0x70000, 1024, 128, 4, 1)), INVALID),
    (dict(dk=(0x80000, 256, 128, 1, 1)), INVALID), (dict(dv=(0x90000, 128, 128, 2, 1)), INVALID), (dict(ws=None), WORKSPACE),
    (dict(wsb=64), WORKSPACE), (dict(ws=0x100010), MISALIGNED), (dict(n=0, m=0, lse=None, ws=None), 0)])
def test_attention_gradient_refuses(L, change, want):
    assert _attention(L, grad=True, **change) == want


def test_workspaces(L):
    w = L.mxfp4_attention_workspace_bytes
    assert w(8192, 8192, 128, 32, 8, 1) == 0          # queries enough for all SMs
    assert w(1, 500, 128, 32, 8, 1) == 0              # too few keys to share out
    assert w(8, 24000, 128, 32, 8, 4) > 0
    # whatever the lists say, a part needs 256 rows of a head's size and four numbers
    assert w(8, 24000, 128, 32, 8, 4) % (256 * (128 * 4 + 16)) == 0
    assert w(8, 24000, 128, 32, 8, 4) < 256 << 20
    for bad in ((-1, 8, 128, 8, 8, 1), (8, 0, 128, 8, 8, 1), (8, 24000, 0, 8, 8, 1), (8, 24000, 128, 8, 3, 1),
                (8, 24000, 128, 8, 8, 0), (8, 24000, 128, 0, 8, 1)):
        assert w(*bad) == 0
    assert L.mxfp4_attention_grad_workspace_bytes(100, 8) == 6400 and L.mxfp4_attention_grad_workspace_bytes(0, 8) == 0
    assert L.mxfp4_qk_norm_rope_grad_workspace_bytes(0, 128) == 0 and L.mxfp4_qk_norm_rope_grad_workspace_bytes(9, 127) == 0
    assert L.mxfp4_qk_norm_rope_grad_workspace_bytes(9, 128) == 1024 * 2 * 128 * 4


def test_binding_refuses_before_the_library():
    import torch

    from mxfp4_precision_gemms_gb300 import attention as att

    q, k = torch.zeros(3, 4, 8).bfloat16(), torch.zeros(3, 2, 8).bfloat16()
    lse = torch.zeros(4, 3)
    rope = mx.Rope([1.0], axis=[0])
    pos = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: mx.attention(q, k, k), lambda: mx.attention_grad(q, k, k, q, lse, q),
                 lambda: mx.qk_norm_rope(q, k, rope, pos), lambda: mx.qk_norm_rope_grad(q, k, q, k, rope, pos),
                 lambda: att.attention(q, k, k), lambda: att.attention(q[None], k, k), lambda: att.attention(q[0], k[0], k[0]),
                 lambda: att.attention(q[None], k[None].expand(2, 3, 2, 8), k[None]),
                 lambda: att.attention(q[None], k[None], k[None], cu_q=pos.int()),
                 lambda: att.qk_norm_rope(q, k[:2], rope, pos), lambda: att.qk_norm_rope(q, k, rope),
                 lambda: att.qk_norm_rope(q, k, rope, pos[:2]), lambda: att.qk_norm_rope(q, k, mx.Rope([1.0], [1]), pos),
                 lambda: mx.Rope([1.0, 2.0], axis=[0])):
        with pytest.raises(ValueError):
            call()
