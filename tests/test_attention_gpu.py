"""Attention over packed sequences and its gradient against 64 bits: lengths from nothing to several tiles, head sizes and
groups, masks that leave rows empty, strides, and what may not reach a sequence."""
import itertools

import pytest

from tests.gpu_util import gpu_ready

pytestmark = pytest.mark.gpu

LENGTHS = [
    ([1], [1]), ([3], [37]), ([128], [128]), ([129], [129]), ([300], [300]), ([257, 1, 0, 130], [257, 1, 0, 130]),
    ([5, 200, 0, 64], [300, 7, 9, 0]),  # more keys than queries, fewer, none of one, none of the other
]


def _inputs(torch, q_lens, k_lens, a, b, D, spare, seed, lean=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    Tq, Tk = sum(q_lens) + spare, sum(k_lens) + spare
    q, k, v, do = rand(Tq, a, D), rand(Tk, b, D), rand(Tk, b, D), rand(Tq, a, D)
    if Tk and lean:  # some rows point firmly at one key
        pick = torch.randint(0, Tk, (Tq, 1), device="cuda", generator=g)
        head = torch.arange(a, device="cuda") // (a // b)
        q = q + lean * torch.rand(Tq, a, 1, device="cuda", generator=g) ** 2 * k[pick, head]
    return [x.bfloat16() for x in (q, k, v, do)]


def _edges(torch, lens):
    return torch.tensor([0, *itertools.accumulate(lens)], dtype=torch.int32, device="cuda")


def _check(torch, q, k, v, do, q_lens, k_lens, causal, scale=None, listed=True, kept=True):
    from mxfp4_precision_gemms_gb300 import binding as mx
    from tests.attention_reference import assert_close, attend

    kw = dict(causal=causal, scale=scale)
    if listed:
        kw |= dict(cu_q=_edges(torch, q_lens), cu_k=_edges(torch, k_lens))
    else:
        kw |= dict(seqs=len(q_lens))
    out, lse, rest = mx.attention(q, k, v, **kw, rest=True)
    grads = mx.attention_grad(q, k, v, out, lse, do, **kw, rest=rest if kept else None)
    assert mx.device_status() == 0
    want, tol = attend(q, k, v, q_lens, k_lens, causal, scale or q.shape[2] ** -0.5, do, kept)
    assert_close(out.double() + rest.double(), want["out"], tol["whole"], "out + rest")
    for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        assert_close(got, want[name], tol[name], name)
    return (out, lse, *grads)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_lengths(lens, D, causal):
    torch = gpu_ready()
    q_lens, k_lens = lens
    q, k, v, do = _inputs(torch, q_lens, k_lens, 4, 2, D, 3, 1)
    _check(torch, q, k, v, do, q_lens, k_lens, causal)


def test_gradients_without_the_rest_of_the_output():
    torch = gpu_ready()
    q, k, v, do = _inputs(torch, [300], [300], 4, 2, 128, 0, 6, lean=2.0)
    _check(torch, q, k, v, do, [300], [300], True, kept=False)


@pytest.mark.parametrize("D", [8, 16, 24, 40, 72, 80, 96, 120])
def test_head_sizes(D):
    torch = gpu_ready()
    q, k, v, do = _inputs(torch, [150], [210], 2, 1, D, 0, 2)
    _check(torch, q, k, v, do, [150], [210], True)


@pytest.mark.parametrize("heads", [(1, 1), (7, 1), (6, 3), (5, 5), (12, 2)])
def test_shared_heads(heads):
    torch = gpu_ready()
    q, k, v, do = _inputs(torch, [70, 140], [70, 140], *heads, 64, 0, 3)
    _check(torch, q, k, v, do, [70, 140], [70, 140], True)


@pytest.mark.parametrize("causal", [True, False])
def test_several_tiles(causal):
    """More tiles of queries and keys than any ring has stages."""
    torch = gpu_ready()
    for D in (64, 128):
        q, k, v, do = _inputs(torch, [1400, 700], [1400, 1300], 2, 1, D, 0, 4, lean=2.0)
        _check(torch, q, k, v, do, [1400, 700], [1400, 1300], causal)


def test_equal_lengths_without_a_list():
    torch = gpu_ready()
    q, k, v, do = _inputs(torch, [190] * 3, [260] * 3, 4, 4, 80, 0, 5)
    a = _check(torch, q, k, v, do, [190] * 3, [260] * 3, True, listed=False)
    b = _check(torch, q, k, v, do, [190] * 3, [260] * 3, True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(8, 2), (3, 3), (7, 1)])
def test_few_queries_over_many_keys(heads, causal):
    """Keys shared out over several CTAs, in as many parts for the shortest sequence as for the longest."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    q_lens, k_lens = [1, 1, 0, 5, 1, 2], [2000, 700, 900, 3000, 90, 0]
    for D in (64, 72, 128):
        assert mx.lib().mxfp4_attention_workspace_bytes(sum(q_lens), sum(k_lens), D, *heads, len(q_lens)) > 0
        q, k, v, do = _inputs(torch, q_lens, k_lens, *heads, D, 3, 7, lean=2.0)
        _check(torch, q, k, v, do, q_lens, k_lens, causal)


@pytest.mark.parametrize("lens", [([200], [3000]), ([30, 70], [4000, 2500]), ([300, 1], [90, 5000])], ids=str)
@pytest.mark.parametrize("heads", [(8, 2), (3, 3)])
def test_many_rows_joined(heads, lens):
    """Parts of pairs of query tiles whose rows are more than the warps of one part's CTAs that join them."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    assert mx.lib().mxfp4_attention_workspace_bytes(sum(lens[0]) + 2, sum(lens[1]) + 2, 128, *heads, len(lens[0])) > 0
    q, k, v, do = _inputs(torch, *lens, *heads, 128, 2, 10, lean=2.0)
    _check(torch, q, k, v, do, *lens, True)


@pytest.mark.parametrize("heads", [(65, 1), (130, 1), (26, 2), (96, 1), (254, 2)])
def test_groups_that_fill_no_tile(heads):
    torch = gpu_ready()
    q, k, v, do = _inputs(torch, [3, 40], [50, 160], *heads, 32, 0, 8)
    _check(torch, q, k, v, do, [3, 40], [50, 160], True)


def test_the_same_bits_on_every_run():
    """Hundreds of short calls one behind the other, in which the warps of a block overtake each other in every way that
    their barriers allow: no wait runs out, and every call gives what the first gave."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    for D, lens in ((128, [288, 400, 1100]), (64, [290, 129, 520])):
        q, k, v, do = _inputs(torch, lens, lens, 32, 8, D, 0, 9)
        cu = _edges(torch, lens)
        first = None
        for _ in range(300):
            out, lse, rest = mx.attention(q, k, v, cu_q=cu, rest=True)
            got = (out, lse, rest, *mx.attention_grad(q, k, v, out, lse, do, cu_q=cu, rest=rest))
            if first is None:
                first = got
            else:
                assert all(torch.equal(x, y) for x, y in zip(got, first))
        assert mx.device_status() == 0
