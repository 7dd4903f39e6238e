"""What masked places may hold, and what the queries that they leave with nothing get."""
import math

import pytest

from tests.gpu_util import gpu_ready
from tests.test_attention_gpu import _edges, _inputs

pytestmark = pytest.mark.gpu


def _all(torch, q, k, v, do, **kw):
    from mxfp4_precision_gemms_gb300 import binding as mx

    out, lse, rest = mx.attention(q, k, v, rest=True, **kw)
    return dict(zip(("out", "lse", "rest", "dq", "dk", "dv"),
                    (out, lse.t(), rest, *mx.attention_grad(q, k, v, out, lse, do, rest=rest, **kw))))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lens", [([300], [180]), ([4, 2], [2, 5000]), ([40, 9], [3, 700])], ids=str)
@pytest.mark.parametrize("heads", [(2, 1), (7, 1)])
def test_queries_that_see_no_key(heads, lens, value):
    """They get zeros, an lse of -infinity and no gradient, whatever the keys that others of their tile see hold."""
    torch = gpu_ready()
    for D in (64, 72, 128):
        q, k, v, do = _inputs(torch, *lens, *heads, D, 0, 1)
        for x in (k, v):
            x[: lens[1][0]] = value  # of the first sequence, with more queries than keys
        got = _all(torch, q, k, v, do, cu_q=_edges(torch, lens[0]), cu_k=_edges(torch, lens[1]))
        none = lens[0][0] - lens[1][0]
        for name in ("out", "rest", "dq"):
            assert not got[name][:none].any(), name
        assert (got["lse"][:none] == -math.inf).all()


@pytest.mark.parametrize("lens", [([150], [150]), ([3], [4000])], ids=str)
def test_scores_that_are_infinite(lens):
    """A query whose scores are all -infinity gets what one that sees no key gets; one of +infinity or NaN makes it NaN."""
    torch = gpu_ready()
    q, k, v, do = _inputs(torch, *lens, 2, 1, 64, 0, 2)
    n = lens[0][0]
    q[..., 0], q[n // 2:, :, 0] = 1.0, 0.0
    k[..., 0] = -math.inf  # the first queries' scores: -infinity, the others': NaN
    got = _all(torch, q, k, v, do)
    for name in ("out", "rest", "dq"):
        assert not got[name][:n // 2].any() and torch.isnan(got[name][n // 2:]).all(), name
    assert (got["lse"][:n // 2] == -math.inf).all() and torch.isnan(got["lse"][n // 2:]).all()
    k[..., 0] = math.inf  # +infinity, and NaN again
    got = _all(torch, q, k, v, do)
    assert torch.isnan(got["out"]).all() and torch.isnan(got["lse"]).all()


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("heads", [(2, 2), (7, 1), (6, 2)])
@pytest.mark.parametrize("lens", [(256, 257), (512, 512), (300, 1100), (700, 255), (6, 3000)], ids=str)
def test_reach_of_hidden_infinities(lens, heads, value):
    """One key's or query's numbers within a sequence.  Results that the formulas keep apart from it keep their bits, but for
    those up to 254 places from where it is seen, which may become infinite or NaN (and nothing else)."""
    torch = gpu_ready()
    n, m = lens
    D, ahead = 64, m - n
    q, k, v, do = _inputs(torch, [n], [m], *heads, D, 0, 3)
    want = _all(torch, q, k, v, do)
    i, j = torch.arange(n, device="cuda"), torch.arange(m, device="cuda")

    def held(a, b, beside, name):
        """beside: how many places from being seen, for each row; 0 or less: the formulas say what becomes of it."""
        near = (beside > 0) & (beside <= 254)
        lost = ~torch.isfinite(a)
        assert (a == b)[beside > 254].all(), name
        assert ((a == b) | lost)[near].all(), name

    for at in sorted({0, 1, 127, 128, m // 2, m - 2, m - 1} & set(range(m))):
        beside = at - ahead - i
        bad = v.clone()
        bad[at] = value
        got = _all(torch, q, k, bad, do)
        for name in ("out", "dq"):
            held(got[name], want[name], beside, f"v {at} {name}")
            assert not torch.isfinite(got[name][(beside <= 0) & (i + ahead >= 0)]).all(-1).any()
        assert torch.equal(got["lse"], want["lse"]) and torch.equal(got["dv"], want["dv"])
        bad = k.clone()
        bad[at] = value
        got = _all(torch, q, bad, v, do)
        held(got["dq"], want["dq"], beside, f"k {at} dq")
        hidden = beside > 0
        assert torch.equal(got["out"][hidden], want["out"][hidden]) and torch.equal(got["lse"][hidden], want["lse"][hidden])
    for at in sorted({0, 1, 17, 127, 128, n // 2, n - 2, n - 1} & set(range(n))):
        beside = j - at - ahead
        others = i != at
        for which in ("q", "do"):
            bad = {"q": q.clone(), "do": do.clone()}
            bad[which][at] = value
            got = _all(torch, bad["q"] if which == "q" else q, k, v, bad["do"] if which == "do" else do)
            for name in ("out", "lse", "dq"):
                assert torch.equal(got[name][others], want[name][others]), (which, at, name)
            for name in ("dk", "dv"):
                held(got[name], want[name], beside, f"{which} {at} {name}")
