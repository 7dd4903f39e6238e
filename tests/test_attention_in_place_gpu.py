"""Outputs of attention and its gradient that are one of its inputs, where that is allowed, and its refusal where it is not."""
import pytest

from tests.gpu_util import gpu_ready
from tests.test_attention_gpu import _edges, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [(4, 2), (7, 1), (1, 1)])
@pytest.mark.parametrize("lens", [([300, 1, 77], [300, 1, 77]), ([1, 5], [2000, 3000])], ids=str)
def test_outputs_that_are_inputs(lens, heads):
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    for D in (64, 128):
        q, k, v, do = _inputs(torch, *lens, *heads, D, 9, 1)
        kw = dict(cu_q=_edges(torch, lens[0]), cu_k=_edges(torch, lens[1]))
        end = sum(lens[0])
        out, lse, rest = mx.attention(q, k, v, rest=True, **kw)
        mine = q.clone()
        got = mx.attention(mine, k, v, out=mine, **kw)
        assert got[0] is mine and torch.equal(mine[:end], out[:end]) and torch.equal(mine[end:], q[end:])
        assert torch.equal(got[1], lse)
        dq, dk, dv = mx.attention_grad(q, k, v, out, lse, do, rest=rest, **kw)
        a, b = q.clone(), do.clone()
        assert torch.equal(mx.attention_grad(a, k, v, out, lse, do, rest=rest, dq=a, **kw)[0][:end], dq[:end])
        got = mx.attention_grad(q, k, v, out, lse, b, rest=rest, dq=b, **kw)
        assert torch.equal(b[:end], dq[:end]) and torch.equal(got[1], dk) and torch.equal(got[2], dv)
        same = torch.empty_like(k)
        for bad in (lambda: mx.attention_grad(q, k, v, out, lse, do, dk=k, **kw),
                    lambda: mx.attention_grad(q, k, v, out, lse, do, dv=v, **kw),
                    lambda: mx.attention_grad(q, k, v, out, lse, do, dk=same, dv=same, **kw)):
            with pytest.raises(mx.Mxfp4Error, match="overlaps"):
                bad()
        if len(q) == len(k) and heads[0] == heads[1]:
            with pytest.raises(mx.Mxfp4Error, match="overlaps"):
                mx.attention(q, k, v, out=k, **kw)
    assert mx.device_status() == 0
