"""Results of the autograd forms changed in place, as a program changes any other operation's."""
import pytest

from tests.gpu_util import gpu_ready
from tests.test_attention_gpu import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batched", [False, True])
def test_norm_and_rotation(batched):
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.attention import Rope, qk_norm_rope

    q, k, _, dy = _inputs(torch, [40], [40], 4, 4, 64, 0, 1)
    lead = (2, 20) if batched else (40,)
    q, k, dy = (x.view(*lead, 4, 64) for x in (q, k, dy))
    rope, pos = Rope([0.7 ** i for i in range(32)]), torch.arange(40, device="cuda").view(lead)
    grads = []
    for in_place in (True, False):
        leaves = [x.clone().requires_grad_() for x in (q, k)]
        a, b = qk_norm_rope(*leaves, rope, pos)
        if in_place:
            a.mul_(2)
            b += 1
        else:
            a, b = a * 2, b + 1
        ((a + b) * dy).sum().backward()
        grads.append((a, b, *(x.grad for x in leaves)))
    assert all(torch.equal(x, y) for x, y in zip(*grads))


@pytest.mark.parametrize("batched", [False, True])
def test_attention(batched):
    """Without gradients in place; with them the backward pass, which needs the result, says that it was changed."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.attention import attention

    q, k, v, _ = _inputs(torch, [40], [40], 4, 4, 64, 0, 2)
    q, k, v = (x.view(2, 20, 4, 64) if batched else x for x in (q, k, v))
    want = attention(q, k, v)
    assert torch.equal(attention(q, k, v).mul_(2), want * 2)
    leaf = q.clone().requires_grad_()
    with torch.no_grad():
        assert torch.equal(attention(leaf, k, v).mul_(2), want * 2)
    y = attention(leaf, k, v)
    y.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y = attention(leaf, k, v).clone()
    y.mul_(2)
    y.sum().backward()
    grad, leaf.grad = leaf.grad, None
    (attention(leaf, k, v) * 2).sum().backward()
    assert torch.equal(grad, leaf.grad)


@pytest.mark.parametrize("lead", [(64,), (2, 32)], ids=str)
def test_linear(lead):
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.linear import mxfp4_linear

    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(*lead, 128, device="cuda", generator=g).bfloat16()
    w = torch.randn(96, 128, device="cuda", generator=g).bfloat16()
    grads = []
    for in_place in (True, False):
        leaves = [t.clone().requires_grad_() for t in (x, w)]
        y = mxfp4_linear(*leaves)
        y = y.add_(1) if in_place else y + 1
        assert y.shape == (*lead, 96)
        y.square().sum().backward()
        grads.append((y, *(t.grad for t in leaves)))
    assert all(torch.equal(a, b) for a, b in zip(*grads))


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_loss(reduction):
    """Divided by the number of micro-batches, say."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.step import linear_cross_entropy

    g = torch.Generator(device="cuda").manual_seed(4)
    h = torch.randn(2, 24, 64, device="cuda", generator=g).bfloat16()
    w = (torch.randn(200, 64, device="cuda", generator=g) / 8).bfloat16()
    targets = torch.randint(0, 200, (2, 24), device="cuda", generator=g)
    grads = []
    for in_place in (True, False):
        leaves = [t.clone().requires_grad_() for t in (h, w)]
        loss = linear_cross_entropy(*leaves, targets, reduction=reduction)
        loss = loss.div_(4) if in_place else loss / 4
        assert loss.shape == (targets.shape if reduction == "none" else ())
        loss.sum().backward()
        grads.append((loss, *(t.grad for t in leaves)))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
