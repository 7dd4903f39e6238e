"""Gains of the norm in the shapes and types in which modules keep them."""
import pytest

from tests.gpu_util import gpu_ready
from tests.test_attention_gpu import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float64"])
@pytest.mark.parametrize("shape", [(64,), (1, 64), (1, 1, 64), (64, 1)], ids=str)
def test_gradients_have_the_gains_shape_and_type(shape, dtype):
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.attention import Rope, qk_norm_rope

    q, k, _, _ = _inputs(torch, [40], [40], 4, 2, 64, 0, 1)
    rope, pos = Rope([0.7 ** i for i in range(32)]), torch.arange(40, device="cuda")
    base = torch.rand(64, device="cuda", dtype=torch.bfloat16) + 0.5

    def grads(shape, dtype):
        gains = [base.to(dtype).view(shape).clone().requires_grad_() for _ in range(2)]
        a, b = qk_norm_rope(q, k, rope, pos, *gains)
        (a.sum() + b.square().sum()).backward()
        assert all(g.grad.shape == g.shape and g.grad.dtype == g.dtype for g in gains)
        return [g.grad.view(64) for g in gains]

    for got, want in zip(grads(shape, getattr(torch, dtype)), grads((64,), torch.float32)):
        assert torch.equal(got, want.to(got.dtype))
