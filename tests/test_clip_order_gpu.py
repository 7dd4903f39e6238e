"""What the norm of mxfp4_clip_grad_norm depends on: the gradients, and not where the clipped ones go."""
import pytest

from tests.gpu_util import gpu_ready

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_norm_does_not_depend_on_the_outputs_place(kind):
    """The same bits in place, into aligned and into unaligned buffers; the clipped values are the same too."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    dtype = getattr(torch, kind)
    for seed in range(8):
        g = torch.Generator(device="cuda").manual_seed(seed)
        grads = [torch.randn(n, device="cuda", generator=g).to(dtype) for n in (100_003, 65536, 1_000_000 + seed)]
        places = []
        for offset in (0, 1, 3):
            outs = [torch.empty(x.numel() + offset, dtype=dtype, device="cuda")[offset:] for x in grads]
            places.append((mx.clip_grad_norm(grads, 5.0, outs=outs), outs))
        places.append((mx.clip_grad_norm(grads, 5.0), grads))
        for norm, outs in places[1:]:
            assert torch.equal(norm, places[0][0])
            assert all(torch.equal(a, b) for a, b in zip(outs, places[0][1]))
