"""Norm and rotation of queries and keys, and their gradient, against 64 bits."""
import pytest

from tests.gpu_util import gpu_ready

pytestmark = pytest.mark.gpu

# tokens, query heads, key heads, head_dim, pairs, interleaved, axes
SHAPES = [(1, 32, 8, 128, 64, False, 1), (7, 3, 1, 64, 32, True, 1), (50, 4, 2, 128, 64, True, 3),
          (33, 5, 5, 72, 33, True, 3), (41, 2, 2, 80, 40, False, 3), (19, 6, 2, 128, 24, False, 1),
          (29, 1, 1, 2, 1, False, 1), (23, 2, 1, 6, 2, False, 2), (300, 2, 1, 256, 128, False, 1),
          (11, 2, 1, 256, 100, True, 1), (1300, 8, 2, 96, 48, False, 1), (9, 2, 2, 250, 125, True, 1),
          (13, 3, 1, 66, 0, False, 1)]


def _case(torch, tokens, a, b, D, P, axes, dtype, norm, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    # slices of one projection's output
    qkv = rand(tokens, a + 2 * b, D).to(dtype)
    q, k = qkv[:, :a], qkv[:, a:a + b]
    dq, dk = rand(tokens, a, D).to(dtype), rand(tokens, b, D).to(dtype)
    gains = [1 + 0.3 * rand(D), 1 + 0.3 * rand(D)] if norm else [None, None]
    positions = torch.randint(-5, 1_000_000, (axes, tokens), device="cuda", generator=g)
    freq = [500000.0 ** (-i / max(P, 1)) for i in range(P)]
    axis = [i % axes for i in range(P)]
    return q, k, dq, dk, gains, positions, freq, axis


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_both_directions(shape, dtype, norm):
    _both_directions(shape, dtype, norm)


# Warps that go through ten slices of heads or more, with head counts that fill no slice.
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", [(5001, 33, 17, 128, 64, False, 1), (5001, 33, 17, 128, 50, True, 2)], ids=str)
def test_many_tokens(shape, norm):
    _both_directions(shape, "bfloat16", norm)


def _both_directions(shape, dtype, norm):
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx
    from tests import attention_reference as ref

    tokens, a, b, D, P, interleaved, axes = shape
    dtype = getattr(torch, dtype)
    q, k, dq, dk, gains, positions, freq, axis = _case(torch, tokens, a, b, D, P, axes, dtype, norm)
    rope = mx.Rope(freq, axis, interleaved)
    eps = 1e-5
    got = mx.qk_norm_rope(q, k, rope, positions, *gains, eps=eps)
    back = mx.qk_norm_rope_grad(q, k, dq, dk, rope, positions, *gains, eps=eps)
    angle = ref.angles(positions, freq, axis) if P else torch.zeros(tokens, 0, dtype=ref.F64, device="cuda")
    own = ref.half_step(dtype)
    # fp32 on the way: the mean of D squares, a root, three products, a cosine and a sine of 2 units and an angle of
    # half a unit of pi, a product and a sum
    steps = (D / 2 + 24) * ref.U_F32
    for x, y, gain in zip((q, k), got, gains):
        want = ref.norm_rope(x, gain, eps, angle, interleaved)
        size = ref.turn_size(ref.norm_rope(x, gain, eps, angle[:, :0], interleaved), angle, interleaved)
        ref.assert_close(y, want, own * want.abs() + (1 + own) * steps * size, "forward")
    for x, dy, gain, dx, dgain in zip((q, k), (dq, dk), gains, back[:2], back[2:]):
        want, want_gain, terms, sums = ref.norm_rope_grad(x, dy, gain, eps, angle, interleaved)
        ref.assert_close(dx, want, own * want.abs() + (1 + own) * 3 * steps * terms, "dx")
        if gain is None:
            assert dgain is None
        else:  # sums over a thread's rows, a CTA's groups and the CTAs, at most 64 + 256 + 64 additions
            ref.assert_close(dgain, want_gain, (3 * steps + 384 * ref.U_F32) * sums, "dgain")
