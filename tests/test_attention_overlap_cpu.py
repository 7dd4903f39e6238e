"""Outputs of attention and its gradient over inputs that are still read, and over each other, are refused on the host."""
import random

import pytest

from tests.test_attention_refusals_cpu import INVALID, PASSED, L, _attention  # noqa: F401

B = 0x10000  # a base; 6 queries and 9 keys, 8 and 2 heads of 128, as in _attention


def _no_gpu():
    import torch

    if torch.cuda.is_available():
        pytest.skip("pointers of this test are not device memory")


@pytest.mark.parametrize("change", [
    dict(out=(0x20000, 1536, 128, 8, 1)), dict(out=(0x30000, 1536, 128, 8, 1)),   # k and v
    dict(out=(0x20000, 1024, 128, 8, 1)),                                         # k, with other strides
    dict(out=(0x20000 + 2 * 1536 * 8, 1536, 128, 8, 1)),                          # k's last row
    dict(rest=(0x40000, 1024, 128, 8, 1)), dict(rest=(0x40000 + 256, 1024, 128, 8, 1)),  # out
    dict(rest=(0x30000, 1536, 128, 8, 1)), dict(out=(B + 256, 1536, 128, 8, 1)),  # v; q shifted by a head
    dict(out=(B + 2 * 1536, 1536, 128, 8, 1))])                                   # q shifted by a token
def test_attention_refuses_outputs_over_inputs(L, change):  # noqa: F811
    assert _attention(L, **change) == INVALID
    assert b"overlaps" in L.mxfp4_last_error()


@pytest.mark.parametrize("change", [
    dict(dk=(0x20000, 1536, 128, 2, 1)), dict(dv=(0x30000, 1536, 128, 2, 1)), dict(dk=(0x30000, 256, 128, 2, 1)),
    dict(dv=(0x80000, 256, 128, 2, 1)), dict(dv=(0x80000 + 256, 256, 128, 2, 1)), dict(dq=(0x80000, 1024, 128, 8, 1)),
    dict(dq=(0x20000, 1536, 128, 8, 1)), dict(dk=(0x60000, 1024, 128, 2, 1)), dict(dv=(B, 1536, 128, 2, 1)),
    dict(dq=(B + 256, 1536, 128, 8, 1)), dict(dq=(0x60000 + 2048, 1024, 128, 8, 1))])
def test_attention_gradient_refuses_outputs_over_inputs(L, change):  # noqa: F811
    assert _attention(L, grad=True, **change) == INVALID
    assert b"overlaps" in L.mxfp4_last_error()


SLICES = dict(q=(B, 1536, 128, 8, 1), k=(B + 2048, 1536, 128, 2, 1), v=(B + 2560, 1536, 128, 2, 1))  # of one projection
GRADS = dict(dq=(0x70000, 1536, 128, 8, 1), dk=(0x70000 + 2048, 1536, 128, 2, 1), dv=(0x70000 + 2560, 1536, 128, 2, 1))


@pytest.mark.parametrize("grad,change", [
    (False, SLICES), (False, dict(out=(B, 1536, 128, 8, 1))), (False, dict(SLICES, out=(B, 1536, 128, 8, 1))),
    (False, dict(rest=(B, 1536, 128, 8, 1))), (False, dict(m=0, k=(0, 0, 128, 2, 1), v=(0, 0, 128, 2, 1))),
    (False, dict(q=(B, 128, 768, 8, 1), out=(B + 2 * 8 * 768, 128, 768, 8, 1))),  # heads of tokens, one behind the other
    (True, dict(SLICES, **GRADS)), (True, dict(dq=(B, 1536, 128, 8, 1))), (True, dict(dq=(0x60000, 1024, 128, 8, 1))),
    (True, dict(SLICES, dq=(B, 1536, 128, 8, 1))), (True, dict(dk=(0x40000, 1024, 128, 2, 1)))])
def test_attention_takes(L, grad, change):  # noqa: F811
    _no_gpu()
    assert _attention(L, grad=grad, **dict(dict(n=6, m=6, seqs=2), **change)) == PASSED


def test_overlap_is_exact_for_equal_strides(L):  # noqa: F811
    """out against k at random places of a small buffer, element by element."""
    _no_gpu()
    rng = random.Random(0)
    far, D, seen = 1 << 30, 8, {True: 0, False: 0}
    for _ in range(3000):
        b, group, n, m = rng.randint(1, 3), rng.randint(1, 2), rng.randint(1, 5), rng.randint(1, 5)
        a = b * group
        if rng.random() < 0.5:  # tokens of heads, or heads of tokens
            head = D * rng.randint(1, 3)
            token = (a - 1) * head + D * rng.randint(1, 6)
        else:
            token = D * rng.randint(1, 3)
            head = (n - 1) * token + D * rng.randint(1, 6)
        at = [B + 16 * rng.randint(0, 60) for _ in range(2)]

        def elements(start, tokens, heads):
            return {start + 2 * (t * token + h * head) + 16 * x for t in range(tokens) for h in range(heads) for x in range(D // 8)}

        want = bool(elements(at[0], n, a) & elements(at[1], m, b))
        got = _attention(L, n=n, m=m, dim=D, seqs=1, q=(far, D * a, D, a, 1), k=(at[1], token, head, b, 1),
                         v=(2 * far, D * b, D, b, 1), out=(at[0], token, head, a, 1))
        assert got == (INVALID if want else PASSED), (a, b, n, m, token, head, at)
        seen[want] += 1
    assert min(seen.values()) > 500
