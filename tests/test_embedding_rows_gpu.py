"""Embedding rows that are moved one element at a time because a base or a width misses the vectors' alignment: fp32 on a
16-byte base that is not a 32-byte one, and widths of a multiple of four.  Against the aligned call: the lookup and the
sums are the same operations in the same order, so the bits are the same."""
import pytest

from tests.gpu_util import gpu_ready

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [40, 3000])
@pytest.mark.parametrize("kind,shift,dim", [("float32", 4, 64), ("float32", 1, 64), ("bfloat16", 4, 64),
                                            ("float32", 0, 36), ("bfloat16", 0, 36)])
def test_rows_off_the_vectors_alignment(tokens, kind, shift, dim):
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    dtype, vocab = getattr(torch, kind), 300
    out = mx._OUT_OF[dtype]

    def shifted(x):
        y = torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")[shift:].view(x.shape)
        return y.copy_(x)

    g = torch.Generator(device="cuda").manual_seed(tokens + dim)
    ids = torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
    pad = (dim + 7) // 8 * 8  # rows of a multiple of eight, with zeros behind the ones compared
    w = torch.zeros(vocab, pad, dtype=dtype, device="cuda")
    dy = torch.zeros(tokens, pad, dtype=dtype, device="cuda")
    w[:, :dim] = torch.randn(vocab, dim, device="cuda", generator=g)
    dy[:, :dim] = torch.randn(tokens, dim, device="cuda", generator=g)
    wo, dyo = shifted(w[:, :dim].contiguous()), shifted(dy[:, :dim].contiguous())
    assert torch.equal(mx.embedding(ids, wo, scale=3.0), mx.embedding(ids, w, scale=3.0)[:, :dim])
    dw0 = torch.randn(vocab, pad, device="cuda", generator=g).to(dtype)
    for accumulate in (False, True):
        a, b = shifted(dw0[:, :dim].contiguous()), dw0.clone()
        mx.embedding_grad(ids, dyo, vocab, scale=3.0, padding_id=5, out_dtype=out, accumulate=accumulate, dw=a)
        mx.embedding_grad(ids, dy, vocab, scale=3.0, padding_id=5, out_dtype=out, accumulate=accumulate, dw=b)
        assert torch.equal(a, b[:, :dim])
    assert mx.device_status() == 0
