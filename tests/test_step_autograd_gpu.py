"""The autograd forms of the embedding, the output layer's cross entropy and gradient clipping: against
torch's own autograd in fp64, and together with MXFP4 linear layers in the example's training run."""
import importlib.util
import math
import os

import pytest

from tests.gpu_util import gpu_ready

pytestmark = pytest.mark.gpu


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_tied_embedding_and_loss_against_fp64(reduction):
    """loss(embedding(ids)) with one table used at both ends, a batch of sequences, padding and ignored
    targets.  Each gradient is rounded to bf16 from dz in bf16 (2^-8 each), and the tied one is the
    rounded sum of two such: 2^-6 in all."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.step import embedding, linear_cross_entropy

    g = torch.Generator(device="cuda").manual_seed(0)
    B, S, V, D, pad = 3, 70, 500, 96, 7
    w = (torch.randn(V, D, device="cuda", generator=g) / 8).bfloat16().requires_grad_()
    m = torch.randn(D, D, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, V, (B, S), device="cuda", generator=g)
    ids[:, -5:] = pad
    targets = torch.where(ids == pad, torch.full_like(ids, -100), ids.roll(-1, 1))
    out = linear_cross_entropy(embedding(ids, w, scale=2.0, padding_id=pad) @ m, w, targets, reduction=reduction)
    assert out.shape == (targets.shape if reduction == "none" else ())
    k = torch.rand(out.shape, device="cuda", generator=g)
    (out * k).sum().backward()

    w64 = w.detach().double().requires_grad_()
    e = torch.nn.functional.embedding(ids, w64, padding_idx=pad) * 2.0
    # the product between the two is rounded to bf16 in the path that is tested
    x = e + ((embedding(ids, w.detach(), scale=2.0) @ m).double() - (e @ m.double())).detach() @ torch.linalg.inv(m.double())
    logits = x @ m.double() @ w64.t()
    want = torch.nn.functional.cross_entropy(logits.reshape(-1, V), targets.reshape(-1), ignore_index=-100,
                                             reduction=reduction).reshape(out.shape)
    (want * k.double()).sum().backward()
    assert _rel(out.detach(), want.detach()) < 1e-5
    assert w.grad.dtype == torch.bfloat16 and _rel(w.grad, w64.grad) < 2.0 ** -6


def test_only_the_gradients_that_are_asked_for():
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.step import linear_cross_entropy

    h = torch.randn(40, 64, device="cuda").bfloat16()
    w = torch.randn(90, 64, device="cuda").bfloat16()
    y = torch.randint(0, 90, (40,), device="cuda")
    hg, wg = h.clone().requires_grad_(), w.clone().requires_grad_()
    linear_cross_entropy(hg, wg, y).backward()
    h1 = h.clone().requires_grad_()
    linear_cross_entropy(h1, w, y).backward()
    w1 = w.clone().requires_grad_()
    linear_cross_entropy(h, w1, y).backward()
    assert torch.equal(h1.grad, hg.grad) and torch.equal(w1.grad, wg.grad)
    t = torch.randn(64, 40, device="cuda").bfloat16()  # columns of a transposed activation
    ht, hc = t.t().requires_grad_(), t.t().contiguous().requires_grad_()
    linear_cross_entropy(ht, w, y).backward()
    linear_cross_entropy(hc, w, y).backward()
    assert torch.equal(ht.grad, hc.grad)
    with pytest.raises(ValueError):
        linear_cross_entropy(h, w, y, reduction="median")


def test_broadcast_and_strided_inputs():
    """Gradients that arrive broadcast (rows or all elements shared), hidden states that are one row repeated, and
    weights that are columns of a wider matrix give what contiguous ones give."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.step import embedding, linear_cross_entropy

    w = torch.randn(50, 24, device="cuda").requires_grad_()
    ids = torch.randint(0, 50, (4, 9), device="cuda")
    v = torch.randn(24, device="cuda")
    for out in (embedding(ids, w), embedding(ids, w) @ torch.diag(v)):
        w.grad = None
        out.sum().backward()
        want = torch.zeros(50, 24, device="cuda").index_add_(0, ids.reshape(-1), (v if out.grad_fn.name() != "EmbeddingFunctionBackward" else torch.ones_like(v)).expand(36, 24))
        assert torch.allclose(w.grad, want, rtol=1e-6, atol=1e-6)
    w.grad = None
    embedding(ids, w).backward(v.expand(4, 9, 24))  # one row for all tokens
    assert torch.allclose(w.grad, torch.zeros(50, 24, device="cuda").index_add_(0, ids.reshape(-1), v.expand(36, 24)), rtol=1e-5)

    h = torch.randn(1, 64, device="cuda").bfloat16().requires_grad_()
    wide = torch.randn(300, 99, device="cuda").bfloat16()
    wo = wide[:, 3:67].detach().requires_grad_()
    y = torch.randint(0, 300, (40,), device="cuda")
    linear_cross_entropy(h.expand(40, 64), wo, y, reduction="sum").backward()
    hc, wc = h.detach().repeat(40, 1).requires_grad_(), wo.detach().contiguous().requires_grad_()
    linear_cross_entropy(hc, wc, y, reduction="sum").backward()
    assert torch.equal(wo.grad, wc.grad)
    assert float((h.grad.float() - hc.grad.float().sum(0)).abs().max()) <= 2.0 ** -7 * float(hc.grad.float().abs().sum(0).max())


def test_concurrent_streams():
    """Calls on three streams at once: each has its own workspace, so each gives what it gives alone."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    g = torch.Generator(device="cuda").manual_seed(5)
    sets = []
    for i in range(3):
        T, V, D = (700, 3000, 256) if i else (2500, 9000, 64)
        sets.append((torch.randn(T, D, device="cuda", generator=g).bfloat16(),
                     (torch.randn(V, D, device="cuda", generator=g) / 8).bfloat16(),
                     torch.randint(0, V, (T,), device="cuda", generator=g)))
    one = torch.ones(1, device="cuda")

    def work(h, w, y, stream=None):
        loss, lse = mx.linear_ce(h, w, y, stream=stream)
        dh, dw = mx.linear_ce_grad(h, w, y, lse, one, stream=stream)
        de = mx.embedding_grad(y, h, w.shape[0], stream=stream)
        e = mx.embedding(y, w, stream=stream)
        norm = mx.clip_grad_norm([dw, dh], 1e-3, stream=stream)
        return loss, lse, dh, dw, de, e, norm

    alone = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        both = [work(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            for x, z in zip(a, b):
                assert torch.equal(x, z)
    assert mx.device_status() == 0


def test_clip_grad_norm_on_parameters():
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.step import clip_grad_norm_

    ps = [torch.zeros(300, 20, device="cuda", requires_grad=True), torch.zeros(7, device="cuda", dtype=torch.bfloat16, requires_grad=True),
          torch.zeros(50, 60, device="cuda", requires_grad=True), torch.zeros(5, device="cuda", requires_grad=True)]
    ps[0].grad, ps[1].grad = torch.randn(300, 20, device="cuda"), torch.randn(7, device="cuda").bfloat16()
    ps[2].grad = torch.randn(60, 50, device="cuda").t()  # other strides; ps[3] has no gradient
    before = [p.grad.double().clone() for p in ps[:3]]
    n = math.sqrt(sum(float((b ** 2).sum()) for b in before))
    norm = clip_grad_norm_(iter(ps), 3.0)
    assert abs(float(norm) - n) < 1e-5 * n and ps[3].grad is None
    for p, b in zip(ps, before):
        # one rounding to bf16 (2^-8), or three fp32 ones
        tol = 2.0 ** -8 if p.dtype == torch.bfloat16 else 1e-5
        assert bool(((p.grad.double() - b * 3.0 / n).abs() <= tol * (b * 3.0 / n).abs()).all())
    assert float(clip_grad_norm_(ps[0], 1e9)) > 0


def test_clip_grad_norm_counts_a_tied_parameter_once():
    """A weight that is listed twice is scaled once, by the factor of the norm that has it once."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.step import clip_grad_norm_

    ps = [torch.zeros(1000, 33, device="cuda", requires_grad=True), torch.zeros(10, device="cuda", requires_grad=True)]
    for p in ps:
        p.grad = torch.randn(p.shape, device="cuda")
    before = [p.grad.double().clone() for p in ps]
    n = math.sqrt(sum(float((b ** 2).sum()) for b in before))
    norm = clip_grad_norm_([ps[0], ps[1], ps[0]], 2.0)
    assert abs(float(norm) - n) < 1e-5 * n
    for p, b in zip(ps, before):
        assert bool(((p.grad.double() - b * 2.0 / n).abs() <= 1e-5 * (b * 2.0 / n).abs()).all())


def test_example_trains():
    """The example's model learns its chain: from about log(vocab) well towards log(4)."""
    gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tiny_lm.py")
    spec = importlib.util.spec_from_file_location("tiny_lm", path)
    lm = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(lm)
    losses = lm.train(steps=40, tokens=1024, vocab=500, dim=128, say=lambda *_: None)
    assert mx.device_status() == 0 and all(math.isfinite(x) for x in losses)
    assert abs(losses[0] - math.log(500)) < 1.0
    assert losses[-1] < losses[0] - 2.0
