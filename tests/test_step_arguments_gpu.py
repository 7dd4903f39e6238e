"""What the step operators take and refuse from Python."""
import pytest

from tests.gpu_util import gpu_ready

pytestmark = pytest.mark.gpu


def test_embedding_takes_a_table_with_other_strides():
    """A transposed table and columns of a wider one give what contiguous ones give, gradients included."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.step import embedding

    ids = torch.randint(0, 50, (3, 11), device="cuda")
    base = torch.randn(24, 50, device="cuda")
    wide = torch.randn(50, 40, device="cuda")
    for w in (base.t(), wide[:, 5:29], wide[:, ::2], wide[:1, :24].expand(50, 24)):
        a, b = w.detach().requires_grad_(), w.detach().contiguous().requires_grad_()
        ya, yb = embedding(ids, a, scale=3.0), embedding(ids, b, scale=3.0)
        assert torch.equal(ya, yb)
        dy = torch.randn_like(ya)
        ya.backward(dy)
        yb.backward(dy)
        assert torch.equal(a.grad, b.grad)


def test_targets_belong_to_their_tokens():
    """Targets of the hidden states' leading shape, or either of the two laid out flat; nothing else, even of the same
    number of elements."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.step import linear_cross_entropy

    h = torch.randn(3, 5, 16, device="cuda").bfloat16()
    w = torch.randn(40, 16, device="cuda").bfloat16()
    y = torch.randint(0, 40, (3, 5), device="cuda")
    want = linear_cross_entropy(h, w, y, reduction="none")
    assert torch.equal(linear_cross_entropy(h, w, y.reshape(-1), reduction="none"), want.reshape(-1))
    assert torch.equal(linear_cross_entropy(h.reshape(-1, 16), w, y, reduction="none"), want)
    for bad in (y.t(), y.reshape(5, 3), y[None], y[:, :4]):
        with pytest.raises(ValueError):
            linear_cross_entropy(h, w, bad)
    for bad in (w[None], w[0]):
        with pytest.raises(ValueError):
            linear_cross_entropy(h, bad, y)


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Every call wants its tensors on the current device (here: another index is made out to be the current one)."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx
    from mxfp4_precision_gemms_gb300 import step

    w = torch.randn(40, 16, device="cuda").bfloat16()
    ids = torch.randint(0, 40, (9,), device="cuda")
    h = torch.randn(9, 16, device="cuda").bfloat16()
    loss, lse = mx.linear_ce(h, w, ids)
    p = torch.zeros(8, device="cuda", requires_grad=True)
    p.grad = torch.ones(8, device="cuda")
    out = torch.empty(8, device="cuda")
    calls = [lambda: mx.embedding(ids, w), lambda: mx.embedding_grad(ids, h, 40), lambda: mx.linear_ce(h, w, ids),
             lambda: mx.linear_ce_grad(h, w, ids, lse, loss), lambda: mx.clip_grad_norm([p.grad], 1.0),
             lambda: mx.clip_grad_norm([p.grad], 1.0, outs=[out]), lambda: step.embedding(ids, w),
             lambda: step.linear_cross_entropy(h, w, ids), lambda: step.clip_grad_norm_([p], 1.0)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(mx, "_current_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


def test_each_tensor_of_a_call_is_looked_at():
    """One tensor on the host among those on the device is refused, whichever it is."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    w = torch.randn(40, 16, device="cuda").bfloat16()
    ids = torch.randint(0, 40, (9,), device="cuda")
    h = torch.randn(9, 16, device="cuda").bfloat16()
    loss, lse = mx.linear_ce(h, w, ids)
    dw, dh = torch.empty(40, 16, device="cuda").bfloat16(), torch.empty_like(h)
    g = torch.ones(8, device="cuda")
    for call, args in ((mx.embedding, (ids, w)), (mx.embedding_grad, (ids, h)), (mx.linear_ce, (h, w, ids)),
                       (mx.linear_ce_grad, (h, w, ids, lse, loss))):
        extra = {"vocab": 40} if call is mx.embedding_grad else {}
        call(*args, **extra)
        for i in range(len(args)):
            with pytest.raises(ValueError):
                call(*(x.cpu() if j == i else x for j, x in enumerate(args)), **extra)
    for bad in (lambda: mx.embedding(ids, w, out=h.cpu()), lambda: mx.embedding_grad(ids, h, 40, dw=dw.cpu()),
                lambda: mx.linear_ce_grad(h, w, ids, lse, loss, dh=dh.cpu()),
                lambda: mx.linear_ce_grad(h, w, ids, lse, loss, dw=dw.cpu()),
                lambda: mx.clip_grad_norm([g, g.cpu()], 1.0), lambda: mx.clip_grad_norm([g], 1.0, outs=[g.cpu()])):
        with pytest.raises(ValueError):
            bad()


def test_cross_entropy_takes_weights_off_16_bytes():
    """Contiguous weights that start anywhere, as a view into a flat buffer may, give what aligned ones give."""
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300.step import linear_cross_entropy

    h = torch.randn(30, 24, device="cuda").bfloat16()
    flat = torch.randn(40 * 24 + 8, device="cuda").bfloat16()
    y = torch.randint(0, 40, (30,), device="cuda")
    for shift in (1, 3, 4):
        w = flat[shift:shift + 40 * 24].view(40, 24)
        a, b = w.detach().requires_grad_(), w.detach().clone().requires_grad_()
        la, lb = linear_cross_entropy(h, a, y), linear_cross_entropy(h, b, y)
        la.backward(), lb.backward()
        assert torch.equal(la, lb) and torch.equal(a.grad, b.grad)
