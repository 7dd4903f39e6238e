"""Linear cross entropy and its gradients (mxfp4_linear_ce, mxfp4_linear_ce_grad) against the formulas in
64 bits on the same bf16 inputs.

Tolerances, element by element (u = 2^-24):
  a logit is a sum of dim exact products, added up in fp32 (each addition within 2u of the running sum, which
  the absolute sum S bounds):  ez = 2u * dim * S.
  lse: ez, plus the error of a sum of exponentials (each within 4u + the rounding of its argument, 2u * |z| *
  log2 e; added in chains no longer than 64 + the vocabulary's tiles): el = ez + u * (128 + vocab / 128 + 8 |lse| +
  8 max|z|);  the loss: el + ez.
  dz = p - [target]: p within p * 2 * (el + ez); rounded to bf16, 2^-8 |dz| (half an ulp is at most 2^-8 of the
  value) -- then products added up in fp32 over n terms: 2u * n * sum|dz||x|.
  A bf16 output adds 2^-8 of the result."""
import math

import pytest

from tests.gpu_util import gpu_ready

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _setup():
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    return torch, mx


def _inputs(torch, T, V, D, seed, ignored=0.0, pitch_h=None, pitch_w=None, sharp=6.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rows(n, pitch):  # what lies between rows is NaN
        x = torch.full((n, pitch or D), float("nan"), dtype=torch.bfloat16, device="cuda")
        x[:, :D] = torch.randn(n, D, device="cuda", generator=g)
        return x[:, :D]

    w = rows(V, pitch_w)
    w *= 1.3 / D ** 0.5
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    h = rows(T, pitch_h)
    h += sharp * torch.rand(T, 1, device="cuda", generator=g).bfloat16() * w[y]
    if ignored:
        out = torch.rand(T, device="cuda", generator=g) < ignored
        y = torch.where(out, torch.full_like(y, -100), y)
        h[out] = float("nan")  # must never be read
        h[out, ::2] = float("inf")
    return h, w, y


def _reference(torch, h, w, y):
    """(keep, z, S, lse, loss) over the counted tokens, fp64."""
    keep = (y >= 0).nonzero()[:, 0]
    hd, wd = h[keep].double(), w.double()
    z = hd @ wd.t()
    S = hd.abs() @ wd.abs().t()
    lse = torch.logsumexp(z, 1)
    loss = lse - z.gather(1, y[keep].long()[:, None])[:, 0]
    return keep, z, S, lse, loss


def _tolerances(torch, z, S, lse, V, D):
    ez = (2 * U * D * S).amax(1)
    el = ez + U * (128 + V / 128 + 8 * lse.abs() + 8 * z.abs().amax(1))
    return ez, el


def _check_forward(torch, mx, h, w, y, ref=None):
    T, D = h.shape
    V = w.shape[0]
    keep, z, S, lse, loss = ref or _reference(torch, h, w, y)
    ez, el = _tolerances(torch, z, S, lse, V, D)
    got, got_lse = mx.linear_ce(h, w, y, reduction=mx.REDUCE_NONE)
    assert mx.device_status() == 0
    assert bool(((got_lse.double()[keep] - lse).abs() <= el).all()), float(((got_lse.double()[keep] - lse).abs() / el).max())
    assert bool(((got.double()[keep] - loss).abs() <= el + ez).all())
    off = torch.ones(T, dtype=torch.bool, device="cuda")
    off[keep] = False
    assert not got[off].any() and not got_lse[off].any()
    total, lse2 = mx.linear_ce(h, w, y, reduction=mx.REDUCE_SUM)
    mean, _ = mx.linear_ce(h, w, y, reduction=mx.REDUCE_MEAN)
    assert torch.equal(lse2, got_lse)
    tol = float((el + ez).sum()) + U * (T / 1024 + 16) * float(loss.abs().sum())
    assert abs(float(total) - float(loss.sum())) <= tol
    n = max(1, len(keep))
    assert abs(float(mean) - float(loss.sum()) / n) <= (tol + 4 * U * float(loss.abs().sum())) / n
    return got_lse


def _check_grad(torch, mx, h, w, y, lse, ref, reduction, out, accumulate=False, dw0=None, seed=0):
    T, D = h.shape
    V = w.shape[0]
    keep, z, S, lse64, loss = ref
    n = len(keep)
    ez, el = _tolerances(torch, z, S, lse64, V, D)
    g = torch.Generator(device="cuda").manual_seed(seed)
    if reduction == mx.REDUCE_NONE:
        dloss = torch.randn(T, device="cuda", generator=g)
        gt = dloss.double()[keep]
        dloss[y < 0] = float("nan")  # of ignored tokens: must not be used
    else:
        dloss = torch.full((1,), 0.7, device="cuda")
        gt = dloss.double().expand(n) / (max(1, n) if reduction == mx.REDUCE_MEAN else 1)
    kind = {mx.OUT_F32: torch.float32, mx.OUT_BF16: torch.bfloat16}[out]
    dw = None if dw0 is None else dw0.clone()
    dh, dw = mx.linear_ce_grad(h, w, y, lse, dloss, reduction=reduction, dh_dtype=out, dw_dtype=out, accumulate=accumulate,
                               dw=dw)
    assert mx.device_status() == 0 and dh.dtype == kind and dw.dtype == kind
    p = torch.exp(z - lse64[:, None])
    dz = p.clone()
    dz[torch.arange(n, device="cuda"), y[keep].long()] -= 1.0
    ed = gt.abs()[:, None] * (p * 2 * (el + ez)[:, None] + (2.0 ** -8 + 4 * U) * dz.abs()) + 2.0 ** -120
    dz *= gt[:, None]
    hd, wd = h[keep].double(), w.double()
    want_h = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    tol_h = want_h.clone()
    want_h[keep] = dz @ wd
    tol_h[keep] = (ed + 2 * U * (V + 32) * dz.abs()) @ wd.abs()
    want_w = dz.t() @ hd
    tol_w = (ed + 2 * U * (n + 32) * dz.abs()).t() @ hd.abs()
    if accumulate:
        want_w = want_w + dw0.double()
        tol_w = tol_w + 2 * U * (want_w.abs() + dw0.double().abs())
    for got, want, tol, name in ((dh, want_h, tol_h, "dh"), (dw, want_w, tol_w, "dw")):
        tol = tol + (2.0 ** -8 if out == mx.OUT_BF16 else 4 * U) * want.abs()
        err = (got.double() - want).abs()
        bad = ~(err <= tol)
        assert not bool(bad.any()), (name, int(bad.sum()), bad.nonzero()[:4].tolist(), float((err / tol).nan_to_num().max()))
        norm = float(want.norm())
        if norm and V >= 255:  # two roundings of at most 2^-8 (with few ids dz cancels below the logits' own error)
            assert float((got.double() - want).norm()) <= 2.0 ** -7 * norm
    off = torch.ones(T, dtype=torch.bool, device="cuda")
    off[keep] = False
    assert not dh[off].any()


SHAPES = [(1, 1, 8), (1, 2, 8), (3, 5, 16), (1, 1000, 64), (7, 255, 72), (127, 257, 64), (128, 256, 128),
          (129, 513, 264), (255, 1000, 40), (257, 4099, 136), (700, 3001, 520), (1500, 777, 256)]


@pytest.mark.parametrize("ignored", [0.0, 0.5])
@pytest.mark.parametrize("T,V,D", SHAPES)
def test_loss_and_gradients(T, V, D, ignored):
    torch, mx = _setup()
    h, w, y = _inputs(torch, T, V, D, T + V, ignored)
    ref = _reference(torch, h, w, y)
    lse = _check_forward(torch, mx, h, w, y, ref)
    for reduction in (mx.REDUCE_MEAN, mx.REDUCE_SUM, mx.REDUCE_NONE):
        for out in (mx.OUT_F32, mx.OUT_BF16):
            _check_grad(torch, mx, h, w, y, lse, ref, reduction, out)


def test_several_pieces_and_accumulation():
    """A vocabulary of several pieces (2048 columns at the least) with a long batch, and dw added to."""
    torch, mx = _setup()
    T, V, D = 40000, 15001, 64
    h, w, y = _inputs(torch, T, V, D, 5, 0.1)
    L = mx.lib()
    # the workspace holds one piece of dz, not tokens x vocab
    assert L.mxfp4_linear_ce_grad_workspace_bytes(T, V, D) < 2 * T * V + 6 * T * D + (1 << 20)
    ref = _reference(torch, h, w, y)
    lse = _check_forward(torch, mx, h, w, y, ref)
    dw0 = torch.randn(V, D, device="cuda")
    _check_grad(torch, mx, h, w, y, lse, ref, mx.REDUCE_SUM, mx.OUT_F32, True, dw0)
    _check_grad(torch, mx, h, w, y, lse, ref, mx.REDUCE_MEAN, mx.OUT_BF16)


def test_pitched_rows_int32_targets_and_other_ignore_index():
    torch, mx = _setup()
    for D, ph, pw in ((64, 65, 72), (136, 144, 160)):
        h, w, y = _inputs(torch, 300, 700, D, D, 0.3, ph, pw)
        ref = _reference(torch, h, w, y)
        lse = _check_forward(torch, mx, h, w, y, ref)
        other = torch.where(y < 0, torch.full_like(y, 699), torch.where(y == 699, torch.full_like(y, 5), y)).int()
        h0 = torch.where((other == 699)[:, None], torch.full_like(h, float("nan")), h)
        a, la = mx.linear_ce(h0, w, other, ignore_index=699, reduction=mx.REDUCE_NONE)
        b, lb = mx.linear_ce(h, w, torch.where(other == 699, torch.full_like(other, -100), other).long(),
                             reduction=mx.REDUCE_NONE)
        assert torch.equal(a, b) and torch.equal(la, lb)
        one = torch.ones(1, device="cuda")
        want_h, want_w = mx.linear_ce_grad(h, w, y, lse, one)
        dh = torch.full((300, D + 3), 7.0, dtype=torch.bfloat16, device="cuda")
        dw = torch.full((700, pw), 7.0, dtype=torch.bfloat16, device="cuda")
        mx.linear_ce_grad(h, w, y, lse, one, dh=dh[:, 1:D + 1], dw=dw[:, :D])
        assert torch.equal(dh[:, 1:D + 1], want_h) and torch.equal(dw[:, :D], want_w)
        assert bool((dh[:, D + 1:] == 7).all()) and bool((dh[:, 0] == 7).all()) and bool((dw[:, D:] == 7).all())
        only_h, none = mx.linear_ce_grad(h, w, y, lse, one, dw_dtype=None)
        assert none is None and torch.equal(only_h, want_h)
        none, only_w = mx.linear_ce_grad(h, w, y, lse, one, dh_dtype=None)
        assert none is None and torch.equal(only_w, want_w)


def test_nothing_counts_and_no_tokens():
    torch, mx = _setup()
    h = torch.full((300, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    w = torch.randn(500, 64, device="cuda").bfloat16()
    y = torch.full((300,), -100, device="cuda")
    one = torch.ones(1, device="cuda")
    for red in (mx.REDUCE_MEAN, mx.REDUCE_SUM, mx.REDUCE_NONE):
        loss, lse = mx.linear_ce(h, w, y, reduction=red)
        assert not loss.any() and not lse.any()
    dh, dw = mx.linear_ce_grad(h, w, y, lse, one)
    assert not dh.any() and not dw.any()
    kept = torch.randn(500, 64, device="cuda")
    dw = kept.clone()
    mx.linear_ce_grad(h, w, y, lse, one, dw=dw, dw_dtype=mx.OUT_F32, accumulate=True)
    assert torch.equal(dw, kept)
    loss, lse = mx.linear_ce(h[:0], w, y[:0])
    assert float(loss) == 0.0 and lse.shape == (0,)
    dh, dw = mx.linear_ce_grad(h[:0], w, y[:0], lse, one)
    assert dh.shape == (0, 64) and not dw.any()
    assert mx.device_status() == 0


def test_bad_targets_are_reported_and_left_out():
    torch, mx = _setup()
    h, w, y = _inputs(torch, 50, 100, 64, 1)
    bad = y.clone()
    bad[3], bad[7], bad[49] = 100, -1, 1 << 40
    a, la = mx.linear_ce(h, w, bad, reduction=mx.REDUCE_NONE)
    assert mx.device_status() == 1 and b"vocabulary" in mx.lib().mxfp4_last_error()
    good = torch.where((bad < 0) | (bad >= 100), torch.full_like(bad, -100), bad)
    b, lb = mx.linear_ce(h, w, good, reduction=mx.REDUCE_NONE)
    assert torch.equal(a, b) and torch.equal(la, lb) and mx.device_status() == 0


def test_extreme_logits():
    """Saturated softmax (a logit far above the rest), equal logits, and infinities / NaN of a counted row,
    which go into its loss and gradients as the formulas say and into no other row's loss."""
    torch, mx = _setup()
    T, V, D = 40, 300, 64
    h, w, y = _inputs(torch, T, V, D, 2, sharp=0.0)
    h[1] = w[y[1]] * 3000  # its target takes everything
    h[2] = w[(y[2] + 1) % V] * 3000  # another id does
    h[3] = 0  # all logits equal
    ref = _reference(torch, h, w, y)
    lse = _check_forward(torch, mx, h, w, y, ref)
    _check_grad(torch, mx, h, w, y, lse, ref, mx.REDUCE_SUM, mx.OUT_F32)
    clean, _ = mx.linear_ce(h, w, y, reduction=mx.REDUCE_NONE)
    h[5, 3], h[6, 0] = float("inf"), float("nan")
    loss, lse = mx.linear_ce(h, w, y, reduction=mx.REDUCE_NONE)
    rest = [t for t in range(T) if t not in (5, 6)]
    assert bool(loss[5:7].isnan().all()) and torch.equal(loss[rest], clean[rest])
    dh, dw = mx.linear_ce_grad(h, w, y, lse, torch.ones(1, device="cuda"))
    assert bool(dh[5:7].isnan().all()) and bool(dw.isnan().all()) and not bool(dh[rest].isnan().any())


def test_gradient_against_differences():
    """Central differences of the summed loss along the gradient's own signs.  h and w lie on grids that
    make the steps exact in bf16; the cubic term of the difference and the bf16 rounding of dz stay
    below 2% of the derivative (a step moves a logit by at most 0.2)."""
    torch, mx = _setup()
    g = torch.Generator(device="cuda").manual_seed(3)
    T, V, D = 64, 300, 64
    h = (torch.randint(-32, 33, (T, D), device="cuda", generator=g) / 32).bfloat16()
    w = (torch.randint(-16, 17, (V, D), device="cuda", generator=g) / 64).bfloat16()
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    y[::5] = -100
    _, lse = mx.linear_ce(h, w, y)
    dh, dw = mx.linear_ce_grad(h, w, y, lse, torch.ones(1, device="cuda"), reduction=mx.REDUCE_SUM,
                               dh_dtype=mx.OUT_F32, dw_dtype=mx.OUT_F32)
    f = lambda a, b: float(mx.linear_ce(a, b, y, reduction=mx.REDUCE_NONE)[0].double().sum())  # noqa: E731
    dirs = torch.sign(dh).bfloat16()
    e = 2.0 ** -6
    want = float((dh.double() * dirs.double()).sum()) * 2 * e
    got = f(h + e * dirs, w) - f(h - e * dirs, w)
    assert abs(got - want) <= 0.02 * abs(want)
    dirs = torch.sign(dw).bfloat16()
    e = 2.0 ** -8
    want = float((dw.double() * dirs.double()).sum()) * 2 * e
    got = f(h, w + e * dirs) - f(h, w - e * dirs)
    assert abs(got - want) <= 0.02 * abs(want)


def test_same_bits_other_stream_and_graph():
    torch, mx = _setup()
    h, w, y = _inputs(torch, 700, 3000, 256, 4, 0.2)
    one = torch.ones(1, device="cuda")
    loss, lse = mx.linear_ce(h, w, y)
    dh, dw = mx.linear_ce_grad(h, w, y, lse, one)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, None):
        loss2, lse2 = mx.linear_ce(h, w, y, stream=stream)
        dh2, dw2 = mx.linear_ce_grad(h, w, y, lse2, one, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(dh, dh2) and torch.equal(dw, dw2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss3, lse3 = mx.linear_ce(h, w, y)
        dh3, dw3 = mx.linear_ce_grad(h, w, y, lse3, one)
    y.copy_(torch.where(y < 0, torch.zeros_like(y), torch.where(y % 3 == 0, torch.full_like(y, -100), y)))
    h.nan_to_num_(0.5, 0.5, 0.5)
    graph.replay()
    torch.cuda.synchronize()
    loss, lse = mx.linear_ce(h, w, y)
    dh, dw = mx.linear_ce_grad(h, w, y, lse, one)
    assert torch.equal(loss, loss3) and torch.equal(lse, lse3) and torch.equal(dh, dh3) and torch.equal(dw, dw3)
    assert mx.device_status() == 0


@pytest.mark.parametrize("T", [5, 100, 200, 256])
def test_few_tokens_with_unaligned_rows(T):
    """Up to 256 tokens the loss reads h where it lies, if its rows are aligned; up to 128 the gradient keeps
    more of dz.  Rows of an odd pitch must give what aligned ones give."""
    torch, mx = _setup()
    h, w, y = _inputs(torch, T, 999, 72, T, 0.4, pitch_h=73)
    ha = h.contiguous()
    one = torch.ones(1, device="cuda")
    ref = _reference(torch, h, w, y)
    lse = _check_forward(torch, mx, h, w, y, ref)
    assert torch.equal(lse, mx.linear_ce(ha, w, y)[1])
    for a, b in zip(mx.linear_ce_grad(h, w, y, lse, one), mx.linear_ce_grad(ha, w, y, lse, one)):
        assert torch.equal(a, b)
    _check_grad(torch, mx, h, w, y, lse, ref, mx.REDUCE_NONE, mx.OUT_F32)


@pytest.mark.parametrize("T", [1, 3, 128])
def test_few_tokens_keep_more_of_dz(T):
    """At most 128 tokens: dz is held to 2^-16, so fp32 gradients are within that of the formula's, far below a
    bf16 rounding (in the 2-norm; the logits' own error is below 2^-16 here as well)."""
    torch, mx = _setup()
    h, w, y = _inputs(torch, T, 3000, 256, T)
    lse = mx.linear_ce(h, w, y)[1]
    dh, dw = mx.linear_ce_grad(h, w, y, lse, torch.ones(1, device="cuda"), dh_dtype=mx.OUT_F32, dw_dtype=mx.OUT_F32)
    hd, wd = h.double(), w.double()
    dz = torch.softmax(hd @ wd.t(), 1)
    dz[torch.arange(T, device="cuda"), y] -= 1
    dz /= T
    for got, want in ((dh, dz @ wd), (dw, dz.t() @ hd)):
        assert float((got.double() - want).norm()) <= 2.0 ** -14 * float(want.norm())


def test_weights_past_2_31_elements():
    torch, mx = _setup()
    T, V, D = 300, 600_000, 4096
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    w[-512:] = torch.randn(512, D, device="cuda", generator=g) / 64
    h = torch.randn(T, D, device="cuda", generator=g).bfloat16()
    y = torch.randint(V - 512, V, (T,), device="cuda", generator=g)
    z = h.double() @ w[-512:].double().t()
    lse = torch.logsumexp(torch.cat([z, torch.full((T, 1), math.log(V - 512), dtype=torch.float64, device="cuda")], 1), 1)
    want = lse - z.gather(1, y[:, None] - (V - 512))[:, 0]
    loss, got = mx.linear_ce(h, w, y, reduction=mx.REDUCE_NONE)
    tol = 2 * U * D * (h.double().abs() @ w[-512:].double().abs().t()).amax(1) + U * (128 + V / 128 + 200)
    assert bool(((got.double() - lse).abs() <= tol).all()) and bool(((loss.double() - want).abs() <= 2 * tol).all())
    dh, dw = mx.linear_ce_grad(h, w, y, got, torch.ones(1, device="cuda"), reduction=mx.REDUCE_SUM)
    dz = torch.exp(z - lse[:, None])
    dz[torch.arange(T, device="cuda"), y - (V - 512)] -= 1
    for a, b in ((dh, dz @ w[-512:].double()), (dw[-512:], dz.t() @ h.double())):
        assert float((a.double() - b).norm()) <= 2.0 ** -7 * float(b.norm())
    p = torch.exp(-lse)[:, None]  # every other id's probability
    other = (p * h.double()).sum(0)
    for v in (0, 12345, V // 2, V - 513):
        assert float((dw[v].double() - other).norm()) <= 2.0 ** -7 * float(other.norm())
    assert mx.device_status() == 0
