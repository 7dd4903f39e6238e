"""Embedding lookup and its gradient (mxfp4_embedding, mxfp4_embedding_grad) against the formulas in
64 bits.  Tolerances: the lookup is one fp32 product and one rounding; the gradient's sum of n
terms in fp32 is off by at most n * 2^-24 * sum|terms| (each addition rounds by 2^-24 of a partial
sum, which the terms' absolute sum bounds; scaling and the addition to dw are two more), and a
bf16 output adds 2^-8 of the result (half an ulp is 2^-9 of the value's binade)."""
import pytest

from tests.gpu_util import gpu_ready

pytestmark = pytest.mark.gpu


def _setup():
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    return torch, mx, {mx.OUT_F32: torch.float32, mx.OUT_BF16: torch.bfloat16}


def _rows(torch, n, dim, pitch, dtype, seed, std=1.0):
    """[n, dim] with `pitch` elements between rows; what lies between rows is NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = torch.full((n, pitch), float("nan"), dtype=dtype, device="cuda")
    full[:, :dim] = torch.randn(n, dim, device="cuda", generator=g) * std
    return full[:, :dim]


@pytest.mark.parametrize("wt,yt", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("tokens,vocab,dim,pitch", [(1, 1, 1, 1), (7, 50, 8, 8), (33, 1000, 129, 131),
                                                    (1000, 777, 264, 272), (300, 100, 4096, 4096),
                                                    (5, 9, 1000, 1001)])
def test_lookup(wt, yt, tokens, vocab, dim, pitch):
    torch, mx, dt = _setup()
    w = _rows(torch, vocab, dim, pitch, dt[wt], 1)
    for ids_t in (torch.int32, torch.int64):
        ids = torch.randint(0, vocab, (tokens,), device="cuda", dtype=ids_t)
        y = mx.embedding(ids, w, scale=0.37, out_dtype=yt)
        want = (w.double()[ids.long()] * 0.37)
        tol = 2.0 ** -22 * want.abs() + (2.0 ** -8 * want.abs() if yt == mx.OUT_BF16 else 0)
        assert bool(((y.double() - want).abs() <= tol).all())
        assert mx.device_status() == 0
    same = mx.embedding(ids, w, out_dtype=wt)  # scale 1, same type: a copy
    assert torch.equal(same, w[ids.long()])


def test_lookup_shapes_and_pitched_output():
    torch, mx, _ = _setup()
    w = _rows(torch, 40, 24, 24, torch.bfloat16, 3)
    ids = torch.randint(0, 40, (2, 3, 5), device="cuda")
    assert torch.equal(mx.embedding(ids, w), w[ids])
    out = torch.zeros(30, 40, dtype=torch.bfloat16, device="cuda")
    mx.embedding(ids, w, out=out[:, 8:32])
    assert torch.equal(out[:, 8:32], w[ids.reshape(-1)]) and not out[:, :8].any() and not out[:, 32:].any()
    assert mx.embedding(ids[:0], w).shape == (0, 3, 5, 24)
    # values pass through the product: infinities, NaN, signed zero
    w2 = torch.tensor([[float("inf"), float("-inf"), float("nan"), -0.0]], device="cuda")
    y = mx.embedding(torch.zeros(1, dtype=torch.int64, device="cuda"), w2, scale=2.0)
    assert torch.equal(y[0, :2], w2[0, :2]) and bool(y[0, 2].isnan()) and bool(torch.signbit(y[0, 3]))


def test_bad_ids_are_reported():
    torch, mx, _ = _setup()
    w = _rows(torch, 10, 16, 16, torch.float32, 4)
    ids = torch.tensor([3, 10, -1, 9], device="cuda")
    y = mx.embedding(ids, w)
    assert mx.device_status() == 1 and b"vocabulary" in mx.lib().mxfp4_last_error()
    assert torch.equal(y[0], w[3]) and torch.equal(y[3], w[9]) and not y[1:3].any()
    dy = _rows(torch, 4, 16, 16, torch.float32, 5)
    dw = mx.embedding_grad(ids, dy, 10)
    assert mx.device_status() == 1
    want = torch.zeros(10, 16, device="cuda")
    want[3], want[9] = dy[0], dy[3]
    assert torch.equal(dw, want)
    assert mx.device_status() == 0


def _ids(torch, kind, tokens, vocab, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "same":
        return torch.full((tokens,), vocab // 2, device="cuda")
    if kind == "distinct":
        return torch.randperm(vocab, device="cuda", generator=g)[:tokens]
    if kind == "few":
        return torch.randint(0, min(3, vocab), (tokens,), device="cuda", generator=g)
    u = torch.rand(tokens, device="cuda", generator=g, dtype=torch.float64)
    return ((vocab + 1.0) ** u - 1).long().clamp_(0, vocab - 1)


def _check_grad(torch, mx, dt, ids, dy, vocab, scale, padding, out, accumulate, pitch=None):
    dim = dy.shape[1]
    dw0 = _rows(torch, vocab, dim, pitch or dim, dt[out], 11) if accumulate or pitch else None
    start = dw0.double().clone() if accumulate else torch.zeros(vocab, dim, dtype=torch.float64, device="cuda")
    got = mx.embedding_grad(ids, dy, vocab, scale=scale, padding_id=padding, out_dtype=out, accumulate=accumulate,
                            dw=dw0)
    assert mx.device_status() == 0
    keep = (ids != padding).nonzero()[:, 0]
    add = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda")
    size = add.clone()
    add.index_put_((ids[keep].long(),), dy.double()[keep] * scale, accumulate=True)
    size.index_put_((ids[keep].long(),), dy.double()[keep].abs() * abs(scale), accumulate=True)
    n = torch.bincount(ids[keep].long(), minlength=vocab).double()[:, None]
    want = start + add
    tol = (n + 4) * 2.0 ** -24 * (size + start.abs()) + (2.0 ** -8 * want.abs() if out == mx.OUT_BF16 else 0)
    bad = ((got.double() - want).abs() > tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())
    if accumulate:  # rows that do not occur are not touched
        assert torch.equal(got[(n == 0)[:, 0]], start[(n == 0)[:, 0]].to(got.dtype))


@pytest.mark.parametrize("kind", ["same", "distinct", "few", "zipf"])
@pytest.mark.parametrize("tokens,vocab,dim", [(1, 5, 8), (31, 40, 16), (32, 33, 129), (65, 511, 1024),
                                              (511, 600, 136), (512, 600, 1032), (513, 600, 136), (545, 600, 33), (1000, 1200, 1032),
                                              (2048, 2500, 16), (2049, 2500, 40), (4097, 5000, 64), (9000, 128256, 72)])
def test_gradient(kind, tokens, vocab, dim):
    torch, mx, dt = _setup()
    ids = _ids(torch, kind, tokens, vocab, tokens)
    dy = _rows(torch, tokens, dim, dim, torch.bfloat16, 7)
    for out in (mx.OUT_F32, mx.OUT_BF16):
        for accumulate in (False, True):
            _check_grad(torch, mx, dt, ids, dy, vocab, 1.7, -1, out, accumulate)


@pytest.mark.parametrize("vocab", [1, 2, 510, 511, 512, 513, 262142, 262143, 262144])
def test_gradient_at_the_sort_digit_borders(vocab):
    """Vocabularies around 2^9 and 2^18, where a pass of the sort is added."""
    torch, mx, dt = _setup()
    ids = _ids(torch, "zipf", 700, vocab, 3)
    ids[::7] = vocab - 1
    dy = _rows(torch, 700, 8, 8, torch.float32, 8)
    _check_grad(torch, mx, dt, ids, dy, vocab, 1.0, vocab - 1, mx.OUT_F32, False)
    _check_grad(torch, mx, dt, ids.int(), dy, vocab, 1.0, -1, mx.OUT_F32, True)


@pytest.mark.parametrize("dyt", [0, 1])
def test_gradient_pitched_and_padding(dyt):
    """Row pitches, aligned and not; padding rows hold NaN and must not be read."""
    torch, mx, dt = _setup()
    for dim, pitch in ((100, 101), (104, 112), (13, 13)):
        ids = _ids(torch, "zipf", 500, 300, 9)
        dy = _rows(torch, 500, dim, pitch, dt[dyt], 10)
        padding = int(ids[0])
        dy[ids == padding] = float("nan")
        keep = ids != padding
        clean = torch.where(keep[:, None], dy, torch.zeros_like(dy))
        for out in (mx.OUT_F32, mx.OUT_BF16):
            got = mx.embedding_grad(ids, dy, 300, padding_id=padding, out_dtype=out)
            assert torch.equal(got, mx.embedding_grad(ids, clean, 300, padding_id=padding, out_dtype=out))
            _check_grad(torch, mx, dt, ids, clean, 300, -0.5, padding, out, True, pitch)
            full = torch.full((300, pitch + 3), 7.0, dtype=dt[out], device="cuda")
            mx.embedding_grad(ids, clean, 300, padding_id=padding, out_dtype=out, dw=full[:, :dim])
            assert torch.equal(full[:, :dim], got) and bool((full[:, dim:] == 7.0).all())


@pytest.mark.parametrize("tokens", [200, 700])
def test_padding_outside_the_vocabulary_and_bad_ids(tokens):
    """Few tokens and many take different kernels: both leave out padding and bad ids, and report the latter.
    (The tolerance of a sum of n terms, as above: which terms are added first depends on all ids.)"""
    torch, mx, _ = _setup()
    ids = torch.arange(tokens, device="cuda") % 50
    dy = _rows(torch, tokens, 24, 24, torch.float32, 3)
    keep = (ids != 4).nonzero()[:, 0]
    want = torch.zeros(50, 24, dtype=torch.float64, device="cuda").index_put_((ids[keep],), dy.double()[keep], accumulate=True)
    size = torch.zeros(50, 24, dtype=torch.float64, device="cuda").index_put_((ids[keep],), dy.double()[keep].abs(), accumulate=True)
    tol = (tokens // 50 + 4) * 2.0 ** -24 * size
    got = mx.embedding_grad(torch.where(ids == 4, torch.full_like(ids, 70), ids), dy, 50, padding_id=70)
    assert mx.device_status() == 0 and bool(((got.double() - want).abs() <= tol).all())
    for bad in (50, -1, -2, 1 << 40):
        got = mx.embedding_grad(torch.where(ids == 4, torch.full_like(ids, bad), ids), dy, 50, padding_id=-1)
        assert mx.device_status() == 1 and bool(((got.double() - want).abs() <= tol).all())


def test_gradient_without_tokens_and_all_padding():
    torch, mx, _ = _setup()
    for dim in (8, 9):
        dw = torch.ones(50, dim, device="cuda")
        none = torch.empty(0, dtype=torch.int64, device="cuda")
        mx.embedding_grad(none, torch.empty(0, dim, device="cuda"), 50, dw=dw, accumulate=True)
        assert bool((dw == 1).all())
        mx.embedding_grad(none, torch.empty(0, dim, device="cuda"), 50, dw=dw)
        assert not dw.any()
        ids = torch.full((100,), 4, device="cuda")
        got = mx.embedding_grad(ids, torch.full((100, dim), float("nan"), device="cuda"), 50, padding_id=4)
        assert not got.any()


def test_gradient_is_the_same_every_time():
    torch, mx, _ = _setup()
    ids = _ids(torch, "zipf", 20000, 3000, 1)
    dy = _rows(torch, 20000, 136, 136, torch.bfloat16, 2)
    first = mx.embedding_grad(ids, dy, 3000, out_dtype=mx.OUT_F32)
    for _ in range(5):
        assert torch.equal(mx.embedding_grad(ids, dy, 3000, out_dtype=mx.OUT_F32), first)


def test_gradient_against_differences():
    """d(sum(y * r))/dw by central differences of the lookup in fp32 (linear in w: exact to rounding)."""
    torch, mx, _ = _setup()
    w = _rows(torch, 20, 8, 8, torch.float32, 5)
    ids = torch.tensor([3, 3, 7, 0, 3, 19], device="cuda")
    r = _rows(torch, 6, 8, 8, torch.float32, 6)
    dw = mx.embedding_grad(ids, r, 20, scale=1.5)
    for v, c in ((3, 0), (7, 5), (0, 7), (1, 1), (19, 2)):
        step = torch.zeros_like(w)
        step[v, c] = 0.5
        f = lambda x: float((mx.embedding(ids, x, scale=1.5).double() * r.double()).sum())  # noqa: E731
        # each lookup rounds its 6 rows by 2^-24 of values below 8, times |r| below 8
        assert abs(f(w + step) - f(w - step) - float(dw[v, c])) < 6 * 2 * 8 * 8 * 2.0 ** -23


def test_other_stream_and_graph():
    torch, mx, _ = _setup()
    ids = _ids(torch, "zipf", 3000, 2000, 1)
    w = _rows(torch, 2000, 256, 256, torch.bfloat16, 2)
    dy = _rows(torch, 3000, 256, 256, torch.bfloat16, 3)
    y0, g0 = mx.embedding(ids, w), mx.embedding_grad(ids, dy, 2000)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y1, g1 = mx.embedding(ids, w, stream=side), mx.embedding_grad(ids, dy, 2000, stream=side)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(g0, g1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, g2 = mx.embedding(ids, w), mx.embedding_grad(ids, dy, 2000)
    ids.copy_(ids.flip(0))
    dy.copy_(dy.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y0.flip(0)) and torch.equal(g2, mx.embedding_grad(ids, dy, 2000))
    assert torch.equal(g2, mx.embedding_grad(ids, dy, 2000)) and mx.device_status() == 0


def test_rows_past_2_31_elements():
    torch, mx, _ = _setup()
    V, D = 600_000, 4096  # 2.46e9 elements
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(3, D, device="cuda").bfloat16()
    w[V - 3:] = last
    ids = torch.tensor([V - 1, 0, V - 3, V - 2], device="cuda")
    y = mx.embedding(ids, w)
    assert torch.equal(y, torch.stack([last[2], w[0], last[0], last[1]]))
    for many in (1, 200):  # few tokens, and enough for the sort
        dw = mx.embedding_grad(ids.repeat(many), y.repeat(many, 1), V, dw=w, accumulate=True)
        assert not dw[1:V - 3].any()
        w[V - 3:] = last
    full = torch.full((V, D), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.embedding_grad(ids.repeat(200), y.repeat(200, 1), V, dw=full)
    assert not full[:V - 3].any() and bool(((full[V - 1].float() - 200 * last[2].float()).abs() <= 2.0 ** -7 * 200 * last[2].float().abs()).all())
    assert mx.device_status() == 0


def test_output_past_2_31_elements():
    torch, mx, _ = _setup()
    w = torch.randn(1000, 4096, device="cuda").bfloat16()
    ids = torch.arange(600_000, device="cuda") % 1000
    y = mx.embedding(ids, w)
    assert torch.equal(y[-1000:], w) and torch.equal(y[299_000:300_000], w)
    # and their gradient: 600 rows of each id, the same every time
    dw = mx.embedding_grad(ids, y, 1000, out_dtype=mx.OUT_F32)
    assert bool(((dw - 600 * w.float()).abs() <= 604 * 2.0 ** -24 * 600 * w.float().abs()).all())
