"""The linear cross entropy at the widths of real models, with bounds near what the kernels lose rather than near the
worst case of a sum: confident tokens' gradients, the loss's error in the mean, and few tokens' gradients.

The logits of both passes are the same numbers (summed in the same runs), so what the tensor cores' truncation
takes from a logit (1e-6 of it in a run of K = 512) moves dz only in proportion: z - lse is off by at most 2e-6 of the
row's largest |z|, and the bounds allow twice that.  What is absolute in p = exp(z - lse) is fp32 rounding (u = 2^-24):
lse to fp32 and times log2 e (u |lse| each), the exponential and the sums that lse came from (32u)."""
import pytest

from tests.gpu_util import gpu_ready

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _setup():
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    return torch, mx


def _confident(torch, T, V, D, seed):
    """Logits that share an offset of about 18, with targets some 10 to 18 above the rest: 1 - p from about 1e-1 to 1e-4
    at target logits of 25 to 40."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = torch.randn(V, D, device="cuda", generator=g) * (1.28 / D ** 0.5)
    w = (n + 18.0 / D).bfloat16()
    y = torch.randperm(V, device="cuda", generator=g)[:T]
    h = 1.0 + 0.5 * torch.randn(T, D, device="cuda", generator=g)
    up = (10.0 + 8.0 * torch.rand(T, 1, device="cuda", generator=g)) / 1.28 ** 2
    return (h + up * n[y]).bfloat16(), w, y


@pytest.mark.parametrize("T", [1, 64, 200, 300])
@pytest.mark.parametrize("D", [1032, 4096, 8192])
def test_gradients_of_confident_tokens(T, D):
    """fp32 gradients of the summed loss, element by element.  dz is off by p (2u |lse| + 32u) and by 4e-6 max|z| of
    itself, and its rounding to bf16 is another 2^-8 of itself (few tokens: 2^-16); fp32 sums over n terms
    that the tensor cores cut off add 2u n of their absolute sum."""
    torch, mx = _setup()
    V = 1000
    h, w, y = _confident(torch, T, V, D, T + D)
    _, lse = mx.linear_ce(h, w, y)
    dh, dw = mx.linear_ce_grad(h, w, y, lse, torch.ones(1, device="cuda"), reduction=mx.REDUCE_SUM,
                               dh_dtype=mx.OUT_F32, dw_dtype=mx.OUT_F32)
    assert mx.device_status() == 0
    hd, wd = h.double(), w.double()
    z = hd @ wd.t()
    lse64 = torch.logsumexp(z, 1, keepdim=True)
    p = torch.exp(z - lse64)
    rows = torch.arange(T, device="cuda")
    rest = 1 - p[rows, y]
    assert T == 1 or (float(rest.min()) < 1e-3 and float(z[rows, y].min()) > 20)  # the case that is meant
    dz = p.clone()
    dz[rows, y] = -torch.exp(torch.logsumexp(z.scatter(1, y[:, None], float("-inf")), 1) - lse64[:, 0])
    ed = p * U * (2 * lse64.abs() + 32) + dz.abs() * (4e-6 * z.abs().amax(1, keepdim=True) + (2.0 ** -16 if T <= 128 else 2.0 ** -8))
    for got, want, tol in ((dh, dz @ wd, (ed + 2 * U * V * dz.abs()) @ wd.abs()),
                           (dw, dz.t() @ hd, (ed + 2 * U * T * dz.abs()).t() @ hd.abs())):
        err = (got.double() - want).abs()
        assert bool((err <= tol + 4 * U * want.abs()).all()), float((err / tol).max())


def _ordinary(torch, T, V, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(V, D, device="cuda", generator=g) * (1.28 / D ** 0.5)).bfloat16()
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    h = torch.randn(T, D, device="cuda", generator=g) + 7.3 * torch.rand(T, 1, device="cuda", generator=g) ** 2 * w[y].float()
    return h.bfloat16(), w, y


@pytest.mark.parametrize("T", [256, 1024])
@pytest.mark.parametrize("D", [4096, 8192])
def test_loss_error_in_the_mean(T, D):
    """Logits summed in one run are 4.2e-6 of themselves too small at width 4096, which is a loss off by 1.7e-5 rms; in
    runs of K = 512 it is off by 1.9e-6.  The bound is the geometric mean of the two, 5.7e-6, for the rms, and half
    of it for the signed mean (an error of one sign would have the two alike)."""
    torch, mx = _setup()
    h, w, y = _ordinary(torch, T, 4000, D, D)
    loss, lse = mx.linear_ce(h, w, y, reduction=mx.REDUCE_NONE)
    z = h.double() @ w.double().t()
    want = torch.logsumexp(z, 1)
    for got, ref in ((lse, want), (loss, want - z.gather(1, y[:, None])[:, 0])):
        err = got.double() - ref
        assert float(err.square().mean().sqrt()) <= 5.7e-6, float(err.square().mean().sqrt())
        assert abs(float(err.mean())) <= 2.85e-6, float(err.mean())


@pytest.mark.parametrize("T", [2, 128])
@pytest.mark.parametrize("D", [4096, 8192])
def test_few_tokens_keep_more_of_dz_at_model_widths(T, D):
    """At most 128 tokens hold dz to 2^-16 of itself; the logits (4e-6 max|z|, |z| up to 14) move it by less than 2^-14 and
    lse's rounding by less than 2^-18: in the 2-norm below 2^-13, where rounding to bf16 alone takes about 2^-9."""
    torch, mx = _setup()
    h, w, y = _ordinary(torch, T, 4000, D, T + D)
    lse = mx.linear_ce(h, w, y)[1]
    dh, dw = mx.linear_ce_grad(h, w, y, lse, torch.ones(1, device="cuda"), dh_dtype=mx.OUT_F32, dw_dtype=mx.OUT_F32)
    hd, wd = h.double(), w.double()
    dz = torch.softmax(hd @ wd.t(), 1)
    dz[torch.arange(T, device="cuda"), y] -= 1
    dz /= T
    for got, want in ((dh, dz @ wd), (dw, dz.t() @ hd)):
        assert float((got.double() - want).norm()) <= 2.0 ** -13 * float(want.norm())
