"""The autograd forms' forward and backward pass captured into a graph and replayed on other numbers, and on another stream."""
import pytest

from tests.gpu_util import gpu_ready
from tests.test_attention_gpu import _edges, _inputs

pytestmark = pytest.mark.gpu


def _pass(torch, leaves, dy, rope, pos, cu):
    from mxfp4_precision_gemms_gb300.attention import attention, qk_norm_rope

    q, k, v, qg, kg = leaves
    a, b = qk_norm_rope(q, k, rope, pos, qg, kg)
    y = attention(a, b, v, cu_q=cu)
    return [y.detach(), *torch.autograd.grad(y, leaves, dy)]


def _case(torch, seed):
    lens = [130, 1, 77]
    q, k, v, dy = _inputs(torch, lens, lens, 4, 2, 64, 0, seed)
    gains = [0.5 + torch.rand(64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed + i)) for i in (1, 2)]
    return [q, k, v, *gains], dy


def test_captured_and_replayed():
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    rope, pos, cu = mx.Rope([0.8 ** i for i in range(32)]), torch.arange(208, device="cuda"), _edges(torch, [130, 1, 77])
    cases = [_case(torch, s) for s in (1, 5)]
    want = [_pass(torch, [x.clone().requires_grad_() for x in leaves], dy, rope, pos, cu) for leaves, dy in cases]
    place = [torch.empty_like(x).requires_grad_() for x in cases[0][0]]
    dy = torch.empty_like(cases[0][1])

    def fill(i):
        with torch.no_grad():
            for to, x in zip([*place, dy], [*cases[i][0], cases[i][1]]):
                to.copy_(x)

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _pass(torch, place, dy, rope, pos, cu)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _pass(torch, place, dy, rope, pos, cu)
    for i in (1, 0, 1):
        fill(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
    assert mx.device_status() == 0


def test_on_streams_of_their_own():
    torch = gpu_ready()
    from mxfp4_precision_gemms_gb300 import binding as mx

    rope, pos, cu = mx.Rope([0.8 ** i for i in range(32)]), torch.arange(208, device="cuda"), _edges(torch, [130, 1, 77])
    cases = [_case(torch, s) for s in (1, 5)]
    run = lambda i: _pass(torch, [x.clone().requires_grad_() for x in cases[i][0]], cases[i][1], rope, pos, cu)
    want = [run(i) for i in (0, 1)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, run(i)))
    torch.cuda.synchronize()
    for i, g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
    assert mx.device_status() == 0
