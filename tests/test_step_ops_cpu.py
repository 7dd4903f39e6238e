"""Refusals of the embedding, cross-entropy and clipping entry points that need no GPU: every argument
is checked on the host before the device is touched."""
import array
import ctypes

import pytest

import __graft_entry__
from mxfp4_precision_gemms_gb300 import binding as mx

P = ctypes.c_void_p
INVALID, SHAPE, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return mx.lib()


def _lookup(L, **kw):
    a = dict(ids=0x1000, it=1, n=4, w=0x2000, wt=1, vocab=10, dim=8, ldw=8, scale=1.0, y=0x3000, yt=1, ldy=8)
    a.update(kw)
    return L.mxfp4_embedding(P(a["ids"]), a["it"], a["n"], P(a["w"]), a["wt"], a["vocab"], a["dim"], a["ldw"],
                             a["scale"], P(a["y"]), a["yt"], a["ldy"], None)


@pytest.mark.parametrize("change,want", [
    (dict(it=2), INVALID), (dict(wt=2), INVALID), (dict(yt=-1), INVALID), (dict(n=-1), INVALID),
    (dict(vocab=-1), INVALID), (dict(dim=-1), INVALID), (dict(ids=None), INVALID), (dict(w=None), INVALID),
    (dict(y=None), INVALID), (dict(ldw=7), INVALID), (dict(ldy=7), INVALID), (dict(vocab=0), SHAPE),
    (dict(n=1 << 31), SHAPE), (dict(vocab=(1 << 31) - 1), SHAPE), (dict(dim=(1 << 20) + 1, ldw=1 << 21, ldy=1 << 21), SHAPE),
    (dict(n=(1 << 31) - 1, dim=1 << 20, ldw=1 << 20, ldy=1 << 20), SHAPE), (dict(ids=0x1004), MISALIGNED), (dict(w=0x2001), MISALIGNED), (dict(y=0x3002, yt=0), MISALIGNED),
    (dict(n=0), 0), (dict(dim=0, ldw=0, ldy=0), 0)])
def test_embedding_refuses(L, change, want):
    assert _lookup(L, **change) == want
    assert (L.mxfp4_last_error() == b"") == (want == 0)


def _grad(L, **kw):
    need = L.mxfp4_embedding_grad_workspace_bytes(4, 10, 8)
    a = dict(ids=0x1000, it=0, n=4, dy=0x2000, dyt=1, lddy=8, vocab=10, dim=8, pad=-1, dw=0x3000, dwt=0, lddw=8, acc=0,
             ws=0x4000, wsb=need)
    a.update(kw)
    return L.mxfp4_embedding_grad(P(a["ids"]), a["it"], a["n"], P(a["dy"]), a["dyt"], a["lddy"], a["vocab"], a["dim"],
                                  1.0, a["pad"], P(a["dw"]), a["dwt"], a["lddw"], a["acc"], P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("change,want", [
    (dict(it=5), INVALID), (dict(dyt=2), INVALID), (dict(dwt=2), INVALID), (dict(acc=2), INVALID), (dict(n=-1), INVALID),
    (dict(dw=None), INVALID), (dict(dy=None), INVALID), (dict(ids=None), INVALID), (dict(lddw=7), INVALID),
    (dict(lddy=7), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(ws=0x4010), MISALIGNED),
    (dict(dw=0x3002), MISALIGNED), (dict(ids=0x1002), MISALIGNED), (dict(n=0, acc=1), 0), (dict(vocab=0), 0)])
def test_embedding_grad_refuses(L, change, want):
    assert _grad(L, **change) == want


def test_embedding_grad_workspace(L):
    f = L.mxfp4_embedding_grad_workspace_bytes
    assert f(0, 10, 8) == 0 and f(-1, 10, 8) == 0 and f(4, 10, 1 << 21) == 0
    # two (id, token) arrays, the list of runs, and two fp32 rows for each chunk of 32 tokens
    assert f(8192, 128256, 4096) == 2 * 8192 * 8 + (16 + 256 * 12 + 255) // 256 * 256 + 256 * 2 * 4096 * 4


def _clip(L, entries, n=None, max_norm=1.0, norm=0x5000, ws=0x6000, wsb=None):
    flat = array.array("q", [x for e in entries for x in e])
    wsb = L.mxfp4_clip_grad_norm_workspace_bytes(len(entries)) if wsb is None else wsb
    return L.mxfp4_clip_grad_norm(P(flat.buffer_info()[0]) if entries else None, len(entries) if n is None else n,
                                  max_norm, P(norm), P(ws), wsb, None)


@pytest.mark.parametrize("entry,want", [
    ((0x1000, 0x2000, 8, 2), INVALID), ((0x1000, 0x2000, -1, 0), INVALID), ((0, 0x2000, 8, 0), INVALID),
    ((0x1000, 0, 8, 0), INVALID), ((0x1000, 0x2000, 8, 1 << 32), INVALID), ((0x1002, 0x2000, 8, 0), MISALIGNED),
    ((0x1000, 0x2001, 8, 1), MISALIGNED), ((0x1000, 0x2000, 1 << 45, 0), SHAPE)])
def test_clip_refuses_a_gradient(L, entry, want):
    assert _clip(L, [(0x1000, 0x1000, 8, 0), entry]) == want


@pytest.mark.parametrize("change,want", [
    (dict(n=-1), INVALID), (dict(max_norm=-1.0), INVALID), (dict(max_norm=float("nan")), INVALID),
    (dict(norm=None), INVALID), (dict(norm=0x5002), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(wsb=8), WORKSPACE),
    (dict(ws=0x6008), MISALIGNED), (dict(n=1 << 21), SHAPE)])
def test_clip_refuses(L, change, want):
    assert _clip(L, [(0x1000, 0x1000, 8, 0)], **change) == want


def test_binding_refuses_before_the_library():
    import torch

    ids, w = torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8)
    for call in (lambda: mx.embedding(ids, w), lambda: mx.embedding_grad(ids, torch.zeros(3, 8), 4),
                 lambda: mx.linear_ce(w, w, ids), lambda: mx.linear_ce_grad(w, w, ids, w[:, 0], w[0, :1]),
                 lambda: mx.clip_grad_norm([w], 1.0), lambda: mx.clip_grad_norm([w], 1.0, outs=[])):
        with pytest.raises(ValueError):
            call()


def _ce(L, **kw):
    need = L.mxfp4_linear_ce_workspace_bytes(4, 100, 64)
    a = dict(h=0x1000, n=4, dim=64, ldh=64, w=0x2000, vocab=100, ldw=64, y=0x3000, it=1, red=2, loss=0x4000, lse=0x5000,
             ws=0x6000, wsb=need)
    a.update(kw)
    return L.mxfp4_linear_ce(P(a["h"]), a["n"], a["dim"], a["ldh"], P(a["w"]), a["vocab"], a["ldw"], P(a["y"]), a["it"],
                             -100, a["red"], P(a["loss"]), P(a["lse"]), P(a["ws"]), a["wsb"], None)


CE_BAD = [(dict(h=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(it=2), INVALID),
          (dict(red=3), INVALID), (dict(red=-1), INVALID), (dict(n=-1), INVALID), (dict(vocab=-1), INVALID),
          (dict(dim=-8), INVALID), (dict(vocab=0), SHAPE), (dict(dim=0), SHAPE), (dict(dim=60), SHAPE),
          (dict(n=(1 << 24) + 1), SHAPE), (dict(vocab=(1 << 28) + 1), SHAPE), (dict(n=1 << 24, vocab=1 << 28), SHAPE), (dict(ldh=63), INVALID),
          (dict(ldw=56), INVALID), (dict(ldw=68), MISALIGNED), (dict(w=0x2008), MISALIGNED), (dict(h=0x1001), MISALIGNED),
          (dict(y=0x3004), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(wsb=64), WORKSPACE),
          (dict(ws=0x6010), MISALIGNED)]


@pytest.mark.parametrize("change,want", CE_BAD + [(dict(loss=None), INVALID), (dict(lse=None), INVALID),
                                                  (dict(loss=0x4002), MISALIGNED), (dict(n=0, red=0), 0)])
def test_linear_ce_refuses(L, change, want):
    assert _ce(L, **change) == want


def _ce_grad(L, **kw):
    need = L.mxfp4_linear_ce_grad_workspace_bytes(4, 100, 64)
    a = dict(h=0x1000, n=4, dim=64, ldh=64, w=0x2000, vocab=100, ldw=64, y=0x3000, it=1, red=2, lse=0x5000, g=0x4000,
             dh=0x7000, ht=1, lddh=64, dw=0x8000, wt=0, lddw=64, acc=0, ws=0x6000, wsb=need)
    a.update(kw)
    return L.mxfp4_linear_ce_grad(P(a["h"]), a["n"], a["dim"], a["ldh"], P(a["w"]), a["vocab"], a["ldw"], P(a["y"]),
                                  a["it"], -100, a["red"], P(a["lse"]), P(a["g"]), P(a["dh"]), a["ht"], a["lddh"],
                                  P(a["dw"]), a["wt"], a["lddw"], a["acc"], P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("change,want", CE_BAD + [
    (dict(lse=None), INVALID), (dict(g=None), INVALID), (dict(ht=2), INVALID), (dict(wt=2), INVALID),
    (dict(acc=2), INVALID), (dict(acc=1, wt=1), INVALID), (dict(lddh=63), INVALID), (dict(lddw=63), INVALID),
    (dict(lddw=66), MISALIGNED), (dict(dw=0x8008), MISALIGNED), (dict(dh=0x7001), MISALIGNED),
    (dict(lse=0x5002), MISALIGNED), (dict(dh=None, dw=None), 0), (dict(n=0, acc=1), 0), (dict(n=0, dw=None), 0)])
def test_linear_ce_grad_refuses(L, change, want):
    assert _ce_grad(L, **change) == want


def test_linear_ce_workspace_holds_no_logits(L):
    """At 8192 x 128256 x 4096 the logits would be 4.2 GB in fp32; one piece of dz is at most 512 MiB."""
    T, V, D = 8192, 128256, 4096
    assert L.mxfp4_linear_ce_workspace_bytes(T, V, D) < 2 * T * D + 8 * T * (2 * 501) + (1 << 20)
    assert L.mxfp4_linear_ce_grad_workspace_bytes(T, V, D) < (512 << 20) + 6 * T * D + (1 << 20)
    assert L.mxfp4_linear_ce_workspace_bytes(0, V, D) == 0 and L.mxfp4_linear_ce_grad_workspace_bytes(T, -1, D) == 0
