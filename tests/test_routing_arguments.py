"""Argument errors of routing, dispatch, combining and the loss over a head matrix, returned on the host before any CUDA call."""

import ctypes

import pytest

import muon_newton_schulz_expert_gb300 as mk
from muon_newton_schulz_expert_gb300 import build as mkbuild

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    mkbuild.build()
    return mk.lib()


def test_route(lib):
    def call(logits=P(256), stride=64, bias=None, rows=4, experts=64, type_=1, top=8, score=0, norm=1, scale=1.0,
             ids=P(256), weights=P(256)):
        return lib.muon_route(logits, stride, bias, rows, experts, type_, top, score, norm, scale, ids, weights, None)

    for bad in (dict(rows=-1), dict(experts=0), dict(type_=2), dict(score=2), dict(score=-1), dict(top=0),
                dict(top=65), dict(stride=63), dict(scale=float("nan")), dict(logits=None), dict(ids=None),
                dict(weights=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(top=33), dict(experts=1025, stride=1025), dict(rows=1 << 28), dict(logits=P(258)),
                dict(ids=P(260)), dict(bias=P(2)), dict(weights=P(2))):
        assert call(**bad) == -2, bad
    assert call(rows=0, logits=None, ids=None, weights=None) == 0


def test_route_backward(lib):
    def call(dw=P(256), logits=P(256), stride=64, ids=P(256), rows=4, experts=64, type_=1, top=8, score=0, norm=1,
             scale=1.0, out=P(256), out_stride=64):
        return lib.muon_route_backward(dw, logits, stride, ids, rows, experts, type_, top, score, norm, scale, out,
                                       out_stride, None)

    for bad in (dict(rows=-1), dict(experts=0), dict(type_=-1), dict(score=7), dict(top=0), dict(top=65),
                dict(stride=1), dict(out_stride=63), dict(scale=float("inf")), dict(dw=None), dict(logits=None),
                dict(ids=None), dict(out=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(top=33), dict(experts=2000, stride=2000, out_stride=2000), dict(out=P(2)), dict(dw=P(2)),
                dict(ids=P(4))):
        assert call(**bad) == -2, bad
    assert call(rows=0, dw=None, logits=None) == 0


def test_dispatch(lib):
    def call(x=P(256), xs=64, ids=P(256), tokens=4, top=2, experts=8, hidden=64, type_=0, rows=P(256), off=P(256),
             place=P(256)):
        return lib.muon_dispatch(x, xs, ids, tokens, top, experts, hidden, type_, rows, off, place, None)

    for bad in (dict(tokens=-1), dict(top=0), dict(experts=0), dict(hidden=0), dict(type_=3), dict(x=None),
                dict(ids=None), dict(rows=None), dict(off=None), dict(place=None), dict(xs=63)):
        assert call(**bad) == -1, bad
    for bad in (dict(top=33), dict(experts=1025), dict(hidden=1 << 21, xs=1 << 21), dict(tokens=1 << 30), dict(x=P(257)),
                dict(rows=P(257)), dict(ids=P(260)), dict(off=P(4)), dict(place=P(4)), dict(type_=1, x=P(258))):
        assert call(**bad) == -2, bad


def test_combine_and_the_gradients(lib):
    def combine(y=P(256), place=P(256), w=P(256), tokens=4, top=2, hidden=64, type_=0, out=P(256), os=64):
        return lib.muon_combine(y, place, w, tokens, top, hidden, type_, out, os, None)

    def dispatch_backward(d=P(256), place=P(256), tokens=4, top=2, hidden=64, type_=0, out=P(256), os=64):
        return lib.muon_dispatch_backward(d, place, tokens, top, hidden, type_, out, os, None)

    def backward(d=P(256), ds=64, y=P(256), place=P(256), w=P(256), tokens=4, top=2, hidden=64, type_=0, dy=P(256),
                 dw=P(256)):
        return lib.muon_combine_backward(d, ds, y, place, w, tokens, top, hidden, type_, dy, dw, None)

    for f in (combine, dispatch_backward, backward):
        for bad in (dict(tokens=-1), dict(top=0), dict(hidden=0), dict(type_=2), dict(place=None)):
            assert f(**bad) == -1, (f, bad)
        for bad in (dict(top=33), dict(tokens=1 << 30), dict(place=P(12))):
            assert f(**bad) == -2, (f, bad)
        assert f(tokens=0, place=None) == 0
    for bad in (dict(y=None), dict(out=None), dict(os=63)):
        assert combine(**bad) == -1, bad
    for bad in (dict(y=P(1)), dict(w=P(2)), dict(out=P(3))):
        assert combine(**bad) == -2, bad
    for bad in (dict(d=None), dict(ds=1), dict(y=None), dict(dy=None, dw=None)):
        assert backward(**bad) == -1, bad
    for bad in (dict(d=P(1)), dict(dy=P(1)), dict(dw=P(2)), dict(w=P(2))):
        assert backward(**bad) == -2, bad


def test_head_loss(lib):
    def call(x=P(256), xs=64, w=P(256), t=P(256), rows=4, vocab=100, hidden=64, loss=P(256), lse=P(256), ws=P(256),
             wsb=0):
        return lib.muon_head_loss(x, xs, w, t, rows, vocab, hidden, loss, lse, ws, wsb, None)

    for bad in (dict(rows=-1), dict(vocab=0), dict(hidden=0), dict(x=None), dict(w=None), dict(t=None),
                dict(loss=None, lse=None), dict(xs=56), dict(ws=P(256 + 16))):
        assert call(**bad) == -1, bad
    for bad in (dict(hidden=60), dict(xs=68), dict(x=P(264)), dict(w=P(8)), dict(t=P(4)), dict(loss=P(2)),
                dict(lse=P(2)), dict(rows=1 << 25), dict(vocab=1 << 31), dict(hidden=1 << 21, xs=1 << 21)):
        assert call(**bad) == -2, bad
    assert call(wsb=16) == -4
    assert call(rows=0, x=None, t=None) == 0


def test_head_loss_backward(lib):
    def call(dl=P(256), dz=None, x=P(256), xs=64, w=P(256), t=P(256), lse=P(256), rows=4, vocab=100, hidden=64,
             dx=P(256), dxs=64, dw=P(256), ws=P(256), wsb=0):
        return lib.muon_head_loss_backward(dl, dz, x, xs, w, t, lse, rows, vocab, hidden, dx, dxs, dw, ws, wsb, None)

    for bad in (dict(rows=-1), dict(vocab=0), dict(hidden=0), dict(dl=None), dict(x=None), dict(w=None), dict(t=None),
                dict(lse=None), dict(dx=None, dw=None), dict(xs=8), dict(dxs=8), dict(ws=P(8))):
        assert call(**bad) == -1, bad
    for bad in (dict(hidden=60), dict(xs=68), dict(dxs=68), dict(x=P(264)), dict(w=P(8)), dict(dw=P(8)), dict(dx=P(8)),
                dict(t=P(4)), dict(dl=P(2)), dict(dz=P(2)), dict(lse=P(2))):
        assert call(**bad) == -2, bad
    assert call(wsb=1000) == -4
    assert call(rows=0, dl=None, dw=None) == 0


def test_workspace_sizes(lib):
    f, b = lib.muon_head_loss_workspace_bytes, lib.muon_head_loss_backward_workspace_bytes
    assert f(100, 5000, 64) >= 100 * 8
    assert b(100, 5000, 64) >= 100 * 5000 * 2              # small: one piece
    # the logits of a piece only
    assert b(4096, 128000, 6144) < 4096 * 128000 * 2 // 2
    for bad in ((0, 10, 64), (1, 0, 64), (1, 10, 60), (1, 10, 0), (1 << 25, 10, 64)):
        assert f(*bad) == 0 and b(*bad) == 0, bad


def test_names_of_the_choices():
    for bad in ("tanh", None, 0):
        with pytest.raises(ValueError, match="score must be one of"):
            mk.muon_route(None, 1, score=bad)
        with pytest.raises(ValueError, match="score must be one of"):
            mk.muon_route_backward(None, None, None, score=bad)


def test_cpu_tensors_are_refused(lib):
    torch = pytest.importorskip("torch")
    x, ids = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int64)
    ops = mk._ops()
    where = (0, 0, True)
    for call in (lambda: ops.route(x, 2, None, 0, True, 1.0, where),
                 lambda: ops.route_backward(x[:, :2], x, ids, 0, True, 1.0, None, where),
                 lambda: ops.dispatch(x, ids, 8, None, where),
                 lambda: ops.dispatch_backward(x, ids, None, where),
                 lambda: ops.combine(x, ids, None, None, where),
                 lambda: ops.combine_backward(x, x, ids, None, None, True, True, where),
                 lambda: ops.head_loss(x, x, ids, None, where),
                 lambda: ops.head_loss_backward(x, x, x, ids, x, None, None, None, True, True, None, where)):
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            call()
        with pytest.raises(TypeError, match="expected"):
            ops.route(x)
