"""Argument errors of the operators around the step, returned on the host before any CUDA call."""

import ctypes
import re

import pytest

import muon_newton_schulz_expert_gb300 as mk
from muon_newton_schulz_expert_gb300 import build as mkbuild

P = ctypes.c_void_p


class NormArgs(ctypes.Structure):
    """muon_block_norm_args"""
    _fields_ = [("rows", ctypes.c_int64), ("hidden", ctypes.c_int64), ("residual_type", ctypes.c_int),
                ("branch_type", ctypes.c_int), ("residual", P), ("residual_stride", ctypes.c_int64), ("block", P),
                ("block_stride", ctypes.c_int64), ("w_post", P), ("gate", P), ("gate_stride", ctypes.c_int64),
                ("w_pre", P), ("scale", ctypes.c_float), ("eps", ctypes.c_float), ("residual_out", P),
                ("residual_out_stride", ctypes.c_int64), ("normed", P), ("normed_stride", ctypes.c_int64),
                ("rstd_post", P), ("rstd_pre", P)]


class NormBackwardArgs(ctypes.Structure):
    """muon_block_norm_backward_args"""
    _fields_ = [("rows", ctypes.c_int64), ("hidden", ctypes.c_int64), ("residual_type", ctypes.c_int),
                ("branch_type", ctypes.c_int), ("dresidual_out", P), ("dresidual_out_stride", ctypes.c_int64),
                ("dnormed", P), ("dnormed_stride", ctypes.c_int64), ("residual", P),
                ("residual_stride", ctypes.c_int64), ("block", P), ("block_stride", ctypes.c_int64), ("w_post", P),
                ("gate", P), ("gate_stride", ctypes.c_int64), ("w_pre", P), ("rstd_post", P), ("rstd_pre", P),
                ("scale", ctypes.c_float), ("dresidual", P), ("dresidual_stride", ctypes.c_int64), ("dblock", P),
                ("dblock_stride", ctypes.c_int64), ("dw_post", P), ("dgate", P), ("dgate_stride", ctypes.c_int64),
                ("dw_pre", P)]


def header_fields(name):
    """The fields of a struct of the header, in order."""
    src = re.sub(r"/\*.*?\*/", "", open(mkbuild.INCLUDE + "/muon.h").read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, src).group(1)
    return [re.sub(r".*[ *]", "", f.strip()) for d in body.split(";") for f in d.split(",") if f.strip()]


def test_structs_follow_the_header():
    assert header_fields("muon_block_norm_args") == [n for n, _ in NormArgs._fields_]
    assert header_fields("muon_block_norm_backward_args") == [n for n, _ in NormBackwardArgs._fields_]


@pytest.fixture(scope="module")
def lib():
    mkbuild.build()
    return mk.lib()


def ffn(lib, x=P(256), xs=64, w=P(256), off=P(256), rows=4, experts=2, hidden=64, ffn_=72, act=0, y=P(256), ys=64,
        gate=None, up=None, ws=P(256), wsb=0):
    return lib.muon_gated_ffn(x, xs, w, w, w, off, rows, experts, hidden, ffn_, act, y, ys, gate, up, ws, wsb, None)


def test_gated_ffn(lib):
    for bad in (dict(rows=-1), dict(experts=0), dict(hidden=0), dict(ffn_=0), dict(act=2), dict(off=None),
                dict(x=None), dict(w=None), dict(y=None), dict(gate=P(256)), dict(up=P(256)), dict(xs=56),
                dict(ys=56), dict(ws=P(256 + 16))):
        assert ffn(lib, **bad) == -1, bad
    for bad in (dict(hidden=60, xs=64), dict(ffn_=4), dict(xs=68), dict(ys=65), dict(x=P(264)), dict(y=P(258)),
                dict(w=P(8)), dict(rows=1 << 31), dict(experts=1 << 17), dict(gate=P(264), up=P(256))):
        assert ffn(lib, **bad) == -2, bad
    assert ffn(lib, wsb=10) == -4
    assert ffn(lib, rows=0, x=None, y=None) == 0


def test_gated_ffn_backward(lib):
    def call(dy=P(256), dys=64, x=P(256), xs=64, gate=P(256), up=P(256), w=P(256), off=P(256), rows=4, experts=2,
             hidden=64, ffn_=72, act=0, dx=P(256), dxs=64, dw1=P(256), dw3=P(256), dw2=P(256), ws=P(256), wsb=0):
        return lib.muon_gated_ffn_backward(dy, dys, x, xs, gate, up, w, w, w, off, rows, experts, hidden, ffn_, act,
                                           dx, dxs, dw1, dw3, dw2, ws, wsb, None)

    for bad in (dict(rows=-1), dict(act=-1), dict(dy=None), dict(x=None), dict(gate=None), dict(up=None),
                dict(w=None), dict(dw1=None), dict(dw2=None), dict(dx=None, dw1=None, dw3=None, dw2=None),
                dict(dys=8), dict(dxs=8), dict(ws=P(8))):
        assert call(**bad) == -1, bad
    for bad in (dict(hidden=68, dys=72, xs=72, dxs=72), dict(dys=68), dict(dw3=P(264))):
        assert call(**bad) == -2, bad
    assert call(wsb=1000) == -4
    assert call(rows=0, dw1=None, dw3=None, dw2=None) == 0


def test_workspace_sizes(lib):
    assert lib.muon_gated_ffn_workspace_bytes(100, 3, 64, 72) >= 100 * 72 * 2
    assert lib.muon_gated_ffn_backward_workspace_bytes(100, 3, 64, 72) >= 3 * 100 * 72 * 2
    for bad in ((0, 1, 64, 72), (1, 0, 64, 72), (1, 1, 60, 72), (1, 1, 64, -8)):
        assert lib.muon_gated_ffn_workspace_bytes(*bad) == 0
        assert lib.muon_gated_ffn_backward_workspace_bytes(*bad) == 0
    assert lib.muon_block_norm_backward_workspace_bytes(0, 64) == 0
    assert lib.muon_block_norm_backward_workspace_bytes(1, 1 << 20) == 0


def test_block_norm(lib):
    def call(**kw):
        base = dict(rows=2, hidden=64, residual=256, residual_stride=64, block=256, block_stride=64, scale=1.0,
                    eps=1e-6, residual_out=256, residual_out_stride=64, normed=256, normed_stride=64)
        return lib.muon_block_norm(ctypes.byref(NormArgs(**{**base, **kw})), None)

    assert lib.muon_block_norm(None, None) == -1
    for bad in (dict(rows=-1), dict(hidden=0), dict(residual_type=2), dict(branch_type=-1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(scale=float("inf")), dict(residual=None), dict(residual_out=None),
                dict(block=None, normed=None), dict(residual_stride=63), dict(block_stride=0),
                dict(normed_stride=10), dict(gate=256, gate_stride=5)):
        assert call(**bad) == -1, bad
    assert call(branch_type=1) == -2
    assert call(hidden=16385, residual_stride=20000) == -2
    assert call(rows=0, residual=None) == 0


def test_block_norm_backward(lib):
    def call(ws=P(256), wsb=0, **kw):
        base = dict(rows=2, hidden=64, dresidual_out=256, dresidual_out_stride=64, dnormed=256, dnormed_stride=64,
                    residual=256, residual_stride=64, block=256, block_stride=64, rstd_post=256, rstd_pre=256,
                    scale=1.0, dresidual=256, dresidual_stride=64, dblock=256, dblock_stride=64, dw_pre=256)
        return lib.muon_block_norm_backward(ctypes.byref(NormBackwardArgs(**{**base, **kw})), ws, wsb, None)

    assert lib.muon_block_norm_backward(None, None, 0, None) == -1
    for bad in (dict(rows=-1), dict(residual_type=7), dict(scale=float("nan")), dict(residual=None),
                dict(rstd_pre=None), dict(rstd_post=None), dict(dnormed=None), dict(block=None),
                dict(dnormed=None, dresidual_out=None, dw_pre=None), dict(dgate=256), dict(gate_stride=-1),
                dict(dresidual=None, dblock=None, dw_pre=None), dict(dblock_stride=3), dict(ws=P(16), wsb=1 << 30)):
        assert call(**bad) == -1, bad
    assert call(hidden=20000) == -2
    assert call(rows=0, dw_pre=None) == 0


def test_token_logprobs(lib):
    def call(x=P(256), stride=100, tokens=P(256), rows=2, vocab=100, type_=0, logp=P(256), entropy=None, lse=None,
             top=0, ids=None, tlp=None):
        return lib.muon_token_logprobs(x, stride, tokens, rows, vocab, type_, logp, entropy, lse, top, ids, tlp, None)

    for bad in (dict(rows=-1), dict(vocab=0), dict(type_=3), dict(stride=99), dict(top=-1), dict(top=5),
                dict(ids=P(256)), dict(x=None), dict(tokens=None), dict(logp=None),
                dict(top=20, ids=P(256), vocab=10)):
        assert call(**bad) == -1, bad
    assert call(top=33, ids=P(256)) == -2
    assert call(rows=0, x=None) == 0

    def back(x=P(256), stride=100, tokens=P(256), lse=P(256), ent=P(256), dlogp=P(256), dent=P(256), rows=2,
             vocab=100, type_=0, out=P(256), out_stride=100):
        return lib.muon_token_logprobs_backward(x, stride, tokens, lse, ent, dlogp, dent, rows, vocab, type_, out,
                                                out_stride, None)

    for bad in (dict(rows=-1), dict(vocab=0), dict(type_=2), dict(stride=1), dict(out_stride=99), dict(x=None),
                dict(lse=None), dict(ent=None), dict(tokens=None), dict(dlogp=None, dent=None), dict(out=None)):
        assert back(**bad) == -1, bad
    assert back(x=P(257)) == -2
    assert back(rows=0) == 0


def test_the_binding_refuses_what_is_no_cuda_tensor(lib):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ops = mk._ops()
    for bad in (None, 3, "x", x):
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            ops.gated_ffn(bad, x, x, x, None, 0, False, None, None, 0)
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            ops.block_norm(bad, None, None, None, None, 1.0, 1e-6, True, None, None, 0)
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            ops.token_logprobs(bad, None, 0, 0)
    for f in (ops.gated_ffn, ops.gated_ffn_backward, ops.block_norm, ops.block_norm_backward, ops.token_logprobs,
              ops.token_logprobs_backward):
        with pytest.raises(TypeError, match="expected"):
            f()
    with pytest.raises(ValueError, match="no address"):
        ops.bind({})


def test_missing_binding_fails_loudly(lib, monkeypatch, tmp_path):
    monkeypatch.setattr(mk, "OPS_PATH", str(tmp_path / "nope.so"))
    monkeypatch.setattr(mk, "_ops_module", None)
    with pytest.raises(mk.MuonLibraryMissing):
        mk._ops()


def test_pointers_off_their_elements_are_refused(lib):
    """On the host: a kernel's access through one would be a misaligned address."""
    assert ffn(lib, off=P(256 + 4)) == -2
    assert lib.muon_gated_ffn_backward(P(256), 64, P(256), 64, P(256), P(256), P(256), P(256), P(256), P(256 + 4), 4, 2,
                                       64, 72, 0, P(256), 64, P(256), P(256), P(256), P(256), 0, None) == -2
    for rt, bt in ((0, 0), (1, 0), (1, 1)):
        for name, fields in (("muon_block_norm", NormArgs), ("muon_block_norm_backward", NormBackwardArgs)):
            base = dict(rows=2, hidden=64, residual_type=rt, branch_type=bt, scale=1.0)
            base |= {f: 256 for f, t in fields._fields_ if t is P}
            base |= {f: 64 for f, _ in fields._fields_ if f.endswith("_stride")}
            for f in (f for f, t in fields._fields_ if t is P):
                size = 4 if f.startswith("rstd") else 4 if (rt if "residual" in f else bt) else 2
                args = fields(**{**base, f: 256 + size // 2})
                extra = (P(256), 0) if "backward" in name else ()   # a workspace of no bytes: no call gets further
                assert getattr(lib, name)(ctypes.byref(args), *extra, None) == -2, (name, f, rt, bt)
    for type_ in (0, 1):
        base = dict(logits=256, tokens=256, logp=256, entropy=256, lse=256, ids=256, values=256)
        size = {"logits": 4 if type_ else 2, "tokens": 8, "ids": 8}
        for k in base:
            v = {**base, k: 256 + size.get(k, 4) // 2}
            assert lib.muon_token_logprobs(v["logits"], 100, v["tokens"], 2, 100, type_, v["logp"], v["entropy"],
                                           v["lse"], 5, v["ids"], v["values"], None) == -2, (k, type_)
        base = dict(logits=256, tokens=256, lse=256, entropy=256, dlogp=256, dentropy=256, out=256)
        for k in base:
            v = {**base, k: 256 + (size["logits"] if k == "out" else size.get(k, 4)) // 2}
            assert lib.muon_token_logprobs_backward(v["logits"], 100, v["tokens"], v["lse"], v["entropy"], v["dlogp"],
                                                    v["dentropy"], 2, 100, type_, v["out"], 100, None) == -2, (k, type_)


def test_what_a_backward_call_does_not_read_may_lie_anywhere(lib):
    def call(x=P(256), xs=64, w=P(256), dx=P(256), dw=P(256), dxs=64):
        return lib.muon_gated_ffn_backward(P(256), 64, x, xs, P(256), P(256), w, w, P(256), P(256), 4, 2, 64, 72, 0, dx,
                                           dxs, dw, dw, dw, P(256), 0, None)

    # past every check of the arguments a workspace of no bytes is what is refused
    assert call(x=P(258)) == call(xs=67) == call(w=P(258)) == call(dxs=67) == -2
    assert call(x=P(258), xs=67, dw=None) == -4
    assert call(w=P(258), dx=None, dxs=67) == -4
    assert call(x=P(258), dx=None) == -2 and call(w=P(258), dw=None) == -2


def test_parts_of_a_cut_sum_go_by_the_device(lib):
    """Scratch of the cut weight gradients: as many parts as pairs of SMs hold, not a fixed number."""
    # one block a SM of 8192 columns, two fp32 sums each
    sms = lib.muon_block_norm_backward_workspace_bytes(1 << 20, 8192) // (2 * 8192 * 4)
    rows, H, F = 1 << 20, 19 * 256, 256

    def up(n):   # regions start on 256 bytes
        return (n + 255) // 256 * 256

    dw13, dw2 = sms // 2 // (19 * 2), sms // 2 // 19   # tiles of 256 x 128 of dW1 and dW3, of 256 x 256 of dW2
    sums = max(2 * dw13 if dw13 > 1 else 0, dw2) * H * F * 4
    want = 3 * up(rows * F * 2) + up(64 * (2 * H + 3 * F) * 2) + up(sums)
    assert lib.muon_gated_ffn_backward_workspace_bytes(rows, 1, H, F) == want
