"""The norms before and after a block, against their definition in 64 bits.

Bounds.  Everything is fp32 but one rounding of each output to its type
(2^-9 relative for bf16, nothing more for fp32).  A mean of squares of up to
16384 terms, each thread adding at most 32 and the rest in a tree, is within
48 * 2^-24 of itself, so a row's factors are within 2^-18; an entry is within
2^-16 of the sum of the magnitudes it is made of (a handful of roundings and
two such factors).  A sum over rows adds at most one rounding per row of a
group and per group: rows * 2^-24 of the sum of magnitudes more.
"""

import pytest
import torch

from tests._util import require_gpu

pytestmark = pytest.mark.gpu
E32 = 2.0 ** -16


@pytest.fixture(scope="module")
def mk():
    return require_gpu()


TYPES = [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")]
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
WIDTHS = [1, 7, 8, 31, 64, 250, 256, 264, 1001, 2056, 4100, 6144, 6152, 8193, 12288, 16384]


def unit(dt):
    return 2.0 ** -8 if dt is torch.bfloat16 else 2.0 ** -23   # twice the rounding


def inputs(T, H, rt, bt, gate, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * T + H)

    def n(*shape, std=1.0, mean=0.0, dt=bt):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dt)

    d = {"r": n(T, H, std=3.0, dt=rt), "b": n(T, H, std=0.5), "w_post": n(H, std=0.2, mean=1.0),
         "w_pre": n(H, std=0.2, mean=1.0), "gate": None, "dr": n(T, H, dt=rt), "dy": n(T, H)}
    if gate == "shared":
        d["gate"] = n(H, std=0.3, mean=0.5)
    elif gate == "rows":
        d["gate"] = n(T, H, std=0.3, mean=0.5)
    return d


def f64(t):
    return None if t is None else t.double()


def forward64(d, scale, eps, post=True):
    """Outputs and the magnitudes that their bounds go by."""
    r, b, wq, wp, g = (f64(d[k]) for k in ("r", "b", "w_post", "w_pre", "gate"))
    mags = r.abs()
    q = None
    if post:
        q = (b.square().mean(1) + eps).pow(-0.5)
        step = scale * b * q[:, None]
        if wq is not None:
            step = step * wq
        if g is not None:
            step = step * g
        r, mags = r + step, mags + step.abs()
    p = (r.square().mean(1) + eps).pow(-0.5)
    w = 1.0 if wp is None else wp
    return r, mags, r * p[:, None] * w, mags * p[:, None] * abs(w), q, p


def within(got, value, mags, name, extra=0.0):
    err = (got.double() - value).abs()
    bound = unit(got.dtype) * value.abs() + (E32 + extra) * mags + 1e-30
    assert bool((err <= bound).all()), (name, float((err / bound).max()))


@pytest.mark.parametrize("gate", ["none", "shared", "rows"])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
def test_forward(mk, H, types, gate):
    rt, bt = (DT[t] for t in types)
    T = 13
    d = inputs(T, H, rt, bt, gate)
    r, y, q, p = mk.muon_block_norm(d["r"], d["b"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"], scale=0.7,
                                    eps=1e-5)
    R, mR, Y, mY, Q, P = forward64(d, 0.7, 1e-5)
    assert r.dtype is rt and y.dtype is bt
    within(r, R, mR, "r")
    within(y, Y, mY, "y")
    within(q, Q, Q, "rstd_post")
    within(p, P, P, "rstd_pre", extra=2 * E32)


def backward64(d, r, q, p, scale, post=True, pre=True):
    """(value, magnitudes) of each gradient, from the stored r', q and p."""
    dr, dy, b, wq, wp, g = (f64(d[k]) for k in ("dr", "dy", "b", "w_post", "w_pre", "gate"))
    r, out = r.double(), {}
    m = torch.zeros_like(r) if dr is None else dr.abs()
    dr = torch.zeros_like(r) if dr is None else dr
    if pre:
        P = p.double()[:, None]
        xh = r * P
        t = dy if wp is None else dy * wp
        m = m + P * (t.abs() + xh.abs() * (t * xh).abs().mean(1, keepdim=True))
        dr = dr + P * (t - xh * (t * xh).mean(1, keepdim=True))
        out["dw_pre"] = ((dy * xh).sum(0), (dy * xh).abs().sum(0))
    out["dresidual"] = (dr, m)
    if post:
        Q = q.double()[:, None]
        bh = b * Q
        G, W = (1.0 if g is None else g), (1.0 if wq is None else wq)
        dn, mn = scale * G * dr, abs(scale * G) * m
        dg, mg = scale * dr * bh * W, (abs(scale) * m * bh * W).abs()
        if g is not None:
            out["dgate"] = (dg, mg) if g.dim() == 2 else (dg.sum(0), mg.sum(0))
        out["dw_post"] = ((dn * bh).sum(0), (mn * bh.abs()).sum(0))
        t, mt = dn * W, mn * abs(W)
        out["dblock"] = (Q * (t - bh * (t * bh).mean(1, keepdim=True)),
                         Q * (mt + bh.abs() * (mt * bh.abs()).mean(1, keepdim=True)))
    return out


@pytest.mark.parametrize("gate", ["none", "shared", "rows"])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("T", [1, 700])
def test_backward(mk, H, types, gate, T):
    if T * H > 5_000_000 and gate == "none":
        T = 300
    rt, bt = (DT[t] for t in types)
    d = inputs(T, H, rt, bt, gate, seed=1)
    r, y, q, p = mk.muon_block_norm(d["r"], d["b"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"], scale=-1.3)
    got = mk.muon_block_norm_backward(d["dr"], d["dy"], r, d["b"], q, p, w_post=d["w_post"], gate=d["gate"],
                                      w_pre=d["w_pre"], scale=-1.3)
    ref = backward64(d, r, q, p, -1.3)
    assert (got.dgate is None) == (gate == "none")
    for k, (value, mags) in ref.items():
        v = getattr(got, k)
        assert v.dtype is (rt if k == "dresidual" else bt) and v.shape == value.shape
        within(v, value, mags, k, extra=T * 2.0 ** -24)
    again = mk.muon_block_norm_backward(d["dr"], d["dy"], r, d["b"], q, p, w_post=d["w_post"], gate=d["gate"],
                                        w_pre=d["w_pre"], scale=-1.3)
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)   # sums in a fixed order


@pytest.mark.parametrize("H", [72, 99])
def test_parts_alone(mk, H):
    d = inputs(9, H, torch.float32, torch.bfloat16, "shared", seed=2)
    # only the norm before a block
    r, y, q, p = mk.muon_block_norm(d["r"], w_pre=d["w_pre"])
    assert r is d["r"] and q is None
    _, _, Y, mY, _, P = forward64(d, 1.0, 1e-6, post=False)
    within(y, Y, mY, "y")
    got = mk.muon_block_norm_backward(None, d["dy"], r, None, None, p, w_pre=d["w_pre"])
    for k, (v, m) in backward64({**d, "dr": None}, r, None, p, 1.0, post=False).items():
        within(getattr(got, k), v, m, k)
    assert got.dblock is None and got.dgate is None and got.dw_post is None
    # only the norm after one, without weights or gate
    r, y, q, p = mk.muon_block_norm(d["r"], d["b"], norm_next=False)
    assert y is None and p is None
    bare = {**d, "w_post": None, "gate": None, "w_pre": None}
    R, mR, _, _, Q, _ = forward64(bare, 1.0, 1e-6)
    within(r, R, mR, "r")
    got = mk.muon_block_norm_backward(d["dr"], None, r, d["b"], q)
    for k, (v, m) in backward64(bare, r, q, None, 1.0, pre=False).items():
        if k in ("dresidual", "dblock"):
            within(getattr(got, k), v, m, k)
    assert got.dw_post is None and got.dw_pre is None


def test_many_rows_with_one_sum_each(mk):
    """Long columns of the pieces alone: one reduction a row, so every row reuses the buffers of the last."""
    d = inputs(5000, 520, torch.float32, torch.float32, "none", seed=3)
    _, _, _, p = mk.muon_block_norm(d["r"], w_pre=d["w_pre"])
    got = mk.muon_block_norm_backward(d["dr"], d["dy"], d["r"], None, None, p, w_pre=d["w_pre"])
    for k, (v, m) in backward64(d, d["r"], None, p, 1.0, post=False).items():
        within(getattr(got, k), v, m, k, extra=5000 * 2.0 ** -24)


def test_in_place_strides_and_no_write_outside(mk):
    d = inputs(33, 136, torch.bfloat16, torch.bfloat16, "rows", seed=4)
    ref = mk.muon_block_norm(d["r"], d["b"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
    for shift in (8, 3):   # aligned to 16 bytes, and not
        wide = {k: torch.full((33, 160), 5.0, dtype=torch.bfloat16, device="cuda") for k in ("r", "b", "gate", "y")}
        view = {k: v[:, shift:shift + 136] for k, v in wide.items()}
        for k in ("r", "b", "gate"):
            view[k].copy_(d[k])
        got = mk.muon_block_norm(view["r"], view["b"], w_post=d["w_post"], gate=view["gate"], w_pre=d["w_pre"],
                                 out=view["r"], normed=view["y"])
        for a, b in zip(got, ref):   # the sums' order differs between the two ways of access
            assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())
        for v in wide.values():
            assert bool((v[:, :shift] == 5).all()) and bool((v[:, shift + 136:] == 5).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_row_stays_alone_and_a_zero_row_is_finite(mk, bad):
    d = inputs(6, 264, torch.float32, torch.bfloat16, "shared", seed=5)
    d["b"][1] = 0.0
    d["r"][1] = 0.0
    ref = mk.muon_block_norm(d["r"], d["b"], gate=d["gate"])
    assert all(bool(t.isfinite().all()) for t in ref)
    d["b"][3, 7] = bad
    got = mk.muon_block_norm(d["r"], d["b"], gate=d["gate"])
    rows = [0, 1, 2, 4, 5]
    for a, b in zip(got, ref):
        assert torch.equal(a[rows], b[rows])
    assert bool(got[1][3].isnan().any())


def test_gradient_agrees_with_differences(mk):
    d = inputs(5, 40, torch.float32, torch.float32, "shared", seed=6)
    r, y, q, p = mk.muon_block_norm(d["r"], d["b"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"], scale=0.6)
    got = mk.muon_block_norm_backward(d["dr"], d["dy"], r, d["b"], q, p, w_post=d["w_post"], gate=d["gate"],
                                      w_pre=d["w_pre"], scale=0.6)
    for k, grad in (("r", got.dresidual), ("b", got.dblock), ("w_post", got.dw_post), ("gate", got.dgate),
                    ("w_pre", got.dw_pre)):
        v = torch.randn(d[k].shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda",
                        dtype=torch.float64)
        slope = 0.0
        for sign in (1, -1):
            moved = dict(d)
            moved[k] = d[k].double() + sign * 1e-5 * v
            R, _, Y, _, _, _ = forward64(moved, 0.6, 1e-6)
            slope += sign * float((R * d["dr"].double()).sum() + (Y * d["dy"].double()).sum()) / 2e-5
        # differences: 1e-10 in the third derivative and 1e-16 / 1e-5; the gradient: 2^-16 of its magnitudes
        assert abs(float((grad.double() * v).sum()) - slope) <= 2.0 ** -12 * float(grad.double().norm() * v.norm()), k


def test_no_rows_and_refusals(mk):
    d = inputs(4, 64, torch.float32, torch.bfloat16, "shared")
    e = {k: (v[:0] if v is not None and v.dim() == 2 else v) for k, v in d.items()}
    r, y, q, p = mk.muon_block_norm(e["r"], e["b"], gate=e["gate"], w_pre=e["w_pre"])
    assert r.shape == (0, 64) and y.shape == (0, 64)
    g = mk.muon_block_norm_backward(e["dr"], e["dy"], r, e["b"], q, p, gate=e["gate"], w_pre=e["w_pre"])
    assert not bool(g.dgate.any()) and not bool(g.dw_pre.any())
    for kw in (dict(w_post=d["w_post"].float()), dict(gate=d["gate"].double())):
        with pytest.raises(TypeError):
            mk.muon_block_norm(d["r"], d["b"], **kw)
    with pytest.raises(TypeError):
        mk.muon_block_norm(d["r"].half(), d["b"])
    for args, kw in (((d["r"], d["b"][:3]), {}), ((d["r"], d["b"]), dict(w_pre=d["w_pre"][:5])),
                     ((d["r"],), dict(gate=d["gate"])), ((d["r"],), dict(norm_next=False)),
                     ((d["r"], d["b"]), dict(norm_next=False, w_pre=d["w_pre"])), ((d["r"][0],), {})):
        with pytest.raises(ValueError):
            mk.muon_block_norm(*args, **kw)
    with pytest.raises(mk.MuonError) as err:
        mk.muon_block_norm(d["r"].bfloat16(), d["b"].float())
    assert err.value.status == -2
    with pytest.raises(ValueError):
        mk.muon_block_norm_backward(None, None, d["r"])
    with pytest.raises(mk.MuonError) as err:
        mk.muon_block_norm_backward(d["dr"], d["dy"], d["r"], None, None, torch.ones(4, device="cuda"),
                                    w_pre=d["w_pre"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert err.value.status == -4
    mk.muon_inject_alloc_failures(1)
    with pytest.raises(mk.MuonError) as err:
        mk.muon_block_norm_backward(d["dr"], d["dy"], d["r"], None, None, torch.ones(4, device="cuda"),
                                    w_pre=d["w_pre"])
    assert err.value.status == -4 and mk.muon_inject_alloc_failures(0) == 0


@pytest.mark.parametrize("T, H, types, gate", [
    (9001, 1032, ("f32", "f32"), "rows"),      # several blocks of one SM, every slot filled several times
    (5000, 2056, ("bf16", "bf16"), "shared"),
    (2500, 6144, ("f32", "bf16"), "rows"),
    (2500, 6144, ("bf16", "bf16"), "none"),
    (1500, 6144, ("f32", "f32"), "rows"),      # too wide for two rows at once
    (1500, 6152, ("f32", "bf16"), "shared"),
    (1700, 8192, ("bf16", "bf16"), "rows"),
    (900, 8200, ("bf16", "bf16"), "shared"),
])
def test_backward_of_rows_that_stream_in(mk, T, H, types, gate):
    """Many rows a block, of arrays with gaps between the rows, which no copy may write to."""
    rt, bt = (DT[t] for t in types)
    d = inputs(T, H, rt, bt, gate, seed=5)
    r, _, q, p = mk.muon_block_norm(d["r"], d["b"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
    wide = {}

    def spread(t):   # the same rows, 16 elements apart
        if t is None or t.dim() == 1:
            return t
        w = torch.full((T, H + 16), 3.0, dtype=t.dtype, device="cuda")
        w[:, 8:H + 8] = t
        wide[len(wide)] = w
        return w[:, 8:H + 8]

    got = mk.muon_block_norm_backward(spread(d["dr"]), spread(d["dy"]), spread(r), spread(d["b"]), q, p,
                                      w_post=d["w_post"], gate=spread(d["gate"]), w_pre=d["w_pre"])
    for k, (value, mags) in backward64(d, r, q, p, 1.0).items():
        within(getattr(got, k), value, mags, k, extra=T * 2.0 ** -24)
    for w in wide.values():
        assert bool((w[:, :8] == 3).all()) and bool((w[:, H + 8:] == 3).all())


@pytest.mark.parametrize("T, H, types, gate", [
    (9001, 1032, ("f32", "f32"), "rows"),
    (5000, 2056, ("bf16", "bf16"), "shared"),
    (2500, 6144, ("f32", "bf16"), "rows"),
    (2500, 6144, ("bf16", "bf16"), "none"),
    (1500, 6152, ("f32", "f32"), "shared"),
    (1700, 8192, ("f32", "f32"), "rows"),
    (900, 16384, ("bf16", "bf16"), "none"),
])
def test_forward_of_rows_that_stream_in(mk, T, H, types, gate):
    """Many rows a block, of arrays with gaps between the rows; the stream is updated in place."""
    rt, bt = (DT[t] for t in types)
    d = inputs(T, H, rt, bt, gate, seed=6)
    R, mR, Y, mY, Q, P = forward64(d, -0.6, 1e-6)
    wide = {}

    def spread(t):
        if t is None or t.dim() == 1:
            return t
        w = torch.full((T, H + 16), 3.0, dtype=t.dtype, device="cuda")
        w[:, 8:H + 8] = t
        wide[len(wide)] = w
        return w[:, 8:H + 8]

    stream, y = spread(d["r"]), spread(torch.zeros(T, H, dtype=bt, device="cuda"))
    r, got, q, p = mk.muon_block_norm(stream, spread(d["b"]), w_post=d["w_post"], gate=spread(d["gate"]),
                                      w_pre=d["w_pre"], scale=-0.6, out=stream, normed=y)
    within(stream, R, mR, "r")
    within(y, Y, mY, "y")
    within(q, Q, Q, "rstd_post")
    within(p, P, P, "rstd_pre", extra=2 * E32)
    for w in wide.values():
        assert bool((w[:, :8] == 3).all()) and bool((w[:, H + 8:] == 3).all())


@pytest.mark.parametrize("size", [1e-17, 1e-15, 1e14, 1e17])
@pytest.mark.parametrize("T, H, types", [(5, 264, ("f32", "f32")), (300, 2056, ("f32", "bf16")),
                                         (7, 1001, ("f32", "f32"))])
def test_gradient_keeps_the_range_of_the_forward_pass(mk, T, H, types, size):
    """Blocks whose mean square is in fp32's range while the cube of their reciprocal norm is not."""
    rt, bt = (DT[t] for t in types)
    d = inputs(T, H, rt, bt, "shared", seed=7)
    d["b"] = (d["b"].float() * (2 * size)).to(bt)
    r, y, q, p = mk.muon_block_norm(d["r"], d["b"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"], scale=0.8,
                                    eps=0.0)
    R, mR, Y, mY, Q, _ = forward64(d, 0.8, 0.0)
    within(r, R, mR, "r")
    within(y, Y, mY, "y")
    within(q, Q, Q, "rstd_post")
    got = mk.muon_block_norm_backward(d["dr"], d["dy"], r, d["b"], q, p, w_post=d["w_post"], gate=d["gate"],
                                      w_pre=d["w_pre"], scale=0.8)
    for k, (value, mags) in backward64(d, r, q, p, 0.8).items():
        within(getattr(got, k), value, mags, k, extra=T * 2.0 ** -24)


def kernels_of(mk, call):
    mk.muon_trace_begin()
    out = call()
    return out, set(mk.muon_trace_end())


@pytest.mark.parametrize("gate", ["none", "shared", "rows"])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("H", [3416, 5120, 6144, 6152, 7000, 8192])
def test_forward_of_staged_rows(mk, H, types, gate):
    """Rows enough to go through shared memory, where their bytes or their width ask for it: which did is looked at."""
    rt, bt = (DT[t] for t in types)
    T = 2100                                     # about 14 rows a block: every slot is filled again
    row = H * (rt.itemsize + bt.itemsize * (2 if gate == "rows" else 1))
    staged = row >= 40 * 1024 or H > 6144        # bytes, or more threads than the plain form's blocks have
    d = inputs(T, H, rt, bt, gate, seed=8)
    (r, y, q, p), names = kernels_of(mk, lambda: mk.muon_block_norm(
        d["r"], d["b"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"], scale=0.9))
    assert names == {"block_norm_staged" if staged else "block_norm"}
    R, mR, Y, mY, Q, P = forward64(d, 0.9, 1e-6)
    within(r, R, mR, "r")
    within(y, Y, mY, "y")
    within(q, Q, Q, "rstd_post")
    within(p, P, P, "rstd_pre", extra=2 * E32)
    again = mk.muon_block_norm(d["r"], d["b"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"], scale=0.9)
    assert all(torch.equal(a, b) for a, b in zip((r, y, q, p), again))


@pytest.mark.parametrize("gate", ["none", "shared", "rows"])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("H", [1032, 6144, 6152, 8192, 8200])
def test_backward_of_staged_rows(mk, H, types, gate):
    rt, bt = (DT[t] for t in types)
    T = 1900                                     # 3 or 12 rows a block
    row = (H * (2 * rt.itemsize + bt.itemsize * (3 if gate == "rows" else 2)) + 127) // 128 * 128
    staged = 2 * row <= 216 * 1024 and H <= 8192
    d = inputs(T, H, rt, bt, gate, seed=9)
    r, _, q, p = mk.muon_block_norm(d["r"], d["b"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"], scale=0.9)
    got, names = kernels_of(mk, lambda: mk.muon_block_norm_backward(
        d["dr"], d["dy"], r, d["b"], q, p, w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"], scale=0.9))
    assert names == {"block_norm_backward_staged" if staged else "block_norm_backward", "norm_weight_sum"}
    for k, (value, mags) in backward64(d, r, q, p, 0.9).items():
        within(getattr(got, k), value, mags, k, extra=T * 2.0 ** -24)
