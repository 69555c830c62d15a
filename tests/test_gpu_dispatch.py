"""Tokens to rows sorted by expert and back, and the gradients.

The sort and the copies are exact.  Bounds of the sums: a sum of n products in
fp32 is within (n + 1) 2^-24 of the sum of the products' magnitudes when added
in turn, and rounded once to its type.  dweights adds at most hidden / 64 + 16
products on a path of its tree: (hidden / 64 + 24) 2^-24.
"""

import pytest
import torch

from tests._util import require_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def mk():
    return require_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def choice(T, k, E, seed=0, holes=0.1, distinct=True):
    g = gen(seed + T * 31 + k * 7 + E)
    if distinct and k <= E:
        ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices
    else:
        ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
    ids[torch.rand(T, k, generator=g, device="cuda") < holes] = -1
    return ids


def plain(x, ids, E):
    T, k = ids.shape
    key = torch.where((ids >= 0) & (ids < E), ids, E).flatten()
    order = torch.sort(key, stable=True).indices
    rows = x[order // k] * (key[order] < E)[:, None]
    rows = torch.where((key[order] < E)[:, None], rows, 0)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=x.device)
    place = torch.where(key < E, place, -1 - place).view(T, k)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=x.device), counts.cumsum(0)])
    offsets[E] = T * k
    return rows, offsets, place


# few slots (one launch) and many (the cluster's sort), experts without slots, one expert, all slots of one
SIZES = [(1, 1, 1, 1), (1, 8, 384, 6144), (3, 2, 5, 40), (64, 8, 32, 264), (257, 8, 384, 72), (300, 7, 1024, 33),
         (1000, 3, 1, 136), (5000, 2, 1024, 8), (4099, 4, 33, 1001), (40, 32, 64, 2056), (33000, 8, 384, 16),
         (256, 8, 31, 100), (2049, 1, 7, 6152)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,H", SIZES)
def test_dispatch(mk, T, k, E, H, dt):
    ids = choice(T, k, E)
    x = torch.randn(T, H, generator=gen(T), device="cuda").to(DT[dt])
    got = mk.muon_dispatch(x, ids, E)
    assert mk.muon_get_device_status() == 0
    rows, offsets, place = plain(x, ids, E)
    assert torch.equal(got.offsets, offsets) and torch.equal(got.place, place) and torch.equal(got.rows, rows)


@pytest.mark.parametrize("T", [64, 9000])
def test_uneven_choices(mk, T):
    x = torch.randn(T, 64, generator=gen(1), device="cuda").bfloat16()
    one = torch.full((T, 4), 5, device="cuda")                  # one expert takes every slot of every token
    none = torch.full((T, 4), -1, device="cuda")
    last = torch.full((T, 4), 15, device="cuda")
    mixed = choice(T, 4, 16, seed=3, holes=0.9, distinct=False)
    for ids in (one, none, last, mixed, torch.full((T, 4), -(1 << 60), device="cuda")):
        got = mk.muon_dispatch(x, ids, 16)
        rows, offsets, place = plain(x, ids, 16)
        assert torch.equal(got.offsets, offsets) and torch.equal(got.place, place) and torch.equal(got.rows, rows)
    assert mk.muon_get_device_status() == 0


@pytest.mark.parametrize("T", [64, 9000])
def test_ids_out_of_range_are_reported_and_not_routed(mk, T):
    x = torch.randn(T, 64, generator=gen(2), device="cuda").bfloat16()
    ids = choice(T, 4, 16, seed=4)
    ids[7, 1], ids[T - 1, 3], ids[0, 0] = 16, 1 << 50, 1 << 32
    got = mk.muon_dispatch(x, ids, 16)
    assert mk.muon_get_device_status() == -6
    rows, offsets, place = plain(x, ids, 16)
    assert torch.equal(got.offsets, offsets) and torch.equal(got.place, place) and torch.equal(got.rows, rows)
    assert mk.muon_get_device_status() == 0


def test_a_nan_in_a_token_that_is_not_routed_goes_nowhere(mk):
    ids = choice(50, 4, 8, holes=0.0)
    ids[3] = -1
    x = torch.randn(50, 96, generator=gen(5), device="cuda")
    x[3] = float("nan")
    got = mk.muon_dispatch(x, ids, 8)
    assert not bool(got.rows.isnan().any())
    y = got.rows.clone()
    y[-4:] = float("inf")                                    # rows of no slot are not read
    w = torch.rand(50, 4, generator=gen(6), device="cuda")
    w[3] = float("nan")
    out = mk.muon_combine(y, got.place, w)
    assert not bool(out.isnan().any()) and not bool(out[3].any())
    dy, dw = mk.muon_combine_backward(x, y, got.place, w)
    assert not bool(dy.isnan().any()) and not bool(dy[-4:].any())
    assert not bool(dw.isnan().any()) and not bool(dw[3].any())
    assert not bool(mk.muon_dispatch_backward(y, got.place).isnan().any())


def given_rows(place, y):
    return torch.where((place >= 0)[:, :, None], y.double()[place.clamp(min=0)], 0.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,H", SIZES)
def test_combine_and_gradients(mk, T, k, E, H, dt):
    t = DT[dt]
    unit = torch.finfo(t).eps / 2
    g = gen(T + H)
    place = mk.muon_dispatch(torch.zeros(T, 1, device="cuda"), choice(T, k, E, seed=9), E).place
    y = torch.randn(T * k, H, generator=g, device="cuda").to(t)
    w = torch.randn(T, k, generator=g, device="cuda")
    dout = torch.randn(T, H, generator=g, device="cuda").to(t)
    dx, out = mk.muon_dispatch_backward(y, place), mk.muon_combine(y, place, w)
    dy, dw = mk.muon_combine_backward(dout, y, place, w)
    assert mk.muon_get_device_status() == 0
    assert dx.dtype is t and out.dtype is t and dy.dtype is t and dw.dtype is torch.float32
    routed = place >= 0
    want_dy = torch.zeros(T * k, H, device="cuda", dtype=torch.float64)
    for a in range(0, T, 4096):                              # the 64-bit forms take 16 times the memory
        s = slice(a, a + 4096)
        rows, d, ww = given_rows(place[s], y), dout[s].double(), w[s].double()[:, :, None]
        for got, terms in ((dx, rows), (out, rows * ww)):
            want, mags = terms.sum(1), terms.abs().sum(1)
            assert bool(((got[s].double() - want).abs() <= unit * want.abs() + (k + 1) * 2.0 ** -24 * mags).all())
        terms = rows * d[:, None, :]
        bound = (H / 64 + 24) * 2.0 ** -24 * terms.abs().sum(2)
        assert bool(((dw[s].double() - terms.sum(2)).abs() <= bound).all())
        want_dy[place[s][routed[s]]] = (ww * d[:, None, :])[routed[s]]
    assert bool(((dy.double() - want_dy).abs() <= unit * want_dy.abs()).all())
    # one of them alone, and without weights
    assert torch.equal(mk.muon_combine_backward(dout, None, place, w, need_dweights=False)[0], dy)
    only = mk.muon_combine_backward(dout, y, place, w, need_dy=False)
    assert only[0] is None and torch.equal(only[1], dw)
    ones = mk.muon_combine_backward(dout, None, place)
    assert ones[1] is None
    want_dy[place[routed]] = dout.double()[:, None, :].expand(T, k, H)[routed]
    assert torch.equal(ones[0].double(), want_dy)
    assert torch.equal(mk.muon_combine(y, place), dx)


def test_gradients_agree_with_differences(mk):
    place = mk.muon_dispatch(torch.zeros(9, 1, device="cuda"), choice(9, 3, 4), 4).place
    g = gen(11)
    y, w = torch.randn(27, 20, generator=g, device="cuda"), torch.randn(9, 3, generator=g, device="cuda")
    dout = torch.randn(9, 20, generator=g, device="cuda")
    dy, dw = mk.muon_combine_backward(dout, y, place, w)
    vy, vw = torch.randn_like(y).double(), torch.randn_like(w).double()
    slope = 0.0
    for sign in (1, -1):
        yy, ww = y.double() + sign * 1e-4 * vy, w.double() + sign * 1e-4 * vw
        slope += sign * float(((given_rows(place, yy) * ww[:, :, None]).sum(1) * dout.double()).sum()) / 2e-4
    got = float((dy.double() * vy).sum() + (dw.double() * vw).sum())
    assert abs(got - slope) <= 2.0 ** -16 * (float(dy.norm()) * float(vy.norm()) + float(dw.norm()) * float(vw.norm()))


def test_there_and_back(mk):
    # without weights a token comes back as many times as it has routed slots
    ids = choice(700, 4, 24, holes=0.3)
    x = torch.randint(-8, 9, (700, 72), generator=gen(12), device="cuda").bfloat16()
    d = mk.muon_dispatch(x, ids, 24)
    assert torch.equal(mk.muon_combine(d.rows, d.place), x * (ids >= 0).sum(1, keepdim=True))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shift,pitch", [(1, 75), (2, 76), (4, 80), (8, 96), (0, 73)])
def test_strides_and_alignment(mk, dt, shift, pitch):
    t, T, k, E, H = DT[dt], 90, 3, 12, 64
    ids = choice(T, k, E)
    wide = torch.randn(T, pitch, generator=gen(13), device="cuda").to(t)
    x = wide[:, shift:shift + H]
    want = mk.muon_dispatch(x.contiguous(), ids, E)
    flat = torch.full((T * k * H + 16,), 5.0, device="cuda", dtype=t)
    out = flat[shift:shift + T * k * H].view(T * k, H)
    got = mk.muon_dispatch(x, ids, E, out=out)
    assert got.rows is out and torch.equal(out, want.rows)
    assert bool((flat[:shift] == 5).all()) and bool((flat[shift + T * k * H:] == 5).all())
    w = torch.rand(T, k, generator=gen(14), device="cuda")
    target = torch.full((T, pitch), 3.0, device="cuda", dtype=t)
    mk.muon_combine(out, want.place, w, out=target[:, shift:shift + H])
    assert torch.equal(target[:, shift:shift + H], mk.muon_combine(want.rows, want.place, w))
    assert bool((target[:, :shift] == 3).all()) and bool((target[:, shift + H:] == 3).all())
    dy, dw = mk.muon_combine_backward(x, out, want.place, w)
    dy2, dw2 = mk.muon_combine_backward(x.contiguous(), want.rows, want.place, w)
    assert torch.equal(dy, dy2)
    # other accesses, other trees: both are within the bound of the sum
    bound = 2 * (H / 64 + 24) * 2.0 ** -24 * (given_rows(want.place, want.rows).abs() * x.double().abs()[:, None]).sum(2)
    assert bool(((dw - dw2).double().abs() <= bound).all())


def test_places_out_of_range_are_reported(mk):
    T, k, H = 20, 2, 40
    place = mk.muon_dispatch(torch.zeros(T, 1, device="cuda"), choice(T, k, 4, holes=0.0), 4).place
    y, w = torch.randn(T * k, H, generator=gen(15), device="cuda"), torch.rand(T, k, generator=gen(16), device="cuda")
    bad = place.clone()
    bad[3, 1], bad[4, 0], bad[5, 1], bad[6, 0] = T * k, 1 << 62, -1 - T * k, -(1 << 63)
    skipped = place.clone()
    skipped[3, 1], skipped[4, 0], skipped[5, 1], skipped[6, 0] = -1, -1, -1, -1
    got = mk.muon_combine(y, bad, w)
    assert mk.muon_get_device_status() == -6
    assert torch.equal(got, mk.muon_combine(y, skipped, w)) and mk.muon_get_device_status() == 0
    dout = torch.randn(T, H, generator=gen(17), device="cuda")
    dy = torch.full((T * k, H), 7.0, device="cuda")
    _, dw = mk.muon_combine_backward(dout, y, bad, w, dy=dy)
    assert mk.muon_get_device_status() == -6
    assert not bool(dw[3, 1]) and not bool(dw[4, 0]) and not bool(dw[5, 1]) and not bool(dw[6, 0])
    assert int((dy == 7).all(1).sum()) == 4                  # the rows that no slot names any more


def test_rows_past_32_bits(mk):
    T, k, H = 70000, 6, 6144                                 # 2.6e9 elements of rows
    ids = choice(T, k, 64)
    x = torch.randn(T, H, generator=gen(18), device="cuda").bfloat16()
    got = mk.muon_dispatch(x, ids, 64)
    for t in (0, 1, T // 2, T - 1):
        for j in range(k):
            p = int(got.place[t, j])
            row = got.rows[p if p >= 0 else -1 - p]
            assert torch.equal(row, x[t]) if p >= 0 else not bool(row.any())
    w = torch.rand(T, k, generator=gen(19), device="cuda")
    back = mk.muon_combine(got.rows, got.place, w)
    total = torch.where(ids >= 0, w, 0.0).sum(1, keepdim=True)
    err = (back.float() - x.float() * total).abs()
    assert bool((err <= 2.0 ** -8 * (x.float() * total).abs() + 8 * 2.0 ** -24 * x.float().abs() * 6).all())
    dy, dw = mk.muon_combine_backward(x, got.rows, got.place, w)
    p = got.place[T - 1]
    for j in range(k):
        if int(p[j]) >= 0:
            assert torch.equal(dy[int(p[j])], (w[T - 1, j] * x[T - 1].float()).bfloat16())
    assert mk.muon_get_device_status() == 0


def test_no_tokens(mk):
    ids = torch.empty(0, 4, device="cuda", dtype=torch.int64)
    got = mk.muon_dispatch(torch.empty(0, 16, device="cuda"), ids, 5)
    assert got.rows.shape == (0, 16) and got.offsets.tolist() == [0] * 6 and got.place.shape == (0, 4)
    assert mk.muon_combine(got.rows, got.place).shape == (0, 16)
    dy, dw = mk.muon_combine_backward(got.rows, got.rows, got.place, torch.empty(0, 4, device="cuda"))
    assert dy.shape == (0, 16) and dw.shape == (0, 4)


def test_refusals(mk):
    x, ids = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 2, device="cuda", dtype=torch.int64)
    with pytest.raises(mk.MuonError, match="INVALID"):
        mk.muon_dispatch(x, ids, 0)
    with pytest.raises(mk.MuonError, match="UNSUPPORTED"):
        mk.muon_dispatch(x, ids, 1025)
    with pytest.raises(mk.MuonError, match="UNSUPPORTED"):
        mk.muon_dispatch(x, ids[:, :1].expand(4, 33).contiguous(), 8)
    with pytest.raises(mk.MuonError, match="INVALID"):
        mk.muon_dispatch(x, ids[:, :0].contiguous(), 8)
    for bad in (x.half(), x.double()):
        with pytest.raises(TypeError, match="torch.bfloat16 or torch.float32"):
            mk.muon_dispatch(bad, ids, 8)
    with pytest.raises(TypeError, match="ids"):
        mk.muon_dispatch(x, ids.int(), 8)
    with pytest.raises(ValueError, match="x must have shape"):
        mk.muon_dispatch(x[:3], ids, 8)
    with pytest.raises(ValueError, match="out"):
        mk.muon_dispatch(x, ids, 8, out=torch.zeros(7, 64, device="cuda"))
    y = torch.zeros(8, 64, device="cuda")
    with pytest.raises(ValueError, match="y must have shape"):
        mk.muon_combine(y[:6], ids)
    with pytest.raises(ValueError, match="weights"):
        mk.muon_combine(y, ids, torch.zeros(4, 3, device="cuda"))
    with pytest.raises(TypeError, match="weights"):
        mk.muon_combine(y, ids, torch.zeros(4, 2, device="cuda").bfloat16())
    with pytest.raises(TypeError, match="y must be"):
        mk.muon_combine_backward(x, y.bfloat16(), ids, torch.zeros(4, 2, device="cuda"))
    with pytest.raises(mk.MuonError, match="INVALID"):
        mk.muon_combine_backward(x, y, ids, torch.zeros(4, 2, device="cuda"), need_dy=False, need_dweights=False)
