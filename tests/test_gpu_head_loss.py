"""Softmax cross entropy over a head matrix without logits, and its gradients, against 64 bits.

Bounds.  z: products of bf16 are exact in fp32, hidden of them are added in
steps of 16 in the tensor core, each step within 2^-22 of the magnitudes S =
sum |x w| so far (its alignment truncates): ez = (hidden / 16 + 4) 2^-22 S.
lse: the largest ez of a row; a term's exponential within 2^-20 of itself; its
sums of at most 2^6 terms in turn, joined in 2^6 steps and a tree: 2^-17; its
own rounding, 2^-23 |lse|.  The gradient's d is rounded to bf16 (2^-8), its p
are within ez + 2^-19 + 2^-23 |lse| of themselves; products with W or x add
these up against |W| or |x|, their sums of n terms another (n / 16 + 4) 2^-22
of the magnitudes, and dx and dW are rounded to bf16 once.  Those are bounds on
every element; roundings that go either way leave less in all: each of the two
is 2^-8 / sqrt(3) at worst in the norm, so 2^-8 for the whole, and what the
errors of p bring besides.  (Logits of thousands: fp32 holds lse = 3424 to 2^-13,
so a p next to 1 is within 1e-4 of itself and d = p - 1 = 1e-9 has no digit right,
whatever computes it from that lse.)
"""

import math

import pytest
import torch

from tests._util import require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def mk():
    return require_gpu()


def inputs(T, V, H, seed=0, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 3 * T + 5 * V + H)
    w = (torch.randn(V, H, generator=g, device="cuda") * std * H ** -0.5).to(BF)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = (torch.randn(T, H, generator=g, device="cuda") + w[t].float()).to(BF)
    if T > 3:
        t[2] = -1
        t[T - 1] = -7
    dl = torch.rand(T, generator=g, device="cuda") + 0.5
    dz = torch.randn(T, generator=g, device="cuda") * 0.1
    return x, w, t, dl, dz


def by_rows(T, V):
    n = max(1, (1 << 27) // V)
    return [slice(a, min(T, a + n)) for a in range(0, T, n)]


def check_forward(got, x, w, t):
    V, H = w.shape
    wd = w.double()
    for s in by_rows(len(t), V):
        z = x[s].double() @ wd.T
        ez = (H / 16 + 4) * 2.0 ** -22 * (x[s].double().abs() @ wd.abs().T).amax(1)
        lse = torch.logsumexp(z, 1)
        zt = z.gather(1, t[s].clamp(min=0)[:, None])[:, 0]
        loss = torch.where(t[s] >= 0, lse - zt, 0.0)
        tol = 2 * ez + 2.0 ** -17 + 2.0 ** -23 * (lse.abs() + zt.abs())
        assert bool(((got.lse[s].double() - lse).abs() <= tol).all())
        assert bool(((got.loss[s].double() - loss).abs() <= tol).all())


def check_backward(got, x, w, t, lse, dl, dz, which=(True, True)):
    T, (V, H) = len(t), w.shape
    wd, wa = w.double(), w.double().abs()
    dw, bw = torch.zeros_like(wd), torch.zeros_like(wd)
    errs, ew = [], torch.zeros_like(wd)
    for s in by_rows(T, V):
        xd = x[s].double()
        on = (t[s] >= 0).double()[:, None]
        xd = torch.where(on > 0, xd, 0.0)
        z = xd @ wd.T
        p = (z - lse[s].double()[:, None]).exp()
        g = on * (dl[s].double() + (dz[s].double() if dz is not None else 0.0))[:, None]
        hit = torch.zeros_like(p).scatter_(1, t[s].clamp(min=0)[:, None], 1.0) * on * dl[s].double()[:, None]
        d = g * p - hit
        ep = (H / 16 + 4) * 2.0 ** -22 * (xd.abs() @ wa.T) + 2.0 ** -19 + 2.0 ** -23 * lse[s].double().abs()[:, None]
        of_p = g.abs() * p * ep
        ed = 2.0 ** -8 * d.abs() + (of_p + 2.0 ** -23 * hit.abs()) * 1.01 + 1e-37
        if which[0]:
            dx = d @ wd
            bound = ed @ wa + (V / 16 + 4) * 2.0 ** -22 * (d.abs() @ wa)
            bound = bound + 2.0 ** -8 * (dx.abs() + bound)
            e = (got[0][s].double() - dx).abs()
            assert bool((e <= bound + 1e-37).all()), float((e / (bound + 1e-37)).max())
            errs.append([float(v.square().sum()) for v in (got[0][s].double() - dx, dx, of_p @ wa)])
        dw += d.T @ xd
        ew += of_p.T @ xd.abs()
        bw += ed.T @ xd.abs() + (T / 16 + 4) * 2.0 ** -22 * (d.abs().T @ xd.abs())
    if which[0]:
        err, norm, more = (sum(v) ** 0.5 for v in zip(*errs))
        assert err <= 2.0 ** -8 * norm + more
    if which[1]:
        bound = bw + 2.0 ** -8 * (dw.abs() + bw) + 1e-37
        e = (got[1].double() - dw).abs()
        assert bool((e <= bound).all()), float((e / bound).max())
        assert float((got[1].double() - dw).norm()) <= 2.0 ** -8 * float(dw.norm()) + float(ew.norm())


# one row to several row tiles; vocabularies that end inside a tile, of one entry, of many tiles for few rows;
# widths of one swizzle row and less, not a multiple of 64, wider than a tile
SIZES = [(1, 1, 8), (1, 7, 16), (3, 100, 64), (5, 257, 72), (128, 512, 128), (129, 1000, 1000), (300, 5003, 136),
         (40, 50003, 256), (257, 30011, 64), (777, 777, 520), (2, 128000, 320), (1025, 4096, 264)]


@pytest.mark.parametrize("T,V,H", SIZES)
def test_forward(mk, T, V, H):
    x, w, t, _, _ = inputs(T, V, H)
    got = mk.muon_head_loss(x, w, t)
    assert mk.muon_get_device_status() == 0
    assert got.loss.dtype is torch.float32 and got.lse.dtype is torch.float32
    check_forward(got, x, w, t)


@pytest.mark.parametrize("T,V,H", SIZES)
def test_backward(mk, T, V, H):
    x, w, t, dl, dz = inputs(T, V, H, seed=1)
    lse = mk.muon_head_loss(x, w, t).lse
    got = mk.muon_head_loss_backward(dl, x, w, t, lse, dlse=dz)
    assert mk.muon_get_device_status() == 0 and got[0].dtype is BF and got[1].dtype is BF
    check_backward(got, x, w, t, lse, dl, dz)
    if T > 3:
        assert not bool(got[0][2].any()) and not bool(got[0][T - 1].any())
    # without dlse, and each gradient alone
    plain = mk.muon_head_loss_backward(dl, x, w, t, lse)
    check_backward(plain, x, w, t, lse, dl, None)
    one = mk.muon_head_loss_backward(dl, x, w, t, lse, need_dweight=False)
    two = mk.muon_head_loss_backward(dl, x, w, t, lse, need_dx=False)
    assert one[1] is None and two[0] is None and torch.equal(two[1], plain[1])
    check_backward(one, x, w, t, lse, dl, None, which=(True, False))


def test_pieces_of_the_vocabulary(mk):
    """A call whose vocabulary is cut, the last piece short: dx is added up over the pieces."""
    T, V, H = 8200, 20003, 72
    x, w, t, dl, dz = inputs(T, V, H)
    got = mk.muon_head_loss(x, w, t)
    check_forward(got, x, w, t)
    grads = mk.muon_head_loss_backward(dl, x, w, t, got.lse, dlse=dz)
    assert mk.muon_get_device_status() == 0
    check_backward(grads, x, w, t, got.lse, dl, dz)
    again = mk.muon_head_loss_backward(dl, x, w, t, got.lse, dlse=dz)
    assert torch.equal(grads[0], again[0]) and torch.equal(grads[1], again[1])
    alone = mk.muon_head_loss_backward(dl, x, w, t, got.lse, dlse=dz, need_dweight=False)   # cut K besides
    check_backward(alone, x, w, t, got.lse, dl, dz, which=(True, False))


@pytest.mark.parametrize("T,V,H", [(5000, 2500, 6144), (8192, 1003, 6144)])
def test_more_row_tiles_than_a_group(mk, T, V, H):
    """Row tiles whose x outgrows a group's share of L2 (16 of them here): a shorter last group, and whole ones.  Sums of 96
    k-blocks, many turns of the ring."""
    x, w, t, dl, dz = inputs(T, V, H)
    got = mk.muon_head_loss(x, w, t)
    check_forward(got, x, w, t)
    grads = mk.muon_head_loss_backward(dl, x, w, t, got.lse, dlse=dz)
    assert mk.muon_get_device_status() == 0
    check_backward(grads, x, w, t, got.lse, dl, dz)


def test_gradients_of_more_rows_than_a_forward_pass(mk):
    T, V, H = 17000, 20003, 24                                  # pieces of the vocabulary besides
    x, w, t, dl, dz = inputs(T, V, H)
    got = mk.muon_head_loss(x, w, t)
    check_forward(got, x, w, t)
    grads = mk.muon_head_loss_backward(dl, x, w, t, got.lse, dlse=dz)
    assert mk.muon_get_device_status() == 0
    check_backward(grads, x, w, t, got.lse, dl, dz)


def test_rows_of_several_passes(mk):
    T, V, H = 16384 * 2 + 5, 700, 24
    x, w, t, _, _ = inputs(T, V, H)
    check_forward(mk.muon_head_loss(x, w, t), x, w, t)
    assert mk.muon_get_device_status() == 0


@pytest.mark.parametrize("T,V,H", [(513, 120000, 8), (700, 40000, 64), (1025, 60001, 16)])
def test_row_tiles_that_end_early_between_others(mk, T, V, H):
    """A pair of CTAs goes from a row tile with rows to one without for most of its warps and back, many times."""
    x, w, t, _, _ = inputs(T, V, H)
    got = mk.muon_head_loss(x, w, t)
    assert mk.muon_get_device_status() == 0
    check_forward(got, x, w, t)
    for _ in range(20):
        again = mk.muon_head_loss(x, w, t)
        assert torch.equal(again.loss, got.loss) and torch.equal(again.lse, got.lse)


def test_weight_past_32_bits(mk):
    T, V, H = 4, 360001, 6144                                   # 2.2e9 elements
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.empty(V, H, device="cuda", dtype=BF)
    for a in range(0, V, 40000):
        b = min(V, a + 40000)
        w[a:b] = (torch.randn(b - a, H, generator=g, device="cuda") * 0.02).to(BF)
    t = torch.tensor([V - 1, 0, V // 2, -1], device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda").to(BF)
    got = mk.muon_head_loss(x, w, t)
    z = torch.cat([x.double() @ w[a:a + 40000].double().T for a in range(0, V, 40000)], 1)
    lse = torch.logsumexp(z, 1)
    loss = torch.where(t >= 0, lse - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    assert float((got.lse.double() - lse).abs().max()) < 1e-3 and float((got.loss.double() - loss).abs().max()) < 1e-3
    dl = torch.ones(T, device="cuda")
    dx, dw = mk.muon_head_loss_backward(dl, x, w, t, got.lse)
    assert mk.muon_get_device_status() == 0
    d = ((z - got.lse.double()[:, None]).exp()).scatter_add_(1, t.clamp(min=0)[:, None], -torch.ones(T, 1, device="cuda", dtype=torch.float64))
    d[3] = 0
    last = slice(V - 300, V)
    want = d[:, last].T @ x.double()
    assert float((dw[last].double() - want).norm()) <= 2.0 ** -8 * float(want.norm())
    want = sum(d[:, a:a + 40000] @ w[a:a + 40000].double() for a in range(0, V, 40000))
    assert float((dx.double() - want).norm()) <= 2.0 ** -8 * float(want.norm())


def test_gradient_agrees_with_differences(mk):
    x, w, t, dl, dz = inputs(6, 50, 16)
    lse = mk.muon_head_loss(x, w, t).lse
    dx, dw = mk.muon_head_loss_backward(dl, x, w, t, lse, dlse=dz)
    g = torch.Generator(device="cuda").manual_seed(4)
    vx = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
    vw = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
    on = t >= 0
    slope = 0.0
    for sign in (1, -1):
        z = (x.double() + sign * 1e-5 * vx) @ (w.double() + sign * 1e-5 * vw).T
        l = torch.logsumexp(z, 1)
        ce = l - z.gather(1, t.clamp(min=0)[:, None])[:, 0]
        slope += sign * float((torch.where(on, dl.double() * ce + dz.double() * l, 0.0)).sum()) / 2e-5
    got = float((dx.double() * vx).sum() + (dw.double() * vw).sum())
    norms = float(dx.double().norm() * vx.norm() + dw.double().norm() * vw.norm())
    assert abs(got - slope) <= 2.0 ** -8 * norms


def test_rows_that_take_no_part(mk):
    """Padding may hold anything; a row whose factors are 0 adds nothing."""
    T, V, H = 300, 1000, 128
    x, w, t, dl, dz = inputs(T, V, H)
    pad = torch.rand(T, generator=torch.Generator().manual_seed(1)).cuda() < 0.3
    t[pad] = -1
    lse = mk.muon_head_loss(x, w, t).lse
    want = mk.muon_head_loss_backward(dl, x, w, t, lse, dlse=dz)
    x2, lse2, dl2, dz2 = x.clone(), lse.clone(), dl.clone(), dz.clone()
    x2[pad], dl2[pad], dz2[pad], lse2[pad] = float("nan"), float("inf"), float("nan"), float("nan")
    f = mk.muon_head_loss(x2, w, t)
    assert not bool(f.loss[pad].any()) and torch.equal(f.lse[~pad], lse[~pad])
    got = mk.muon_head_loss_backward(dl2, x2, w, t, lse2, dlse=dz2)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not bool(got[0][pad].any())
    none = torch.full_like(t, -1)
    got = mk.muon_head_loss_backward(dl, x2, w, none, lse2)
    assert not bool(got[0].any()) and not bool(got[1].any())


def test_a_nan_row_stays_a_row(mk):
    T, V, H = 300, 3000, 64
    x, w, t, dl, _ = inputs(T, V, H)
    clean = mk.muon_head_loss(x, w, t)
    x[5, 3], x[200, 0] = float("nan"), float("inf")
    t[5], t[200] = 4, 9
    got = mk.muon_head_loss(x, w, t)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[5] = keep[200] = False
    assert torch.equal(got.loss[keep], clean.loss[keep]) and torch.equal(got.lse[keep], clean.lse[keep])
    assert bool(got.loss[~keep].isnan().all()) and bool(got.lse[~keep].isnan().all())
    dx, _ = mk.muon_head_loss_backward(dl, x, w, t, got.lse)
    assert bool(dx[~keep].isnan().all()) and not bool(dx[keep].isnan().any())


def test_large_logits(mk):
    # logits of several hundred: the largest is the reference, no exponential overflows
    x, w, t, dl, _ = inputs(70, 900, 64, std=60.0)
    got = mk.muon_head_loss(x, w, t)
    assert float(got.lse.max()) > 200 and bool(got.loss.isfinite().all())
    check_forward(got, x, w, t)
    check_backward(mk.muon_head_loss_backward(dl, x, w, t, got.lse), x, w, t, got.lse, dl, None)


def exact_logits(V, power, seed=0):
    """x, weight, targets and logits in 64 bits whose products have one term each: z is exact, with many equal ones.

    Of each eight rows the last has negative logits alone; every other target is the largest logit.
    """
    g = torch.Generator(device="cuda").manual_seed(seed + V)
    w = torch.randn(V, 8, generator=g, device="cuda").clamp(-3.9, 3.9).to(BF)
    w[:, 7] = -w[:, 7].abs() - 0.0625
    x = torch.zeros(24, 8, device="cuda", dtype=BF)
    x[torch.arange(24), torch.arange(24) % 8] = 2.0 ** power
    z = x.double() @ w.double().T
    t = torch.randint(0, V, (24,), generator=g, device="cuda")
    t[::2] = z[::2].argmax(1)
    return x, w, t, z


# below 2^23 and above, around 2^30 and up to the largest that are allowed
@pytest.mark.parametrize("power", [0, 8, 20, 23, 25, 28, 29, 30, 31, 33, 50, 100, 124])
@pytest.mark.parametrize("V", [1, 40, 300, 5003])
def test_logits_of_any_size(mk, V, power):
    """Bounds as above without z's error: 2^-17, and what rounds the results themselves."""
    x, w, t, z = exact_logits(V, power)
    got = mk.muon_head_loss(x, w, t)
    lse = torch.logsumexp(z, 1)
    most = z.amax(1)
    loss = (most - z.gather(1, t[:, None])[:, 0]) + (z - most[:, None]).exp().sum(1).log()
    assert bool(((got.lse.double() - lse).abs() <= 2.0 ** -17 + 2.0 ** -22 * lse.abs()).all())
    assert bool(((got.loss.double() - loss).abs() <= 2.0 ** -17 + 2.0 ** -21 * loss.abs()).all())


def test_logits_of_minus_infinity(mk):
    """Columns that no row takes, a whole tile's share of them among others; a row with nothing else has lse -inf."""
    x, w, t, _ = exact_logits(5003, 3)
    x[:, 1:], x[:, 0] = 0.0, 1.0
    w[64:96, 0] = w[100:1000:3, 0] = w[1024:2048, 0] = -math.inf
    w[5000, 0] = 1.0
    t[:] = 5000
    z = w[:, 0].double()
    got = mk.muon_head_loss(x, w, t)
    lse = float(torch.logsumexp(z, 0))
    assert float((got.lse.double() - lse).abs().max()) <= 2.0 ** -17 + 2.0 ** -22 * abs(lse)
    assert float((got.loss.double() - (lse - 1.0)).abs().max()) <= 2.0 ** -17 + 2.0 ** -21 * abs(lse)
    w[:, 0] = -math.inf
    assert bool((mk.muon_head_loss(x, w, t).lse == -math.inf).all())


@pytest.mark.parametrize("power", [8, 13, 20, 23, 28, 31, 50, 100])
def test_gradients_of_certain_targets(mk, power):
    """Where the target's logit is lse itself and the others far below, p is 1 and d nothing but what dlse adds."""
    V = 40
    x = torch.zeros(24, 8, device="cuda", dtype=BF)
    x[torch.arange(24), torch.arange(24) % 8] = 2.0 ** power
    t = torch.arange(24, device="cuda") % 8 + 11
    w = torch.zeros(V, 8, device="cuda", dtype=BF)
    w[11 + torch.arange(8), torch.arange(8)] = (1 + torch.arange(8, device="cuda") * 2.0 ** -7 * 9).to(BF)
    lse = (x.float() @ w.float().T).amax(1)             # one term each: exact
    assert float(lse.min()) > 104                       # exp(-lse) is nothing in fp32
    one, dz = torch.ones(24, device="cuda"), torch.rand(24, device="cuda")
    dx, dw = mk.muon_head_loss_backward(one, x, w, t, lse)
    assert not bool(dx.any()) and not bool(dw.any())
    # d = dlse at the target, which dx and dw have as their one term: roundings of d and of the results
    dx, dw = mk.muon_head_loss_backward(one, x, w, t, lse, dlse=dz)
    want = dz.double()[:, None] * w.double()[t]
    assert bool(((dx.double() - want).abs() <= 2.0 ** -6.9 * want.abs() + 2.0 ** -22 * w.double()[t]).all())
    want = torch.zeros(V, 8, device="cuda", dtype=torch.float64).index_add_(0, t, dz.double()[:, None] * x.double())
    most = torch.zeros(V, 8, device="cuda", dtype=torch.float64).index_add_(0, t, x.double())
    assert bool(((dw.double() - want).abs() <= 2.0 ** -6.9 * want.abs() + 2.0 ** -22 * most).all())


@pytest.mark.parametrize("power", [5, 8, 13, 20, 23, 26, 29, 31, 50, 100])
def test_lse_is_rounded_once(mk, power):
    """One logit far above the others: lse is that logit, and a certain target has no gradient through both calls."""
    V = 300
    x = torch.zeros(24, 8, device="cuda", dtype=BF)
    x[torch.arange(24), torch.arange(24) % 8] = 2.0 ** power
    t = torch.arange(24, device="cuda") % 8 + 250
    w = torch.full((V, 8), -1.0, device="cuda", dtype=BF)
    w[250 + torch.arange(8), torch.arange(8)] = (2 + torch.arange(8, device="cuda") * 2.0 ** -6 * 9).to(BF)
    z = x.float() @ w.float().T                         # one term each: exact, 2^5 times 3 apart
    got = mk.muon_head_loss(x, w, t)
    assert torch.equal(got.lse, z.amax(1))              # exp(-96) is nothing beside the rounding of 64
    if power >= 8:
        dx, dw = mk.muon_head_loss_backward(torch.ones(24, device="cuda"), x, w, t, got.lse)
        assert not bool(dx.any()) and not bool(dw.any())


@pytest.mark.parametrize("power", [10, 13, 16, 20])
def test_lse_within_its_own_rounding(mk, power):
    x, w, t, z = exact_logits(5003, power, seed=5)
    lse = torch.logsumexp(z, 1)
    tol = 2.0 ** -17 + 2.0 ** -24 * (1 + 2.0 ** -6) * lse.abs()   # its terms' and sums' part, then one rounding
    assert bool(((mk.muon_head_loss(x, w, t).lse.double() - lse).abs() <= tol).all())


@pytest.mark.parametrize("V", [1, 2, 33, 300, 5003])
def test_losses_are_not_negative(mk, V):
    """Targets that are all of their row's sum, or all but a little: 0 within the exponentials' error, and never below."""
    g = torch.Generator(device="cuda").manual_seed(V)
    T = 3000
    x = torch.zeros(T, 8, device="cuda", dtype=BF)
    x[:, 0] = (5 + 35 * torch.rand(T, generator=g, device="cuda")).to(BF)
    x[:, 1] = (x[:, 0].float() - 8 - 40 * torch.rand(T, generator=g, device="cuda")).to(BF)
    w = torch.zeros(V, 8, device="cuda", dtype=BF)
    w[:, 1] = 1.0
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    w[t[0]], t[:] = torch.tensor([1.0] + 7 * [0.0], device="cuda", dtype=BF), int(t[0])
    got = mk.muon_head_loss(x, w, t)
    z = x.double() @ w.double().T
    zt = z[torch.arange(T), t]
    rest = (z - zt[:, None]).exp()
    rest[torch.arange(T), t] = 0.0
    want = torch.log1p(rest.sum(1))                     # all others are 8 or more below the target
    assert bool((got.loss >= 0).all())
    assert bool(((got.loss.double() - want).abs() <= 2.0 ** -17 + 2.0 ** -21 * want).all())


def test_targets_out_of_range_are_reported(mk):
    x, w, t, dl, _ = inputs(10, 100, 64)
    want = mk.muon_head_loss(x, w, t)
    bad = t.clone()
    bad[4], bad[6] = 100, 1 << 40
    got = mk.muon_head_loss(x, w, bad)
    assert mk.muon_get_device_status() == -6
    assert bool(got.loss[[4, 6]].isnan().all()) and torch.equal(got.lse, want.lse)
    assert torch.equal(got.loss[:4], want.loss[:4])
    grads = mk.muon_head_loss_backward(dl, x, w, bad, got.lse)
    assert mk.muon_get_device_status() == -6
    dropped = torch.where(bad >= 100, -1, bad)
    other = mk.muon_head_loss_backward(dl, x, w, dropped, got.lse)
    assert torch.equal(grads[0], other[0]) and torch.equal(grads[1], other[1]) and mk.muon_get_device_status() == 0


def test_strides_outputs_and_workspaces(mk):
    T, V, H = 200, 3001, 136
    x, w, t, dl, dz = inputs(T, V, H)
    wide = torch.full((T, 160), float("nan"), device="cuda", dtype=BF)
    xs = wide[:, 8:8 + H]
    xs.copy_(x)
    want = mk.muon_head_loss(x, w, t)
    ws = torch.empty(mk.muon_head_loss_workspace_bytes(T, V, H), dtype=torch.uint8, device="cuda")
    got = mk.muon_head_loss(xs, w, t, workspace=ws)
    assert torch.equal(got.loss, want.loss) and torch.equal(got.lse, want.lse)
    grads = mk.muon_head_loss_backward(dl, x, w, t, want.lse, dlse=dz)
    ws = torch.full((mk.muon_head_loss_backward_workspace_bytes(T, V, H),), 255, dtype=torch.uint8, device="cuda")
    dx = torch.full((T, 160), 5.0, device="cuda", dtype=BF)
    dw = torch.full((V, H), 5.0, device="cuda", dtype=BF)
    view = dx[:, 16:16 + H]
    out = mk.muon_head_loss_backward(dl, xs, w, t, want.lse, dlse=dz, dx=view, dweight=dw, workspace=ws)
    assert out[0] is view and out[1] is dw
    assert torch.equal(view, grads[0]) and torch.equal(dw, grads[1])
    assert bool((dx[:, :16] == 5).all()) and bool((dx[:, 16 + H:] == 5).all())
    for f in (lambda: mk.muon_head_loss(x, w, t, workspace=ws[:256]),
              lambda: mk.muon_head_loss_backward(dl, x, w, t, want.lse, workspace=ws[:256])):
        with pytest.raises(mk.MuonError, match="NO_MEMORY"):
            f()


def test_a_copy_that_is_not_made_takes_no_workspace(mk):
    """Rows that begin on 128 bytes are read where they are; so are few rows, and rows over few entries."""
    T, V, H = 300, 50003, 192
    x, w, t, _, _ = inputs(T, V, H)
    wide = torch.zeros(T, 200, device="cuda", dtype=BF)
    off = wide[:, 8:]
    off.copy_(x)
    need = mk.muon_head_loss_workspace_bytes(T, V, H)
    copy = T * H * 2
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = mk.muon_head_loss(off, w, t, workspace=ws)
    got = mk.muon_head_loss(x, w, t, workspace=ws[:need - copy])
    assert torch.equal(got.loss, want.loss) and torch.equal(got.lse, want.lse)
    with pytest.raises(mk.MuonError, match="NO_MEMORY"):
        mk.muon_head_loss(off, w, t, workspace=ws[:need - copy])
    # targets' logits and statistics alone, 8 bytes a row and part of 256 or fewer entries
    for rows, vocab in ((100, 50003), (2000, 300)):
        small = mk.muon_head_loss_workspace_bytes(rows, vocab, 6144)
        assert small <= rows * 4 + rows * -(-vocab // 64) * 8 + 512
        xs, ws_, ts, _, _ = inputs(rows, vocab, 136)    # off 128 bytes
        check_forward(mk.muon_head_loss(xs, ws_, ts, workspace=torch.empty(
            mk.muon_head_loss_workspace_bytes(rows, vocab, 136), dtype=torch.uint8, device="cuda")), xs, ws_, ts)


def test_allocation_failure_launches_nothing(mk):
    x, w, t, dl, _ = inputs(20, 300, 64)
    lse = mk.muon_head_loss(x, w, t).lse
    for f in (lambda: mk.muon_head_loss(x, w, t), lambda: mk.muon_head_loss_backward(dl, x, w, t, lse)):
        mk.muon_inject_alloc_failures(1)
        before = mk.muon_launch_count()
        with pytest.raises(mk.MuonError, match="NO_MEMORY"):
            f()
        assert mk.muon_launch_count() == before and mk.muon_inject_alloc_failures(0) == 0


def test_no_rows(mk):
    w = torch.ones(30, 64, device="cuda", dtype=BF)
    x, t, f = torch.empty(0, 64, device="cuda", dtype=BF), torch.empty(0, device="cuda", dtype=torch.int64), torch.empty(0, device="cuda")
    assert mk.muon_head_loss(x, w, t).loss.shape == (0,)
    dx, dw = mk.muon_head_loss_backward(f, x, w, t, f)
    assert dx.shape == (0, 64) and dw.shape == (30, 64) and not bool(dw.any())


def test_refusals(mk):
    x, w, t, dl, _ = inputs(8, 40, 64)
    lse = torch.zeros(8, device="cuda")
    with pytest.raises(mk.MuonError, match="UNSUPPORTED"):
        mk.muon_head_loss(x[:, :60].contiguous(), w[:, :60].contiguous(), t)
    with pytest.raises(ValueError, match="weight must have shape"):
        mk.muon_head_loss(x, w[:, :32].contiguous(), t)
    with pytest.raises(TypeError, match="x must be"):
        mk.muon_head_loss(x.float(), w, t)
    with pytest.raises(TypeError, match="weight must be"):
        mk.muon_head_loss(x, w.float(), t)
    with pytest.raises(TypeError, match="targets"):
        mk.muon_head_loss(x, w, t.int())
    with pytest.raises(ValueError, match="targets"):
        mk.muon_head_loss(x, w, t[:4])
    with pytest.raises(ValueError, match="weight must be contiguous"):
        mk.muon_head_loss(x, w.T.contiguous().T, t)
    with pytest.raises(mk.MuonError, match="INVALID"):
        mk.muon_head_loss_backward(dl, x, w, t, lse, need_dx=False, need_dweight=False)
    with pytest.raises(ValueError, match="dlse"):
        mk.muon_head_loss_backward(dl, x, w, t, lse, dlse=lse[:3])
    with pytest.raises(ValueError, match="dweight"):
        mk.muon_head_loss_backward(dl, x, w, t, lse, dweight=w[:5])
