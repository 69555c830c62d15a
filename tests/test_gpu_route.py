"""A router's choice of experts, its weights and their gradient, against 64 bits.

Bounds.  A score is an exponential, a sum and a division in fp32: within 2^-21
of itself, and a softmax's sum of up to 1024 positive terms within 36
roundings, 2^-18 together; a difference x - m of fp32 logits is exact to
2^-24 |x - m|, in the exponential absolutely, with |x - m| < 32 here 2^-19.
Weights divide two such: 2^-16 of themselves.  The gradient multiplies a few
of them: 2^-15 of the sum of its terms' magnitudes, and its type's rounding.
"""

import math

import pytest
import torch

from tests._util import require_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = math.inf
KINDS = [(s, n) for s in ("softmax", "sigmoid") for n in (True, False)]


@pytest.fixture(scope="module")
def mk():
    return require_gpu()


def inputs(T, E, dt, seed=0, masked=True):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + E)
    x = torch.randn(T, E, generator=g, device="cuda") * 2
    if masked and E > 3:
        x[torch.rand(T, E, generator=g, device="cuda") < 0.1] = -INF
        if T > 2:
            x[1] = -INF
            x[2, 1:] = -INF
    return x.to(dt), torch.randn(E, generator=g, device="cuda") * 0.05


def score64(x, score):
    x = x.double()
    if score == "sigmoid":
        return x.sigmoid()
    return torch.where((x > -INF).any(1, keepdim=True), x, 0.0).softmax(1)


def chosen64(x, bias, score, top):
    key = x.double() if bias is None else score64(x, score) + bias.double()
    key = torch.where((x > -INF) & (True if bias is None else bias > -INF), key, -INF)
    values, ids = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(values[:, :top] > -INF, ids[:, :top], -1)


def weights64(x, ids, score, normalize, scale):
    w = torch.where(ids >= 0, score64(x, score).gather(1, ids.clamp(min=0)), 0.0)
    if normalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return scale * w


SIZES = [(1, 1, 1), (3, 2, 2), (9, 31, 4), (5, 33, 32), (1, 64, 8), (300, 100, 6), (7, 129, 1), (1000, 384, 8),
         (2, 511, 32), (33, 1000, 16), (6, 1024, 8)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("score,normalize", KINDS)
@pytest.mark.parametrize("T,E,top", SIZES)
def test_choice_and_weights(mk, T, E, top, score, normalize, bias, dt):
    x, b = inputs(T, E, DT[dt])
    b = b if bias else None
    got = mk.muon_route(x, top, bias=b, score=score, normalize=normalize, scale=2.5)
    assert mk.muon_get_device_status() == 0
    ids = chosen64(x, b, score, top)
    assert got.ids.dtype is torch.int64 and torch.equal(got.ids, ids)
    want = weights64(x, ids, score, normalize, 2.5)
    assert got.weights.dtype is torch.float32
    assert bool(((got.weights.double() - want).abs() <= 2.0 ** -16 * want.abs()).all())


def test_equal_logits_take_the_lowest_index(mk):
    x = torch.zeros(3, 200, device="cuda", dtype=torch.bfloat16)
    x[1, 150:] = 1.0
    x[2, ::2] = -0.0                                   # equal to 0
    for bias in (None, torch.zeros(200, device="cuda")):
        ids = mk.muon_route(x, 8, bias=bias, score="sigmoid").ids.cpu()
        assert ids[0].tolist() == list(range(8)) and ids[1].tolist() == list(range(150, 158))
        assert ids[2].tolist() == list(range(8))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sums_that_fp32_cannot_tell_apart(mk, score):
    """Pairs of experts whose s + bias differ by about 1e-9, at the border of the choice and inside it."""
    g = torch.Generator(device="cuda").manual_seed(5)
    T, E = 2000, 40
    bias = torch.rand(E, generator=g, device="cuda") * 0.2
    x = torch.randn(T, E, generator=g, device="cuda") * 0.3 - 3
    if score == "sigmoid":
        first, second = torch.randperm(E, generator=g, device="cuda")[:2].tolist()
        x[:, first] = 1.0 + 0.5 * torch.rand(T, generator=g, device="cuda")
        s = x[:, first].double().sigmoid() + bias[first].double() - bias[second].double()
        x[:, second] = torch.logit(s).float()           # the nearest fp32 logit: sums within 2^-25 or so
    else:
        x[:, 7] = x[:, 30]
        bias[30] = bias[7] = 0.3
        x[::2, 7] = torch.nextafter(x[::2, 7], torch.full_like(x[::2, 7], INF))
        x[1::4, 30] = torch.nextafter(x[1::4, 30], torch.full_like(x[1::4, 30], INF))
    for top in (1, 2, 5):
        assert torch.equal(mk.muon_route(x, top, bias=bias, score=score).ids, chosen64(x, bias, score, top))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bias", ["none", "zeros", "levels", "near", "infinite"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,top", [(16, 2), (30, 1), (64, 8), (70, 1), (128, 8), (200, 32), (384, 8), (384, 31), (1000, 16), (1024, 32)])
def test_many_equal_keys(mk, E, top, score, bias, dt):
    """Logits and biases of a few levels each, so that hundreds of keys meet at the border of the choice."""
    g = torch.Generator(device="cuda").manual_seed(E + top)
    T = 200
    x = torch.randint(-2, 3, (T, E), generator=g, device="cuda").float()
    x[0] = 0.0                                         # a router before its first step
    x[1], x[1, top // 2:] = 1.0, -0.0
    x[2], x[2, -top:] = -INF, 0.5                      # as many as are asked for
    x[3], x[3, E // 2] = torch.finfo(torch.bfloat16).min, -INF
    x[4], x[4, :40] = 3.0, INF if score == "sigmoid" else 3.5
    x[100:150] = torch.randn(50, E, generator=g, device="cuda")
    x = x.to(DT[dt])
    b = {"none": None, "zeros": torch.zeros(E, device="cuda"),
         "levels": torch.randint(0, 3, (E,), generator=g, device="cuda") * 0.125,
         # sums a step or two apart, which only 64 bits put in order
         "near": 0.25 + torch.randint(0, 3, (E,), generator=g, device="cuda") * 2.0 ** -25,
         "infinite": torch.where(torch.rand(E, generator=g, device="cuda") < 0.3, INF, 0.0)}[bias]
    if bias == "infinite":
        b[::7] = -INF
    got = mk.muon_route(x, top, bias=b, score=score)
    ids = chosen64(x, b, score, top)
    assert torch.equal(got.ids, ids)
    want = weights64(x, ids, score, True, 1.0)
    assert bool(((got.weights.double() - want).abs() <= 2.0 ** -16 * want.abs()).all())


@pytest.mark.parametrize("spread", [0.3, 3.0])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,top", [(60000, 64, 8), (30000, 100, 16), (20000, 384, 8), (20000, 1000, 32)])
def test_many_rows_choose_as_64_bits(mk, T, E, top, score, spread):
    """So many rows that some hold sums which meet by chance, of unlike scores and biases."""
    g = torch.Generator(device="cuda").manual_seed(E)
    x = torch.randn(T, E, generator=g, device="cuda") * spread
    b = torch.randn(E, generator=g, device="cuda") * (2.0 / E if score == "softmax" else 0.1)
    assert torch.equal(mk.muon_route(x, top, bias=b, score=score).ids, chosen64(x, b, score, top))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_more_candidates_than_lanes_at_the_border(mk, score):
    # sums with a bias of 1000 are multiples of 2^-14 in fp32: nearly all are equal there, none in 64 bits
    x = torch.arange(100, device="cuda").flip(0).repeat(3, 1) * 2.0 ** -13
    x = x[:, torch.randperm(100, generator=torch.Generator().manual_seed(1)).cuda()].contiguous()
    bias = torch.full((100,), 1000.0, device="cuda")
    for top in (1, 8, 32):
        assert torch.equal(mk.muon_route(x, top, bias=bias, score=score).ids, chosen64(x, bias, score, top))


def test_masks(mk):
    E = 96
    low = torch.finfo(torch.float32).min
    x = torch.randn(6, E, generator=torch.Generator().manual_seed(3)).cuda()
    x[0] = -INF                     # nothing is left
    x[1, 3:] = -INF                 # fewer than are asked for
    x[2, 5:] = low                  # the type's lowest value is a logit like any other
    x[3] = low
    for score, normalize in KINDS:
        got = mk.muon_route(x, 8, score=score, normalize=normalize)
        ids = chosen64(x, None, score, 8)
        assert torch.equal(got.ids, ids)
        assert got.ids[0].tolist() == [-1] * 8 and sorted(got.ids[1].tolist()[:3]) == [0, 1, 2]
        assert got.ids[1].tolist()[3:] == [-1] * 5
        assert not bool(got.weights[0].any()) and not bool(got.weights[1, 3:].any())
        want = weights64(x, ids, score, normalize, 1.0)
        assert bool(((got.weights.double() - want).abs() <= 2.0 ** -16 * want.abs()).all())
    # a bias of -inf switches an expert off
    bias = torch.zeros(E, device="cuda")
    bias[:90] = -INF
    ids = mk.muon_route(x, 8, bias=bias).ids
    assert torch.equal(ids, chosen64(x, bias, "softmax", 8)) and int(ids[4].max()) >= 90 and ids[4, 6:].tolist() == [-1, -1]


def test_nan_and_infinity_stay_in_their_row(mk):
    x, b = inputs(6, 200, torch.float32, masked=False)
    clean = x.clone()
    x[1, 77] = math.nan
    x[3, 5] = INF
    for score, normalize in KINDS:
        for bias in (None, b):
            got = mk.muon_route(x, 4, bias=bias, score=score, normalize=normalize)
            want = mk.muon_route(clean, 4, bias=bias, score=score, normalize=normalize)
            keep = [0, 2, 4, 5]
            assert torch.equal(got.ids[keep], want.ids[keep]) and torch.equal(got.weights[keep], want.weights[keep])
            assert int(got.ids.min()) >= -1 and int(got.ids.max()) < 200
            assert bool(got.weights[1].isnan().any())
            if bias is None:
                assert int(got.ids[1, 0]) == 77 and int(got.ids[3, 0]) == 5


def grad64(x, ids, dw, score, normalize, scale):
    """(gradient, magnitudes of its terms), by rows; slots of one expert add up."""
    given = ids >= 0
    at = ids.clamp(min=0)
    p = score64(x, score)
    p = torch.where(x > -INF, p, 0.0)
    s = torch.where(given, p.gather(1, at), 0.0)
    g = torch.where(given, scale * dw.double(), 0.0)
    if normalize:
        total = s.sum(1, keepdim=True)
        share = torch.where(total > 0, s / total, 0.0)
        spread = (share[:, None, :] * (g[:, :, None] - g[:, None, :]))
        v, m = share * spread.sum(2), share * spread.abs().sum(2)
        if score == "sigmoid":
            q = torch.where(given, (-x.double()).sigmoid().gather(1, at), 0.0)
            v, m = v * q, m * q
    elif score == "sigmoid":
        q = torch.where(given, (-x.double()).sigmoid().gather(1, at), 0.0)
        v = g * s * q
        m = v.abs()
    else:
        dp = torch.zeros_like(p).scatter_add_(1, at, g)
        # p_e sum_v p_v (dp_e - dp_v)
        want = torch.stack([pr * ((pr[None, :] * (d[:, None] - d[None, :])).sum(1)) for pr, d in zip(p, dp)])
        mags = torch.stack([pr * ((pr[None, :] * (d[:, None] - d[None, :]).abs()).sum(1)) for pr, d in zip(p, dp)])
        return want, mags
    zero = torch.zeros_like(p)
    return zero.scatter_add(1, at, torch.where(given, v, 0.0)), zero.scatter_add(1, at, torch.where(given, m, 0.0))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("score,normalize", KINDS)
@pytest.mark.parametrize("T,E,top", [s for s in SIZES if s[0] <= 300])
def test_gradient(mk, T, E, top, score, normalize, dt):
    x, _ = inputs(T, E, DT[dt], seed=1)
    ids = mk.muon_route(x, top, score=score, normalize=normalize).ids
    dw = torch.randn(T, top, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
    if top > 2:
        ids[0, 1] = ids[0, 0]                           # the same expert twice
    got = mk.muon_route_backward(dw, x, ids, score=score, normalize=normalize, scale=2.5)
    assert mk.muon_get_device_status() == 0 and got.dtype is DT[dt]
    want, mags = grad64(x, ids, dw, score, normalize, 2.5)
    unit = torch.finfo(DT[dt]).eps / 2
    assert bool(((got.double() - want).abs() <= unit * want.abs() + 2.0 ** -15 * mags + 1e-37).all())
    over = x.clone()
    mk.muon_route_backward(dw, over, ids, score=score, normalize=normalize, scale=2.5, out=over)
    assert torch.equal(over, got)


@pytest.mark.parametrize("score,normalize", KINDS)
def test_gradient_agrees_with_differences(mk, score, normalize):
    x, _ = inputs(5, 37, torch.float32, seed=2, masked=False)
    ids = mk.muon_route(x, 6, score=score).ids
    dw = torch.randn(5, 6, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    got = mk.muon_route_backward(dw, x, ids, score=score, normalize=normalize, scale=1.5).double()
    v = torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda", dtype=torch.float64)
    slope = 0.0
    for sign in (1, -1):
        w = weights64(x.double() + sign * 1e-5 * v, ids, score, normalize, 1.5)
        slope += sign * float((w * dw.double()).sum()) / 2e-5
    assert abs(float((got * v).sum()) - slope) <= 2.0 ** -12 * float(got.norm() * v.norm())


def test_one_score_that_is_nearly_all_of_the_sum(mk):
    """Gradients of scores next to 1 keep their relative precision."""
    x = torch.zeros(2, 20, device="cuda")
    x[:, 4] = 14.0
    dw = torch.tensor([[1.0, -2.0, 0.5], [0.3, 0.3, 0.3]], device="cuda")
    for score, normalize in KINDS:
        ids = mk.muon_route(x, 3, score=score).ids
        got = mk.muon_route_backward(dw, x, ids, score=score, normalize=normalize).double()
        want, _ = grad64(x, ids, dw, score, normalize, 1.0)
        assert bool(((got - want).abs() <= 2.0 ** -14 * want.abs() + 1e-12).all()), (score, normalize)


def test_ids_out_of_range_are_reported(mk):
    x, _ = inputs(4, 50, torch.float32, masked=False)
    dw = torch.ones(4, 3, device="cuda")
    ids = mk.muon_route(x, 3).ids
    bad = ids.clone()
    bad[1, 2] = 50
    bad[2, 0] = 1 << 40
    dropped = torch.where(bad >= 50, -1, bad)
    for score, normalize in KINDS:
        got = mk.muon_route_backward(dw, x, bad, score=score, normalize=normalize)
        assert mk.muon_get_device_status() == -6
        assert torch.equal(got, mk.muon_route_backward(dw, x, dropped, score=score, normalize=normalize))
        assert mk.muon_get_device_status() == 0


def test_strides_and_offsets(mk):
    base, b = inputs(40, 130, torch.float32)
    for dt in DT.values():
        wide = torch.full((40, 151), 7.0, device="cuda", dtype=dt)
        view = wide[:, 3:133]
        view.copy_(base)
        want = mk.muon_route(view.contiguous(), 5, bias=b)
        got = mk.muon_route(view, 5, bias=b)
        assert torch.equal(got.ids, want.ids) and torch.equal(got.weights, want.weights)
        dw = torch.randn(40, 5, device="cuda")
        out = torch.full((40, 151), 9.0, device="cuda", dtype=dt)
        mk.muon_route_backward(dw, view, got.ids, out=out[:, 5:135], normalize=False)
        assert torch.equal(out[:, 5:135], mk.muon_route_backward(dw, view.contiguous(), got.ids, normalize=False))
        assert bool((out[:, :5] == 9).all()) and bool((out[:, 135:] == 9).all())


def test_no_rows(mk):
    x = torch.empty(0, 16, device="cuda")
    got = mk.muon_route(x, 4)
    assert got.ids.shape == (0, 4) and got.weights.shape == (0, 4)
    assert mk.muon_route_backward(got.weights, x, got.ids).shape == (0, 16)


def test_refusals(mk):
    x = torch.zeros(4, 64, device="cuda")
    for bad, message in ((lambda: mk.muon_route(x, 0), "INVALID"), (lambda: mk.muon_route(x, 65), "INVALID"),
                         (lambda: mk.muon_route(x, 33), "UNSUPPORTED"),
                         (lambda: mk.muon_route(torch.zeros(2, 1030, device="cuda"), 2), "UNSUPPORTED")):
        with pytest.raises(mk.MuonError, match=message):
            bad()
    with pytest.raises(TypeError, match="torch.bfloat16 or torch.float32"):
        mk.muon_route(x.half(), 2)
    with pytest.raises(TypeError, match="bias"):
        mk.muon_route(x, 2, bias=torch.zeros(64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="bias"):
        mk.muon_route(x, 2, bias=torch.zeros(63, device="cuda"))
    with pytest.raises(ValueError, match="logits"):
        mk.muon_route(x[0], 2)
    with pytest.raises(ValueError, match="last axis"):
        mk.muon_route(x.T, 2)
    ids = torch.zeros(4, 2, device="cuda", dtype=torch.int64)
    with pytest.raises(ValueError, match="dweights"):
        mk.muon_route_backward(torch.zeros(4, 3, device="cuda"), x, ids)
    with pytest.raises(TypeError, match="ids"):
        mk.muon_route_backward(torch.zeros(4, 2, device="cuda"), x, ids.int())


def test_a_refused_count_allocates_nothing(mk):
    x = torch.zeros(4000, 64, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.max_memory_allocated()
    with pytest.raises(mk.MuonError, match="INVALID"):
        mk.muon_route(x, 1_000_000)
    assert torch.cuda.max_memory_allocated() - before < 1 << 24
