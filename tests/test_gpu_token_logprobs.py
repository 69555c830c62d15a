"""Log probabilities of given tokens, entropy, top alternatives and their gradient, against 64 bits.

Bounds.  Sums of up to 2^18 positive terms in fp32, a thread adding at most
2^10 and the rest in a tree: within 2^-13 at worst and 2^-16 where the
roundings' signs differ, as here (2^-16 taken for the sums, so for lse
absolutely).  x - m and x - lse round to 2^-24 of the logits' magnitude.  A
weight exp(t) is within 2^-22 (1 + |t|) of itself.  The gradient adds its own
type's rounding (2^-9 for bf16).
"""

import math

import pytest
import torch

from tests._util import require_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = math.inf


@pytest.fixture(scope="module")
def mk():
    return require_gpu()


def inputs(T, V, dt, seed=0, std=3.0, masked=True):
    g = torch.Generator(device="cuda").manual_seed(seed + T * 7 + V)
    x = torch.randn(T, V, generator=g, device="cuda") * std
    tok = torch.randint(0, V, (T,), generator=g, device="cuda")
    if masked and V > 4:
        x[torch.rand(T, V, generator=g, device="cuda") < 0.1] = -INF
        x[torch.arange(T, device="cuda"), tok] = 1.0
    if T > 2:
        tok[2] = -1
    return x.to(dt), tok, torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")


def ref64(x):
    x = x.double()
    logp = torch.log_softmax(x, 1)
    p = logp.exp()
    spread = torch.where(p > 0, p * (x - x.amax(1, keepdim=True)).abs(), 0.0).sum(1)
    return logp, p, torch.logsumexp(x, 1), -torch.special.xlogy(p, p).sum(1), spread


def tol(x):
    return 2.0 ** -16 + 2.0 ** -22 * float(x[x.isfinite()].abs().max())


def check_forward(got, x, tok, top):
    logp, p, lse, ent, spread = ref64(x)
    t = tol(x.float())
    assert float((got.lse.double() - lse).abs().max()) <= t
    assert bool(((got.entropy.double() - ent).abs() <= t + 2.0 ** -16 * 2 * (1 + spread)).all())
    want = torch.where(tok >= 0, logp.gather(1, tok.clamp(min=0)[:, None])[:, 0], 0.0)
    assert float((got.logp.double() - want).abs().max()) <= t
    if top:
        ids = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(got.top_ids, ids)
        w = logp.gather(1, ids)
        assert torch.equal(got.top_logp == -INF, w == -INF)
        fin = w > -INF
        assert float((got.top_logp.double() - w)[fin].abs().max()) <= t


SIZES = [(1, 1), (3, 2), (5, 31), (4, 33), (1, 1000), (3, 4099), (2, 16384), (1, 32771), (7, 50003), (4, 131080),
         (1, 262144), (400, 777)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("top", [0, 1, 5, 32])
@pytest.mark.parametrize("T,V", SIZES)
def test_forward(mk, T, V, dt, top):
    top = min(top, V)
    x, tok, _, _ = inputs(T, V, DT[dt])
    got = mk.muon_token_logprobs(x, tok, top=top)
    assert mk.muon_get_device_status() == 0
    check_forward(got, x, tok, top)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", SIZES)
def test_backward(mk, T, V, dt):
    x, tok, dl, de = inputs(T, V, DT[dt], seed=1)
    f = mk.muon_token_logprobs(x, tok)
    logp, p, lse, ent, _ = ref64(x)
    hot = torch.zeros_like(p).scatter_(1, tok.clamp(min=0)[:, None], 1.0)
    given = (tok >= 0).double()[:, None]
    unit = 2.0 ** -8 if dt == "bf16" else 2.0 ** -23
    for a, b in ((dl, None), (None, de), (dl, de)):
        got = mk.muon_token_logprobs_backward(x, tok, f.lse, f.entropy, a, b)
        assert got.dtype is DT[dt]
        da = (a.double()[:, None] if a is not None else 0.0) * given
        db = b.double()[:, None] if b is not None else torch.zeros_like(given)
        pl = torch.special.xlogy(p, p)
        want = da * (hot - p) - db * (pl + p * ent[:, None])
        mags = (da.abs() if a is not None else 0.0) * (hot + p) + db.abs() * (pl.abs() + p * (1 + ent[:, None]))
        # p through x - lse: lse's own bound, and exp's
        bound = unit * want.abs() + 4 * tol(x.float()) * (mags + db.abs() * p) + 1e-30
        err = (got.double() - want).abs()
        assert bool((err <= bound).all()), float((err / bound).max())
    buf = x.clone()
    mk.muon_token_logprobs_backward(buf, tok, f.lse, f.entropy, dl, de, out=buf)   # over the logits
    assert torch.equal(buf, got)


def test_gradient_agrees_with_differences(mk):
    x, tok, dl, de = inputs(4, 37, torch.float32, seed=2, masked=False)
    f = mk.muon_token_logprobs(x, tok)
    got = mk.muon_token_logprobs_backward(x, tok, f.lse, f.entropy, dl, de).double()
    v = torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda",
                    dtype=torch.float64)
    slope = 0.0
    for sign in (1, -1):
        logp, p, lse, ent, _ = ref64(x.double() + sign * 1e-5 * v)
        chosen = torch.where(tok >= 0, logp.gather(1, tok.clamp(min=0)[:, None])[:, 0], 0.0)
        slope += sign * float((chosen * dl.double() + ent * de.double()).sum()) / 2e-5
    assert abs(float((got * v).sum()) - slope) <= 2.0 ** -12 * float(got.norm() * v.norm())


@pytest.mark.parametrize("V", [40, 70000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_masks(mk, V, dt):
    t = DT[dt]
    low = torch.finfo(t).min
    x = torch.randn(8, V, generator=torch.Generator().manual_seed(V)).to(t).cuda()
    x[0] = -INF                  # nothing is left
    x[1, 1:] = -INF              # one entry is left
    x[2] = low                   # a mask of the type's lowest value over everything: uniform
    x[3, :-1] = low              # and over all but one
    x[4] = -INF
    x[4, V - 2:] = torch.tensor([-1e30, -1e30]).to(t)   # two equal, far below zero
    x[5, 3] = float("nan")
    x[6, 5] = INF
    x[7, 9] = torch.finfo(t).max
    tok = torch.tensor([0, 0, 7, V - 1, V - 1, 4, 5, 9], device="cuda")
    got = mk.muon_token_logprobs(x, tok, top=3)
    assert mk.muon_get_device_status() == 0
    lse, logp, ent = (v.tolist() for v in (got.lse, got.logp, got.entropy))
    assert lse[0] == -INF and logp[0] == -INF and ent[0] == 0 and got.top_ids[0].tolist() == [0, 1, 2]
    assert got.top_logp[0].tolist() == [-INF] * 3
    assert logp[1] == 0 and ent[1] == 0 and got.top_ids[1].tolist() == [0, 1, 2]
    assert got.top_logp[1].tolist() == [0, -INF, -INF]
    assert abs(logp[2] + math.log(V)) < 1e-3 and abs(ent[2] - math.log(V)) < 1e-3
    assert got.top_ids[2].tolist() == [0, 1, 2]
    assert logp[3] == 0 and ent[3] == 0 and got.top_ids[3].tolist() == [V - 1, 0, 1]
    assert abs(logp[4] + math.log(2)) < 1e-5 and abs(ent[4] - math.log(2)) < 1e-5
    assert got.top_ids[4].tolist() == [V - 2, V - 1, 0]
    assert math.isnan(logp[5]) and math.isnan(ent[5]) and got.top_ids[5].tolist()[0] == 3
    assert math.isnan(logp[6]) and math.isnan(ent[6]) and got.top_ids[6].tolist()[0] == 5
    assert logp[7] == 0 and ent[7] == 0
    one = torch.ones(8, device="cuda")
    d = mk.muon_token_logprobs_backward(x, tok, got.lse, got.entropy, one, one).float()
    assert not bool(d[0].any()) and not bool(d[1].any()) and not bool(d[3].any())
    assert bool((d[4, :V - 2] == 0).all()) and bool(d[4].isfinite().all())
    assert bool(d[[2, 7]].isfinite().all())
    assert bool(d[5].isnan().any()) and bool(d[6].isnan().any())


def test_ties_and_signed_zeros_go_to_the_lowest_index(mk):
    for V in (100, 40000):
        x = torch.zeros(3, V, device="cuda")
        x[0, ::2] = -0.0
        x[1, 50:] = 2.0
        x[2] = torch.arange(V, device="cuda") % 7
        got = mk.muon_token_logprobs(x, top=32)
        assert got.logp is None
        assert torch.equal(got.top_ids, torch.sort(x, dim=1, descending=True, stable=True).indices[:, :32])
        asc = torch.arange(V, device="cuda", dtype=torch.float32)[None]   # every element enters the list
        assert mk.muon_token_logprobs(asc, top=32).top_ids[0].tolist() == list(range(V - 1, V - 33, -1))


def test_row_strides_alignment_and_no_write_outside(mk):
    for dt in (torch.bfloat16, torch.float32):
        x, tok, dl, de = inputs(6, 1003, dt, seed=3)
        ref = mk.muon_token_logprobs(x, tok, top=4)
        d_ref = mk.muon_token_logprobs_backward(x, tok, ref.lse, ref.entropy, dl, de)
        for shift in (0, 1, 5):
            wide = torch.full((6, 1019), 9.0, dtype=dt, device="cuda")
            v = wide[:, shift:shift + 1003]
            v.copy_(x)
            got = mk.muon_token_logprobs(v, tok, top=4)
            assert torch.equal(got.top_ids, ref.top_ids)
            check_forward(got, x, tok, 4)
            out = torch.full((6, 1030), 9.0, dtype=dt, device="cuda")
            o = out[:, 2:1005]
            mk.muon_token_logprobs_backward(v, tok, ref.lse, ref.entropy, dl, de, out=o)
            assert torch.equal(o, d_ref)   # an element's gradient depends on it and its row alone
            assert bool((out[:, :2] == 9).all()) and bool((out[:, 1005:] == 9).all())


def test_a_row_past_32_bit_offsets(mk):
    V = 131072
    T = (1 << 31) // V + 3                        # element offsets past 2^31
    x = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    x[-1, 77] = 20.0
    x[-2, V - 1] = 3.0
    tok = torch.full((T,), 77, device="cuda")
    got = mk.muon_token_logprobs(x, tok, top=1)
    assert got.top_ids[-1, 0] == 77 and got.top_ids[-2, 0] == V - 1 and got.top_ids[0, 0] == 0
    want = 20.0 - math.log(math.exp(20.0) + V - 1)
    assert abs(float(got.logp[-1]) - want) < 1e-4
    d = mk.muon_token_logprobs_backward(x, tok, got.lse, None, torch.ones(T, device="cuda"))
    assert abs(float(d[-1, 77]) - (1 - math.exp(want))) < 1e-4 and float(d[-1, 0]) < 0


def test_token_out_of_range_is_reported(mk):
    x, tok, dl, de = inputs(3, 100, torch.float32)
    tok[1] = 100
    got = mk.muon_token_logprobs(x, tok)
    assert mk.muon_get_device_status() == -6
    assert bool(got.logp[1].isnan()) and bool(got.lse.isfinite().all())
    mk.muon_token_logprobs_backward(x, tok, got.lse, None, dl)
    assert mk.muon_get_device_status() == -6 and mk.muon_get_device_status() == 0


def test_no_rows_and_refusals(mk):
    x, tok, dl, de = inputs(3, 100, torch.float32)
    assert mk.muon_token_logprobs(x[:0], tok[:0], top=2).top_ids.shape == (0, 2)
    assert mk.muon_token_logprobs_backward(x[:0], tok[:0], dl[:0], None, dl[:0]).shape == (0, 100)
    f = mk.muon_token_logprobs(x, tok)
    for bad in (lambda: mk.muon_token_logprobs(x.half(), tok), lambda: mk.muon_token_logprobs(x, tok.int()),
                lambda: mk.muon_token_logprobs(x.cpu(), tok)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: mk.muon_token_logprobs(x, tok[:2]), lambda: mk.muon_token_logprobs(x[0], tok),
                lambda: mk.muon_token_logprobs(x.T, tok),
                lambda: mk.muon_token_logprobs_backward(x, None, f.lse, None, dl),
                lambda: mk.muon_token_logprobs_backward(x, tok, f.lse, None, dl, de)):
        with pytest.raises(ValueError):
            bad()
    for top, status in ((33, -2), (-1, -1)):
        with pytest.raises(mk.MuonError) as e:
            mk.muon_token_logprobs(x, tok, top=top)
        assert e.value.status == status
    with pytest.raises(mk.MuonError) as e:
        mk.muon_token_logprobs_backward(x, tok, f.lse)
    assert e.value.status == -1


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V, shift", [(33, 0), (40, 3), (999, 0), (50003, 0), (50003, 5), (131075, 1)])
def test_top_alternatives_of_rows_far_below_zero(mk, dt, V, shift):
    """Nothing but very low finite values, some of them before or after the row's whole vectors."""
    t = DT[dt]
    low = torch.finfo(t).min
    g = torch.Generator(device="cuda").manual_seed(V + shift)
    wide = torch.zeros(5, (V + shift + 7) // 8 * 8, dtype=t, device="cuda")   # rows start alike
    x = wide[:, shift:shift + V]
    x[0] = low                                  # one mask of the type's lowest value: ties to the lowest index
    x[1] = -2e30                                # two masks, the larger of them in the middle, the lower one last
    x[1, V // 2] = -1e30
    x[1, V - 1] = -1e35
    x[2] = -1e35
    x[2, V // 3] = -0.95e30
    x[2, 0] = x[2, V - 1] = -3e30
    x[3] = -(10.0 ** (29.7 + 8.5 * torch.rand(V, generator=g, device="cuda"))).to(t)
    x[4] = -INF
    x[4, 1], x[4, V - 2], x[4, V - 1] = -1e33, -1e32, low
    for top in (1, 3, 20):
        got = mk.muon_token_logprobs(x, top=top)
        assert mk.muon_get_device_status() == 0
        assert torch.equal(got.top_ids, torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :top])
        assert torch.equal(got.lse[1:], x.float().amax(1)[1:])   # exp of any other difference is 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 30, 2.0 ** 60, 2.0 ** 100])
def test_gradient_of_masked_entries_under_large_factors(mk, dt, scale):
    """dlogp and dentropy scaled (as a scaled loss sends them): masked entries still get 0."""
    x, tok, dl, de = inputs(6, 1003, DT[dt], seed=8)
    low = torch.rand(x.shape, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") < 0.1
    low[torch.arange(6, device="cuda"), tok.clamp(min=0)] = False
    x[low] = torch.finfo(x.dtype).min
    masked = low | (x == -INF)
    f = mk.muon_token_logprobs(x, tok)
    plain = mk.muon_token_logprobs_backward(x, tok, f.lse, f.entropy, dl, de).float()
    got = mk.muon_token_logprobs_backward(x, tok, f.lse, f.entropy, dl * scale, de * scale).float()
    assert bool((got[masked] == 0).all()) and bool((plain[masked] == 0).all())
    # a power of two moves the exponent of every step and rounds nothing otherwise (no entry is near either limit)
    assert torch.equal(got, plain * scale)
