"""The gated feed-forward block over expert matrices, against its definition in 64 bits.

Bounds.  The kernels round h (forward), dg, du and h (backward) and every
output once to bf16 (half a unit in the last place: 2^-9 relative) and sum in
fp32 (at most K 2^-24 of the sum of magnitudes, K <= 1100 here: 2^-13.9).  An
entry is therefore within 2^-8 of |value| + sum |a| |b| over its last product,
twice the first-order bound; and because independent roundings add up by their
squares, an array of many entries (4096 or more, where the sums' own
cancellations average out) is within 2^-8 in the Frobenius norm, each of the
two roundings being at most 2^-9 of it.
"""

import ctypes
import math

import pytest
import torch

from tests._util import require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def mk():
    return require_gpu()


# rows of each expert, hidden, ffn: ends of tiles (256 rows, 64 rows of a gradient's sum, 128 and 256 columns), experts
# without rows, one row, widths of 8
SHAPES = [
    ([1], 8, 8),
    ([3], 136, 40),
    ([1, 0, 1, 2], 264, 136),
    ([0, 17, 0, 0, 64, 1], 200, 328),
    ([255, 256, 257], 72, 264),
    ([63, 65, 0, 128, 129], 520, 120),
    ([700, 5], 1000, 328),
    ([0, 0], 64, 64),
    ([33], 1096, 1032),
    ([2] * 37, 128, 256),
]


def inputs(sizes, H, F, seed=0):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed + H + F + len(sizes))
    T, E = sum(sizes), len(sizes)

    def n(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    off = torch.tensor([0] + sizes, device="cuda").cumsum(0)
    return {"x": n(T, H), "w1": n(E, H, F, std=H ** -0.5), "w3": n(E, H, F, std=H ** -0.5),
            "w2": n(E, F, H, std=F ** -0.5), "off": off, "gate": n(T, F), "up": n(T, F), "dy": n(T, H), "sizes": sizes}


def act64(g, act):
    return torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")


def groups(d):
    a = 0
    for e, n in enumerate(d["sizes"]):
        yield e, slice(a, a + n)
        a += n


def forward64(d, act):
    """(value, sum of magnitudes of the last product) of y, gate, up."""
    out = {k: [] for k in ("y", "gate", "up")}
    for e, r in groups(d):
        x, w1, w3, w2 = d["x"][r].double(), d["w1"][e].double(), d["w3"][e].double(), d["w2"][e].double()
        g, u = x @ w1, x @ w3
        h = act64(g, act) * u
        out["y"].append((h @ w2, h.abs() @ w2.abs()))
        out["gate"].append((g, x.abs() @ w1.abs()))
        out["up"].append((u, x.abs() @ w3.abs()))
    return {k: tuple(torch.cat([p[i] for p in v]) for i in (0, 1)) for k, v in out.items()}


def backward64(d, act):
    dx, dw1, dw3, dw2 = [], [], [], []
    for e, r in groups(d):
        x, w1, w3, w2 = d["x"][r].double(), d["w1"][e].double(), d["w3"][e].double(), d["w2"][e].double()
        g, u, dy = d["gate"][r].double().requires_grad_(), d["up"][r].double(), d["dy"][r].double()
        with torch.enable_grad():
            a = act64(g, act)
            da, = torch.autograd.grad(a.sum(), g)
        a = a.detach()
        dh = dy @ w2.T
        dg, du, h = dh * u * da, dh * a, a * u
        dx.append((dg @ w1.T + du @ w3.T, dg.abs() @ w1.abs().T + du.abs() @ w3.abs().T))
        dw1.append((x.T @ dg, x.abs().T @ dg.abs()))
        dw3.append((x.T @ du, x.abs().T @ du.abs()))
        dw2.append((h.T @ dy, h.abs().T @ dy.abs()))
    both = lambda v, f: tuple(f([p[i] for p in v]) for i in (0, 1))  # noqa: E731
    return {"dx": both(dx, torch.cat), "dw1": both(dw1, torch.stack), "dw3": both(dw3, torch.stack),
            "dw2": both(dw2, torch.stack)}


def check(got, ref, name):
    value, mags = ref
    got = got.double()
    assert got.shape == value.shape, name
    err = (got - value).abs()
    assert bool((err <= U * (value.abs() + mags) + 1e-30).all()), (name, float((err / (mags + 1e-30)).max()))
    norm = float(value.norm())
    if value.numel() >= 4096:
        assert float((got - value).norm()) <= U * norm + 1e-30, (name, float((got - value).norm()) / max(norm, 1e-30))


def forward(mk, d, act, **kw):
    return dict(zip(("y", "gate", "up"), mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"], act=act,
                                                           keep=True, **kw)))


def backward(mk, d, act, **kw):
    return dict(zip(("dx", "dw1", "dw3", "dw2"), mk.muon_gated_ffn_backward(
        d["dy"], d["x"], d["gate"], d["up"], d["w1"], d["w3"], d["w2"], d["off"], act=act, **kw)))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("sizes,H,F", SHAPES)
def test_forward(mk, sizes, H, F, act):
    d = inputs(sizes, H, F)
    got = forward(mk, d, act)
    assert mk.muon_get_device_status() == 0
    ref = forward64(d, act)
    for k in got:
        check(got[k], ref[k], k)
    served = mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"], act=act)
    check(served, ref["y"], "served y")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("sizes,H,F", SHAPES)
def test_backward(mk, sizes, H, F, act):
    d = inputs(sizes, H, F, seed=1)
    dw = tuple(torch.full_like(d[k], float("nan")) for k in ("w1", "w3", "w2"))   # overwritten, not added to
    got = backward(mk, d, act, dw=dw)
    assert mk.muon_get_device_status() == 0
    ref = backward64(d, act)
    for k in got:
        check(got[k], ref[k], k)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 31, 32, 33, 64, 100])
@pytest.mark.parametrize("experts,H,F", [(1, 1032, 520), (5, 520, 264), (1, 4096, 1792)])
def test_few_rows(mk, rows, experts, H, F):
    """Serving: a few rows, spread unevenly over the experts."""
    g = torch.Generator().manual_seed(rows + experts)
    picks = torch.randint(0, experts, (rows,), generator=g)
    d = inputs(torch.bincount(picks, minlength=experts).tolist(), H, F, seed=2)
    y = mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"])
    assert mk.muon_get_device_status() == 0
    check(y, forward64(d, "silu")["y"], "y")


def test_one_expert_without_offsets(mk):
    d = inputs([77], 136, 264, seed=3)
    w = [d[k][0] for k in ("w1", "w3", "w2")]
    y, gate, up = mk.muon_gated_ffn(d["x"], *w, keep=True)
    y2, gate2, up2 = mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"], keep=True)
    assert torch.equal(y, y2) and torch.equal(gate, gate2) and torch.equal(up, up2)
    a = mk.muon_gated_ffn_backward(d["dy"], d["x"], gate, up, *w)
    b = mk.muon_gated_ffn_backward(d["dy"], d["x"], gate, up, d["w1"], d["w3"], d["w2"], d["off"])
    for p, q in zip(a, b):
        assert torch.equal(p, q.reshape(p.shape))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_agrees_with_differences(mk, act):
    """d/dt of sum(c * y) along random directions, by central differences of the 64-bit forward form."""
    d = inputs([40, 0, 25], 72, 48, seed=4)
    f = forward(mk, d, act)
    c = d["dy"]
    got = dict(zip(("x", "w1", "w3", "w2"), mk.muon_gated_ffn_backward(
        c, d["x"], f["gate"], f["up"], d["w1"], d["w3"], d["w2"], d["off"], act=act)))
    gen = torch.Generator(device="cuda").manual_seed(9)
    for k, grad in got.items():
        v = torch.randn(d[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        v = v + grad.double() / grad.double().std()   # mostly along the gradient, so that the slope is not near zero
        eps = 1e-5
        slope = 0.0
        for sign in (1, -1):
            moved = dict(d)
            moved[k] = d[k].double() + sign * eps * v
            slope += sign * float((forward64(moved, act)["y"][0] * c.double()).sum()) / (2 * eps)
        # the gradient's own error (2^-7: gate and up rounded too) along v, and v's random part against it
        assert abs(float((grad.double() * v).sum()) - slope) <= 2 * U * float(grad.double().norm() * v.norm()), k


def test_row_strides_and_no_write_outside(mk):
    d = inputs([30, 35], 136, 72, seed=5)
    T, H = d["x"].shape
    wide = torch.full((T, H + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    x = wide.clone()[:, 8:8 + H]
    x.copy_(d["x"])
    dy = wide.clone()[:, 16:16 + H]
    dy.copy_(d["dy"])
    buf = wide.clone()
    out = buf[:, 24:24 + H]
    y = mk.muon_gated_ffn(x, d["w1"], d["w3"], d["w2"], d["off"], out=out)
    assert y is out
    assert torch.equal(out, mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"]))
    assert bool((buf[:, :24] == 7).all()) and bool((buf[:, 24 + H:] == 7).all())
    dxb = wide.clone()
    got = mk.muon_gated_ffn_backward(dy, x, d["gate"], d["up"], d["w1"], d["w3"], d["w2"], d["off"],
                                     dx=dxb[:, 8:8 + H])
    ref = mk.muon_gated_ffn_backward(d["dy"], d["x"], d["gate"], d["up"], d["w1"], d["w3"], d["w2"], d["off"])
    for p, q in zip(got, ref):
        assert torch.equal(p, q)
    assert bool((dxb[:, :8] == 7).all()) and bool((dxb[:, 8 + H:] == 7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("sizes", [[30, 35, 64], [3, 1, 2], [300, 3, 70]])
def test_one_experts_nan_stays_with_it(mk, sizes, bad):
    d = inputs(sizes, 136, 264, seed=6)
    ref_f, ref_b = forward(mk, d, "silu"), backward(mk, d, "silu")
    served = mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"])
    a, b = sizes[0], sizes[0] + sizes[1]
    for k in ("x", "dy", "gate", "up"):
        d[k] = d[k].clone()
        d[k][a:b] = bad
    for k in ("w1", "w3", "w2"):
        d[k] = d[k].clone()
        d[k][1] = bad
    got_f, got_b = forward(mk, d, "silu"), backward(mk, d, "silu")
    served2 = mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"])
    rows = torch.ones(sum(sizes), dtype=torch.bool, device="cuda")
    rows[a:b] = False
    for k in ("y", "gate", "up"):
        assert torch.equal(got_f[k][rows], ref_f[k][rows]), k
        assert not bool(got_f[k][a:b].isfinite().any()), k
    assert torch.equal(served2[rows], served[rows])
    assert torch.equal(got_b["dx"][rows], ref_b["dx"][rows])
    for k in ("dw1", "dw3", "dw2"):
        assert torch.equal(got_b[k][[0, 2]], ref_b[k][[0, 2]]), k
        assert not bool(got_b[k][1].isfinite().any()), k


def test_large_pre_activations_keep_their_limits(mk):
    """act(g) tends to g for large g and to 0 for large -g, without overflow on the way."""
    d = inputs([4], 64, 64, seed=7)
    g = torch.tensor([300.0, -300.0, 40.0, -40.0], device="cuda").bfloat16()
    d["gate"][:] = g[:, None]
    for act in ("silu", "gelu"):
        got, ref = backward(mk, d, act), backward64(d, act)
        for k in got:
            assert bool(got[k].isfinite().all()), (act, k)
            check(got[k], ref[k], k)


def test_repeated_calls_give_the_same_bits_on_other_streams_and_workspaces(mk):
    d = inputs([63, 65, 0, 128, 129], 520, 120, seed=8)
    T, E = d["x"].shape[0], 5
    first_f, first_b = forward(mk, d, "silu"), backward(mk, d, "silu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws_f = torch.full((mk.muon_gated_ffn_workspace_bytes(T, E, 520, 120),), 255, dtype=torch.uint8, device="cuda")
    ws_b = torch.full((mk.muon_gated_ffn_backward_workspace_bytes(T, E, 520, 120),), 255, dtype=torch.uint8,
                      device="cuda")
    with torch.cuda.stream(side):   # the current stream is where the work goes by default
        f = forward(mk, d, "silu", workspace=ws_f)
        b = backward(mk, d, "silu", workspace=ws_b, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for got, ref in ((f, first_f), (b, first_b)):
        for k in ref:
            assert torch.equal(got[k], ref[k]), k


@pytest.mark.parametrize("sizes,H,F", [([3], 136, 40), ([300, 0, 70], 264, 136)])
def test_captured_in_a_graph(mk, sizes, H, F):
    """Captured once, replayed on new inputs and new group sizes (the sizes are read on the device)."""
    d = inputs(sizes, H, F, seed=12)
    T, E = d["x"].shape[0], len(sizes)
    ws = torch.empty(mk.muon_gated_ffn_backward_workspace_bytes(T, E, H, F), dtype=torch.uint8, device="cuda")
    kept = {k: d[k].clone() for k in ("x", "off", "dy", "gate", "up")}
    step = {**d, **kept}
    forward(mk, step, "silu", workspace=ws), backward(mk, step, "silu", workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = forward(mk, step, "silu", workspace=ws)
        b = backward(mk, step, "silu", workspace=ws)
    new = inputs(sizes[::-1], H, F, seed=13)
    for k, v in kept.items():
        v.copy_(new[k])
    graph.replay()
    mixed = {**new, "w1": d["w1"], "w3": d["w3"], "w2": d["w2"]}
    for got, ref in ((f, forward(mk, mixed, "silu")), (b, backward(mk, mixed, "silu"))):
        for k in ref:
            assert torch.equal(got[k], ref[k]), k
    assert mk.muon_get_device_status() == 0


def test_rows_past_32_bit_offsets(mk):
    """rows * ffn past 2^31 elements: the last rows against 64 bits."""
    T, H, F = 270_000, 64, 8192
    d = inputs([T], H, F, seed=14)
    f = forward(mk, d, "silu")
    tail = {**d, "sizes": [200], **{k: d[k][-200:] for k in ("x", "dy", "gate", "up")}}
    ref = forward64(tail, "silu")
    for k in f:
        check(f[k][-200:], ref[k], k)
    del f
    b = backward(mk, d, "silu")
    check(b["dx"][-200:], backward64(tail, "silu")["dx"], "dx")
    assert all(bool(b[k].isfinite().all()) for k in b)
    assert mk.muon_get_device_status() == 0


def test_what_is_not_needed_is_left_out(mk):
    d = inputs([30, 35], 136, 72, seed=10)
    ref = backward(mk, d, "silu")
    a = backward(mk, d, "silu", need_dw=False)
    assert torch.equal(a["dx"], ref["dx"]) and a["dw1"] is None
    b = backward(mk, d, "silu", need_dx=False)
    assert b["dx"] is None and all(torch.equal(b[k], ref[k]) for k in ("dw1", "dw3", "dw2"))


@pytest.mark.parametrize("offsets", [[0, 40, 30, 65], [0, 10, 20, 60], [5, 30, 40, 65], [-4, 30, 40, 65],
                                     [0, 30, 2 ** 40, 65]])
def test_offsets_out_of_order_or_range_are_reported(mk, offsets):
    d = inputs([20, 20, 25], 136, 72, seed=11)
    d["off"] = torch.tensor(offsets, device="cuda")
    forward(mk, d, "silu")
    assert mk.muon_get_device_status() == -6
    mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"])
    assert mk.muon_get_device_status() == -6
    backward(mk, d, "silu")
    assert mk.muon_get_device_status() == -6
    assert mk.muon_get_device_status() == 0


def test_no_rows(mk):
    d = inputs([0, 0, 0], 64, 72)
    dw = tuple(torch.full_like(d[k], 3.0) for k in ("w1", "w3", "w2"))
    assert forward(mk, d, "silu")["y"].shape == (0, 64)
    got = backward(mk, d, "silu", dw=dw)
    assert all(not bool(got[k].any()) for k in ("dw1", "dw3", "dw2"))


def test_refusals(mk):
    d = inputs([4, 4], 64, 72)
    x, w1, w3, w2, off = (d[k] for k in ("x", "w1", "w3", "w2", "off"))
    for bad in ((x.float(), w1, w3, w2, off), (x.cpu(), w1, w3, w2, off), (x, w1, w3, w2, off.int())):
        with pytest.raises(TypeError):
            mk.muon_gated_ffn(*bad)
    for bad in ((x[:, :56], w1, w3, w2, off), (x, w1, w3[:, :, :64], w2, off), (x, w1, w3, w2.mT, off),
                (x, w1, w3, w2, off[:2]), (x, w1, w3, w2, None), (x.T.contiguous().T, w1, w3, w2, off)):
        with pytest.raises(ValueError):
            mk.muon_gated_ffn(*bad)
    with pytest.raises(ValueError):
        mk.muon_gated_ffn(x, w1, w3, w2, off, act="relu")
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(mk.MuonError) as e:
        mk.muon_gated_ffn(x, w1, w3, w2, off, workspace=small)
    assert e.value.status == -4
    with pytest.raises(mk.MuonError) as e:   # 12 columns: no multiple of 8
        mk.muon_gated_ffn(x[:, :12].contiguous(), w1[:, :12].contiguous(), w3[:, :12].contiguous(),
                          w2[:, :, :12].contiguous(), off)
    assert e.value.status == -2
    mk.muon_inject_alloc_failures(1)
    with pytest.raises(mk.MuonError) as e:
        mk.muon_gated_ffn(x, w1, w3, w2, off)
    assert e.value.status == -4 and mk.muon_inject_alloc_failures(0) == 0
    assert mk.muon_get_device_status() == 0


@pytest.mark.parametrize("sizes,H,F", [
    ([9001], 136, 72),               # 16 parts, the last k-block of 41 rows
    ([3000, 0, 211], 264, 136),      # an expert without rows, one with fewer k-blocks than it has parts
    ([0, 2, 5500, 1], 256, 264),
    ([4096, 4096], 520, 392),
])
def test_weight_gradients_of_long_cut_sums(mk, sizes, H, F):
    """Few tiles and many rows: the rows are cut into parts."""
    d = inputs(sizes, H, F, seed=11)
    dw = tuple(torch.full_like(d[k], float("nan")) for k in ("w1", "w3", "w2"))
    got = backward(mk, d, "silu", dw=dw)
    assert mk.muon_get_device_status() == 0
    ref = backward64(d, "silu")
    for k in got:
        check(got[k], ref[k], k)
    again = backward(mk, d, "silu")
    for k in got:
        assert torch.equal(got[k], again[k])
    for i, n in enumerate(sizes):
        if n == 0:
            assert all(not bool(t[i].any()) for t in dw)


def test_an_unaligned_x_is_no_hindrance_where_only_dx_is_wanted(mk):
    d = inputs([30, 35], 136, 72, seed=10)
    ref = backward(mk, d, "silu")
    wide = torch.zeros(65, 139, dtype=torch.bfloat16, device="cuda")
    d["x"] = wide[:, 3:]
    assert torch.equal(backward(mk, d, "silu", need_dw=False)["dx"], ref["dx"])
    with pytest.raises(mk.MuonError) as e:
        backward(mk, d, "silu")
    assert e.value.status == -2


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [4, 300])   # the kernels of few rows and of many
def test_pre_activations_whose_square_overflows(mk, rows, act):
    """act'(g) is 1 or 0 there, in the gradient as in the forward pass."""
    d = inputs([rows], 64, 64, seed=15)
    d["gate"][0], d["gate"][1], d["gate"][2], d["gate"][3] = 1e20, -1e20, 1e25, -1e25
    got, ref = backward(mk, d, act), backward64(d, act)
    for k in got:
        assert bool(got[k].isfinite().all()), k
        check(got[k], ref[k], k)


def test_an_argument_without_a_truth_value(mk):
    d = inputs([4, 4], 64, 72)
    with pytest.raises(RuntimeError, match="[Bb]oolean value of Tensor"):
        mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"], keep=d["off"])
    with pytest.raises(RuntimeError, match="[Bb]oolean value of Tensor"):
        backward(mk, d, "silu", need_dx=d["off"])


LONG = [700, 100, 1900, 64, 2500, 1283, 0, 3000]   # 41 row tiles, whole and partial k-blocks of 64


@pytest.mark.parametrize("H,F", [(1024, 1536),    # both multiples of 64: 128-column operands load in one piece
                                 (1000, 1320)])   # neither
def test_many_tiles_a_pair(mk, H, F):
    """More than two tiles for each of the 76 pairs in all six products: 451 or more of UP, 164 of DOWN and DX, 246 of
    DH, 192 of dW2, 352 or more of dW1 and dW3.  The accumulators, the ring and the output boxes go round."""
    d = inputs(LONG, H, F, seed=16)
    got_f = forward(mk, d, "silu")
    got_b = backward(mk, d, "silu", dw=tuple(torch.full_like(d[k], float("nan")) for k in ("w1", "w3", "w2")))
    assert mk.muon_get_device_status() == 0
    for got, ref in ((got_f, forward64(d, "silu")), (got_b, backward64(d, "silu"))):
        for k in got:
            check(got[k], ref[k], k)
    for got, again in ((got_f, forward(mk, d, "silu")), (got_b, backward(mk, d, "silu"))):
        for k in got:
            assert torch.equal(got[k], again[k]), k


def test_one_experts_nan_stays_with_it_in_wide_loads(mk):
    """Widths that are multiples of 64 and several k-blocks an expert: the last, partial one next to the NaNs."""
    sizes = [300, 3, 470, 129]
    d = inputs(sizes, 128, 256, seed=17)
    ref = backward(mk, d, "silu")
    for k in ("x", "dy", "gate", "up"):
        d[k] = d[k].clone()
        d[k][300:303] = float("nan")
    got = backward(mk, d, "silu")
    rows = torch.ones(sum(sizes), dtype=torch.bool, device="cuda")
    rows[300:303] = False
    assert torch.equal(got["dx"][rows], ref["dx"][rows])
    for k in ("dw1", "dw3", "dw2"):
        assert torch.equal(got[k][[0, 2, 3]], ref[k][[0, 2, 3]]), k
        assert not bool(got[k][1].isfinite().any()), k


def test_weight_gradients_of_rows_past_32_bit_offsets(mk):
    """rows * ffn past 2^31 elements and a gradient in the last rows alone: their sums against 64 bits."""
    T, H, F = 270_000, 64, 8192
    d = inputs([T], H, F, seed=18)
    d["dy"][:-200] = 0
    got = backward(mk, d, "silu")
    assert mk.muon_get_device_status() == 0
    ref = backward64({**d, "sizes": [200], **{k: d[k][-200:] for k in ("x", "dy", "gate", "up")}}, "silu")
    for k in ("dw1", "dw3", "dw2"):
        check(got[k], ref[k], k)
    assert not bool(got["dx"][:-200].any())
    check(got["dx"][-200:], ref["dx"], "dx")
