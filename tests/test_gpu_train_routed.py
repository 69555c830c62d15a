"""Norms, router, dispatch, experts, combining and loss in a run together: the gradients against 64 bits.

Between a parameter and the loss lie at most about ten roundings to bf16 (x,
g, u, h, y, out, last, d, and as many on the way back), each within 2^-8 of
what it rounds; they are independent, so their squares add: sqrt(20) 2^-8 / sqrt(3)
= 0.010 of the norm at worst, and the norms' and the router's factors of about
two leave 0.04.
"""

import math

import pytest
import torch

from tests._util import require_gpu

pytestmark = pytest.mark.gpu


def rms(v, w):
    return v * (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w


def loss64(block, p, tokens, targets, ids):
    """The block's mean loss in 64 bits, dense over the experts, with the choice given."""
    stream = p["embed"][tokens]
    x = rms(stream, p["w_in"])
    score = (x @ p["router"].T).sigmoid()
    given = torch.zeros_like(score).scatter_add(1, ids.clamp(min=0), (ids >= 0).double())
    weight = score * given
    weight = weight / weight.sum(1, keepdim=True).clamp(min=1e-30)
    out = 0
    for e in range(block.experts):
        h = torch.nn.functional.silu(x @ p["w1"][e]) * (x @ p["w3"][e])
        out = out + weight[:, e:e + 1] * (h @ p["w2"][e])
    last = rms(stream + rms(out, p["w_post"]), p["w_out"])
    on = targets >= 0
    return torch.nn.functional.cross_entropy((last @ p["head"].T)[on], targets[on])


def test_gradients_of_the_whole_block():
    mk = require_gpu()
    from examples.train_routed import RoutedBlock
    block = RoutedBlock(vocab=200, hidden=128, ffn=136, experts=6, top=3)
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens = torch.randint(0, 200, (700,), generator=g, device="cuda")
    targets = torch.randint(0, 200, (700,), generator=g, device="cuda")
    targets[::9] = -1
    loss, grads, ids = block.gradients(tokens, targets)
    assert mk.muon_get_device_status() == 0
    assert bool((ids[::9] == -1).all()) and bool((ids[1::9] >= 0).all())
    p = {k: v.double().requires_grad_() for k, v in {**block.p, **block.w}.items()}
    want = loss64(block, p, tokens, targets, ids)
    assert abs(float(loss.sum() / (targets >= 0).sum()) - want.item()) < 0.02 * want.item()
    for (k, v), d in zip(p.items(), torch.autograd.grad(want, list(p.values()))):
        err = float((grads[k].double() - d).norm() / d.norm())
        assert err < 0.04, (k, err)


def test_a_step_moves_each_parameter_against_its_own_gradient():
    """The first step of AdamW is lr sign(g) wherever g is far above eps; the router's bias goes towards the experts with
    less than the mean load.  Muon's step is the gradient with its singular values made one (0.7 to 1.2 by five steps),
    so the product of the two is the sum of those, at least the gradient's norm by matrix: of 6 matrices of
    rank 128 their cosine is at least 0.7 / 1.2 / sqrt(6 128) = 0.021.
    """
    require_gpu()
    from examples.train_routed import RoutedBlock
    block = RoutedBlock(vocab=200, hidden=128, ffn=136, experts=6, top=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    tokens = torch.randint(0, 200, (700,), generator=g, device="cuda")
    targets = torch.randint(0, 200, (700,), generator=g, device="cuda")
    targets[::9] = -1
    before = {k: v.clone() for k, v in {**block.p, **block.w, "bias": block.bias}.items()}
    _, grads, ids = block.gradients(tokens, targets)
    block.step(tokens, targets, adam_lr=0.25)           # above the rounding of parameters of about 1
    for k in block.p:
        move, d = block.p[k].double() - before[k].double(), grads[k].double()
        clear = d.abs() > 1e-6                          # eps is 1e-8
        assert bool(clear.any()) and bool((move[clear] * d[clear] < 0).all()), k
    for k in block.w:
        move, d = block.w[k].double() - before[k].double(), grads[k].double()
        assert float((move * d).sum()) < -0.02 * float(move.norm() * d.norm()), k
    load = torch.stack([(ids == e).sum() for e in range(block.experts)]).double()
    moved = block.bias.double() - before["bias"].double()
    assert bool((moved.sign() == (load.mean() - load).sign()).all())


def test_the_example_runs():
    require_gpu()
    from examples.train_routed import main
    history = main(steps=4, rows=1000)
    assert len(history) == 4 and all(math.isfinite(v) and v > 0 for v in history)
