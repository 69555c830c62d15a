"""The example that runs the operators together with the Muon step learns what it is given."""

import math

import pytest

from tests._util import require_gpu

pytestmark = pytest.mark.gpu


def test_the_block_learns_a_fixed_successor():
    require_gpu()
    from examples.train_block import main
    history = main(steps=60)
    assert history[0][0] < -0.8 * math.log(512)            # it starts near (or below) a uniform guess
    assert history[-1][0] > -0.5 * math.log(512)           # and more than halves that loss
    assert all(math.isfinite(v) for pair in history for v in pair)
