"""The training example: forward, backward, clipping and the update together."""
import pytest

from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu


def test_the_loss_falls():
    load_moe()
    from examples import train_step
    losses = train_step.main(steps=40)
    assert all(v == v and v < 1e3 for v in losses)
    assert sum(losses[-5:]) < 0.9 * sum(losses[:5])
