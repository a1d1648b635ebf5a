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


@pytest.mark.parametrize("optimizer", ["adamw", "adamw8"])
@pytest.mark.parametrize("score", [None, "softmax", "sigmoid"])
def test_it_runs_with_adamw_and_other_scores(optimizer, score):
    load_moe()
    from examples import train_step
    losses = train_step.main(steps=3, T=300, optimizer=optimizer, score=score)
    assert len(losses) == 3 and all(v == v and v < 1e3 for v in losses)
