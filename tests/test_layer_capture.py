"""The workspaces that a captured graph holds addresses of stay allocated when
a longer batch replaces them.  Launches and the capture's state are replaced,
so nothing here needs a device."""
import weakref

import pytest
import torch

BF = torch.bfloat16
D, E, K, F = 64, 8, 2, 128


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


@pytest.fixture
def world(monkeypatch):
    from token_dispatch_grouped_fp32_gb300 import build
    build.build()
    from token_dispatch_grouped_fp32_gb300 import moe
    capturing, used = [False], []
    monkeypatch.setattr(moe, "_stream", lambda s: 7 if s is None else int(s))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: empty(*a, **kw).as_subclass(OnDevice))
    monkeypatch.setattr(moe, "moe_forward", lambda cfg, *a, stream=None: used.append(weakref.ref(a[-1])))
    monkeypatch.setattr(moe, "moe_backward", lambda cfg, *a, stream=None: used.append(weakref.ref(a[-1])))
    lay = moe.MoELayer(torch.zeros(E, D), torch.zeros(E, D, 2 * F, dtype=BF),
                       torch.zeros(E, F, D, dtype=BF), K)

    def step(T):
        """The workspaces of one forward and backward of T tokens."""
        x = torch.zeros(T, D, dtype=BF)
        lay(x)
        lay.backward(x, torch.zeros_like(x))
        return used[-2:]
    return capturing, step


def test_captured_workspaces_outlive_a_longer_batch(world):
    capturing, step = world
    step(16)  # allocated before the capture, as a warm-up does
    capturing[0] = True
    captured = step(16)
    capturing[0] = False
    later = step(4000)
    assert all(a() is not None and a() is not b() for a, b in zip(captured, later))
    step(8000)
    assert all(a() is not None for a in captured)


def test_other_workspaces_go(world):
    _, step = world
    first = step(16)
    step(4000)
    assert all(a() is None for a in first)
