"""Whose memory AdamW uses when it steps on a stream that is not the one it was made on: every
tensor of a step is recorded there, once for each stream.  torch's streams are replaced by
stand-ins and the launches left out, so nothing here needs a device."""
import contextlib

import pytest
import torch

BF = torch.bfloat16
HERE, SIDE = 7, 1234  # stream handles


class OnDevice(torch.Tensor):
    device = property(lambda self: torch.device("cuda", 0))


@pytest.fixture
def world(monkeypatch):
    from token_dispatch_grouped_fp32_gb300 import build
    build.build()
    from token_dispatch_grouped_fp32_gb300 import moe
    current, recorded, launched = [HERE], [], []
    monkeypatch.setattr(moe, "_stream", lambda s: current[-1] if s is None else int(s))

    @contextlib.contextmanager
    def stream(s):
        current.append(int(s))
        yield
        current.pop()
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    zeros, empty = torch.zeros, torch.empty
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **kw: zeros(*a, **kw).as_subclass(OnDevice))
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw).as_subclass(OnDevice))
    monkeypatch.setattr(moe, "_on_current", lambda device: None)
    monkeypatch.setattr(moe, "moe_clip_grad_norm", lambda *a, **kw: launched.append(current[-1]))
    monkeypatch.setattr(moe, "moe_adamw_step", lambda *a, **kw: launched.append(current[-1]))
    return moe, recorded, launched, current


def optimizer(moe, **kw):
    def t(n, dt=BF):
        return torch.ones(n, dtype=dt).as_subclass(OnDevice)
    params, grads = [t(700), t(5, torch.float32)], [t(700), t(5, torch.float32)]
    return moe.AdamW(params, grads, 1e-3, **kw)


def tensors(opt):
    all_ = [t for d in opt.tensors for t in d.values() if isinstance(t, torch.Tensor)]
    return {t.data_ptr() for t in (*all_, opt.norm, opt._ws, opt._scalars) if t is not None}


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("kw,n", [(dict(), 0), (dict(max_norm=1.0), 2), (dict(max_norm=1.0, capturable=True), 3)])
def test_a_step_on_another_stream(world, bits, kw, n):
    moe, recorded, launched, _ = world
    opt = optimizer(moe, bits=bits, **kw)
    per = (6 if bits == 8 else 4)  # parameter, gradient, states, scales
    assert len(tensors(opt)) == 2 * per + 1 + n  # one master
    opt.step(stream=SIDE)
    assert set(launched) == {SIDE}
    assert {p for p, s in recorded if s == SIDE} == tensors(opt)
    assert {s for _, s in recorded} == {SIDE}
    k = len(recorded)
    opt.step(stream=SIDE)  # the memory stays until both are done with it: once is enough
    assert len(recorded) == k
    opt.step(stream=0)
    assert {p for p, s in recorded if s == 0} == tensors(opt)


def test_a_current_stream_that_is_another(world):
    moe, recorded, launched, current = world
    opt = optimizer(moe, max_norm=1.0)
    current.append(SIDE)
    opt.step()
    assert {p for p, s in recorded if s == SIDE} == tensors(opt)


def test_scalars_are_written_on_the_replay_s_stream(world):
    moe, recorded, launched, current = world
    opt = optimizer(moe, capturable=True)
    current.append(SIDE)
    opt.advance()
    assert (opt._scalars.data_ptr(), SIDE) in recorded


def test_its_own_stream_needs_no_records(world):
    moe, recorded, launched, _ = world
    opt = optimizer(moe, max_norm=1.0, capturable=True)
    opt.step()
    opt.step(stream=HERE)
    assert not recorded and set(launched) == {HERE}
