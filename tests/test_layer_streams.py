"""Whose memory MoELayer uses when it is called with a stream that is not the
current one: what it allocates comes from that stream's pool, and what crosses
between the two streams is recorded on the other.  torch's streams are replaced
by stand-ins and the launches left out, so nothing here needs a device
(tests/test_gpu_layer_streams.py runs the same on one)."""
import contextlib

import pytest
import torch

BF = torch.bfloat16
D, E, K, F = 64, 8, 2, 128
HERE, SIDE = 7, 1234  # stream handles


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


@pytest.fixture
def world(monkeypatch):
    """The module, the allocations (size, stream) and the tensors recorded."""
    from token_dispatch_grouped_fp32_gb300 import build
    build.build()
    from token_dispatch_grouped_fp32_gb300 import moe
    current, made, recorded = [HERE], {}, []
    monkeypatch.setattr(moe, "_stream", lambda s: current[-1] if s is None else int(s))

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def spy(fn):
        def make(*args, **kw):
            t = fn(*args, **kw)
            made[t.data_ptr()] = current[-1]
            return t
        return make
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: current[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: recorded.append((t.data_ptr(), s)))
    empty, like = torch.empty, torch.empty_like
    monkeypatch.setattr(torch, "empty", spy(empty))
    monkeypatch.setattr(torch, "empty_like", spy(like))
    used = []
    monkeypatch.setattr(moe, "moe_forward", lambda cfg, *a, stream=None: used.append((a, stream)))
    monkeypatch.setattr(moe, "moe_backward", lambda cfg, *a, stream=None: used.append((a, stream)))
    return moe, made, recorded, used


def layer(moe):
    return moe.MoELayer(torch.zeros(E, D).as_subclass(OnDevice), torch.zeros(E, D, 2 * F, dtype=BF),
                        torch.zeros(E, F, D, dtype=BF), K)


@pytest.mark.parametrize("side", [SIDE, 0])
def test_a_stream_that_is_not_current(world, side):
    moe, made, recorded, used = world
    lay, x, dout = layer(moe), torch.zeros(16, D, dtype=BF), torch.zeros(16, D, dtype=BF)
    out = lay.forward(x, stream=side)
    grads = lay.backward(x, dout, stream=side)
    (_, _, _, _, _, fout, ws), s = used[0]
    assert fout is out and s == side
    assert used[1][1] == side and used[1][0][4] is ws
    bwd_ws = used[1][0][-1]
    # everything allocated for the calls belongs to the stream that uses it
    for t in (out, ws, bwd_ws, *grads.values()):
        assert made[t.data_ptr()] == side
    # and returned to its pool only after the current stream is done with it
    for t in (out, *grads.values()):
        assert (t.data_ptr(), HERE) in recorded
    # the caller's tensors stay until that stream is done with them
    for t in (x, dout):
        assert (t.data_ptr(), side) in recorded


def test_buffers_of_the_caller(world):
    moe, made, recorded, used = world
    lay, x, dout = layer(moe), torch.zeros(16, D, dtype=BF), torch.zeros(16, D, dtype=BF)
    out = torch.zeros_like(x)
    grads = {"x": torch.zeros_like(x), "Wr": torch.zeros(E, D), "W_gate_up": torch.zeros_like(lay.W_gate_up),
             "W_down": torch.zeros_like(lay.W_down)}
    lay.forward(x, out, stream=SIDE)
    assert lay.backward(x, dout, grads, stream=SIDE) is grads
    for t in (x, dout, out, *grads.values()):
        assert (t.data_ptr(), SIDE) in recorded and (t.data_ptr(), HERE) not in recorded


def test_a_workspace_that_grows(world):
    moe, made, recorded, used = world
    lay = layer(moe)
    for n in (16, 4000):
        ws = lay.workspace(n, SIDE)
        assert made[ws.data_ptr()] == SIDE
    assert made[lay.workspace(16).data_ptr()] == HERE


@pytest.mark.parametrize("stream", [None, HERE])
def test_the_current_stream_needs_no_records(world, stream):
    moe, made, recorded, used = world
    lay, x = layer(moe), torch.zeros(16, D, dtype=BF)
    lay.forward(x, stream=stream)
    lay.backward(x, torch.zeros_like(x), stream=stream)
    assert not recorded and set(made.values()) == {HERE}
