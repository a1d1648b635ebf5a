"""MoELayer.backward runs on the intermediates of the latest forward on its
stream, or not at all.  The two launches are replaced, so nothing here needs a
device: what is checked is which calls reach them, and with which workspace."""
import pytest
import torch

BF = torch.bfloat16
D, E, K, F = 64, 8, 2, 128


@pytest.fixture
def moe(monkeypatch):
    from token_dispatch_grouped_fp32_gb300 import build
    build.build()
    from token_dispatch_grouped_fp32_gb300 import moe as m
    monkeypatch.setattr(m, "_stream", lambda stream: 7 if stream is None else int(stream))
    m_calls = []

    def forward(cfg, x, Wr, bias, Wgu, Wd, out, ws, **kw):
        for t in (x, out, ws):
            m._ptr(t)  # the binding's own refusal of strided tensors
        m_calls.append(("forward", ws))

    def backward(cfg, x, Wr, Wgu, Wd, fwd_ws, *rest, **kw):
        m_calls.append(("backward", fwd_ws))
    monkeypatch.setattr(m, "moe_forward", forward)
    monkeypatch.setattr(m, "moe_backward", backward)
    m.calls = m_calls
    yield m
    del m.calls


def layer(moe, **kw):
    return moe.MoELayer(torch.zeros(E, D), torch.zeros(E, D, 2 * F, dtype=BF),
                        torch.zeros(E, F, D, dtype=BF), K, **kw)


def rows(n):
    return torch.zeros(n, D, dtype=BF)


def refused(moe, lay, x):
    n = len(moe.calls)
    with pytest.raises(RuntimeError, match="latest forward"):
        lay.backward(x, rows(x.shape[0]))
    assert len(moe.calls) == n


def test_backward_gets_the_forward_workspace(moe):
    lay, x = layer(moe), rows(16)
    lay(x)
    for _ in range(2):  # one forward, any number of gradients
        lay.backward(x, rows(16))
    assert [c for c, _ in moe.calls] == ["forward", "backward", "backward"]
    assert all(ws is moe.calls[0][1] for _, ws in moe.calls)
    lay.backward(x.view(16, D), rows(16))  # the same rows through another tensor object


def test_after_a_longer_batch_was_refused(moe):
    """The longer batch grew the workspace before its tensors were refused."""
    lay, x = layer(moe), rows(16)
    lay(x)
    with pytest.raises(ValueError):
        lay(rows(8000)[::2])
    refused(moe, lay, x)
    lay(x)
    lay.backward(x, rows(16))


def test_after_the_workspace_was_grown_by_the_caller(moe):
    lay, x = layer(moe), rows(16)
    lay(x)
    lay.workspace(16)  # large enough: nothing changes
    lay.backward(x, rows(16))
    lay.workspace(4000)
    refused(moe, lay, x)


def test_after_a_forward_that_failed(moe, monkeypatch):
    """A forward that raised may have launched some of its kernels."""
    lay, x = layer(moe), rows(16)
    lay(x)

    def fail(*args, **kw):
        raise moe.MoEError(moe.MOE_ERR_CUDA, "moe_forward", "a test's error")
    with monkeypatch.context() as mp:
        mp.setattr(moe, "moe_forward", fail)
        with pytest.raises(moe.MoEError):
            lay(x)
    refused(moe, lay, x)


def test_another_batch_of_the_same_length(moe):
    """An evaluation batch between the passes: its routing is in the workspace."""
    lay, x, other = layer(moe), rows(16), rows(16)
    lay(x)
    lay(other)
    refused(moe, lay, x)
    lay.backward(other, rows(16))


def test_rows_that_changed_since(moe):
    lay, x = layer(moe), rows(16)
    lay(x)
    x.add_(1)
    refused(moe, lay, x)
    lay(x, out=x)  # the layer's output took the rows' place
    refused(moe, lay, x)


def test_inference_tensors_have_no_version(moe):
    lay = layer(moe)
    with torch.inference_mode():
        x = rows(16)
    lay(x)
    lay.backward(x, rows(16))


@pytest.mark.parametrize("captured", ["forward", "backward"])
def test_writes_between_a_capture_and_its_replays_do_not_count(moe, monkeypatch, captured):
    """A captured forward reads x again at every replay, whatever was written
    to it since the capture; a captured backward has no count to compare."""
    lay, x = layer(moe), rows(16)
    with monkeypatch.context() as mp:
        if captured == "forward":
            mp.setattr(moe, "_version", lambda t: None)
        lay(x)
    if captured == "forward":
        x.add_(1)
    else:
        monkeypatch.setattr(moe, "_version", lambda t: None)
    lay.backward(x, rows(16))


@pytest.mark.parametrize("name,value", [("k", 3), ("renormalize", False), ("scale_inputs", True)])
def test_a_layer_that_changed_since(moe, name, value):
    """These sizes and modes decide where the workspace keeps its parts."""
    lay, x = layer(moe), rows(16)
    lay(x)
    setattr(lay, name, value)
    refused(moe, lay, x)


def test_streams_are_kept_apart(moe):
    lay, x, y = layer(moe), rows(16), rows(16)
    lay(x)
    with pytest.raises(RuntimeError, match="latest forward"):
        lay.backward(x, rows(16), stream=9)
    lay.forward(y, rows(16), stream=9)
    grads = lay.backward(x, rows(16))  # stream 9's batch does not disturb this one's
    lay.backward(y, rows(16), grads, stream=9)
    assert moe.calls[0][1] is moe.calls[2][1] and moe.calls[1][1] is moe.calls[3][1]
    assert moe.calls[0][1] is not moe.calls[1][1]


def test_empty_batches_need_no_forward(moe):
    lay, x = layer(moe), rows(0)
    lay.backward(x, x)
    assert moe.calls[-1][0] == "backward"
