"""MoELayer.backward refuses buffers that its kernels would write past or could
not reach, before any launch."""
import pytest
import torch

BF = torch.bfloat16
D, E, K, F = 64, 8, 2, 128


@pytest.fixture
def lay(monkeypatch):
    from token_dispatch_grouped_fp32_gb300 import build
    build.build()
    from token_dispatch_grouped_fp32_gb300 import moe
    monkeypatch.setattr(moe, "_stream", lambda s: 7 if s is None else int(s))
    calls = []
    monkeypatch.setattr(moe, "moe_forward", lambda *a, **kw: None)
    monkeypatch.setattr(moe, "moe_backward", lambda *a, **kw: calls.append(a))
    layer = moe.MoELayer(torch.zeros(E, D), torch.zeros(E, D, 2 * F, dtype=BF),
                         torch.zeros(E, F, D, dtype=BF), K)
    layer.calls = calls
    return layer


def buffers(lay, x):
    return {"x": torch.empty_like(x), "Wr": torch.empty_like(lay.Wr),
            "W_gate_up": torch.empty_like(lay.W_gate_up), "W_down": torch.empty_like(lay.W_down)}


def test_a_bias_gradient_without_a_bias(lay):
    """The bias gradient is written whenever its buffer is given."""
    x = torch.zeros(16, D, dtype=BF)
    lay(x)
    grads = buffers(lay, x)
    for bad in (torch.zeros(E - 1), torch.zeros(E, dtype=BF), torch.zeros(0)):
        with pytest.raises(ValueError, match="logit_bias"):
            lay.backward(x, x.clone(), {**grads, "logit_bias": bad})
    assert not lay.calls
    bias = torch.zeros(E)
    lay.backward(x, x.clone(), {**grads, "logit_bias": bias})
    assert lay.calls[0][9] is bias
    lay.backward(x, x.clone(), {**grads, "logit_bias": None})
    assert lay.calls[1][9] is None


@pytest.mark.parametrize("name", ["dout", "x", "Wr", "W_gate_up", "W_down", "logit_bias"])
def test_tensors_of_another_device(lay, name):
    x = torch.zeros(16, D, dtype=BF)
    lay(x)
    grads, dout = {**buffers(lay, x), "logit_bias": torch.zeros(E)}, x.clone()
    if name == "dout":
        dout = dout.to("meta")
    else:
        grads[name] = grads[name].to("meta")
    with pytest.raises(ValueError, match="device|gradient of " + name):
        lay.backward(x, dout, grads)
    assert not lay.calls
