"""AdamW.step on a stream that is not the tensors' own: what it reads and writes there is
not given to others before that stream is done with it, also when the optimizer is
dropped right after the call."""
import pytest
import torch

from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    return load_moe()


@pytest.mark.parametrize("way", ["stream", "handle", "current"])
@pytest.mark.parametrize("bits,master,max_norm", [(32, True, 1.0), (8, False, None)])
def test_dropped_after_a_step_elsewhere(moe, bits, master, max_norm, way):
    sizes = [1 << 20, 3_000_001, 700]
    gen = torch.Generator(device="cuda").manual_seed(bits)
    start = [torch.randn(n, generator=gen, device="cuda").to(BF) for n in sizes]
    grads = [torch.randn(n, generator=gen, device="cuda").to(BF) for n in sizes]
    results = []
    for held in (False, True):
        params = [p.clone() for p in start]
        opt = moe.AdamW(params, [g.clone() for g in grads], 1e-2, bits=bits, master=master, max_norm=max_norm)
        torch.cuda.synchronize()
        if not held:
            opt.step()
            del opt
            torch.cuda.empty_cache()  # (no free memory for what is allocated below but the dropped)
        else:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                torch.cuda._sleep(100_000_000)
                if way == "current":
                    opt.step()
            if way != "current":
                opt.step(stream=side if way == "stream" else side.cuda_stream)
            sizes_of = {t.numel() * t.element_size() for d in opt.tensors for t in d.values()
                        if isinstance(t, torch.Tensor)}
            del opt  # its gradients too
            fill = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in sizes_of for _ in range(6)]
            assert not side.query()  # still held up
            side.synchronize()
            del fill
        torch.cuda.synchronize()
        assert moe.moe_last_device_error() == moe.MOE_OK
        results.append(params)
    for a, b in zip(*results):
        assert torch.equal(a, b)
