"""The library's first calls on a device made by several host threads at once,
each on a stream of its own: what is set up on the device's first use is seen
whole by every thread, so their results are the serial ones, bit for bit."""
import os
import subprocess
import sys

import pytest

from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import threading
import torch
from token_dispatch_grouped_fp32_gb300 import moe

def run(dtype, T, d, E, k, f):
    g = torch.Generator(device="cuda").manual_seed(T)
    def randn(*shape, std=1.0, t=dtype):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(t)
    w = (randn(E, d, std=d ** -0.5, t=torch.float32), randn(E, d, 2 * f, std=d ** -0.5),
         randn(E, f, d, std=f ** -0.5))
    x, dout = randn(T, d), randn(T, d)
    torch.cuda.synchronize()
    n, results, errors = 3, [None] * 3, []
    barrier = threading.Barrier(n)

    def thread(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                layer = moe.MoELayer(*w, k)
                out = torch.empty_like(x)
                barrier.wait()
                layer(x, out)
                grads = layer.backward(x, dout)
            stream.synchronize()
            results[i] = {"out": out, **grads}
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=thread, args=(i,)) for i in range(n)]
    for t in threads: t.start()
    for t in threads: t.join()
    assert not errors, errors
    layer = moe.MoELayer(*w, k)
    want = {"out": layer(x), **layer.backward(x, dout)}
    torch.cuda.synchronize()
    moe.moe_last_device_error()
    for r in results:
        for name in want:
            assert torch.equal(r[name], want[name]), name

run(torch.bfloat16, 1500, 256, 16, 4, 256)
run(torch.bfloat16, 20, 256, 16, 4, 256)
run(torch.float32, 200, 128, 8, 2, 128)
print("equal")
"""


def test_first_calls_of_several_threads():
    load_moe()
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "equal", r.stdout + r.stderr
