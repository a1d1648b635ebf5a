"""Failure detection of the gradient's matrix products, without a GPU fault:
the test hook makes each product's first wait run out (1 ms); the call is
reported as a timeout, the context stays usable, and the next call gives the
same gradients as one made before.  CTA pairs, single CTAs, both, and
segments whose ends cut a K step."""
import pytest
import torch

from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return load_moe()


@pytest.mark.parametrize("T,E,k", [(2048, 4, 2), (70, 16, 2), (1000, 16, 2)])
def test_timeout_is_reported_and_recoverable(moe, T, E, k):
    d, f = 256, 384
    g = torch.Generator(device="cuda").manual_seed(T)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
    layer = moe.MoELayer(randn(E, d).float(), randn(E, d, 2 * f) / 16, randn(E, f, d) / 16, k)
    x, dout = randn(T, d), randn(T, d)
    layer(x)
    want = {n: t.clone() for n, t in layer.backward(x, dout).items()}
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    try:
        moe.moe_set_wait_limit_ns(1_000_000)
        moe.moe_debug_inject_wait_timeout(True)
        layer.backward(x, dout)
        status = moe.moe_last_device_error(raise_on_error=False)
    finally:
        moe.moe_debug_inject_wait_timeout(False)
        moe.moe_set_wait_limit_ns(0)
    assert status == moe.MOE_ERR_DEVICE_TIMEOUT
    got = layer.backward(x, dout)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_timeout_in_clusters_that_share_a_tile(moe):
    """Few tiles with a long K axis: every CTA of a cluster must still reach
    the cluster's barriers after its wait ran out."""
    T, E, k, d, f = 24, 2, 1, 2048, 2048
    g = torch.Generator(device="cuda").manual_seed(T)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
    layer = moe.MoELayer(randn(E, d).float(), randn(E, d, 2 * f) / 45, randn(E, f, d) / 45, k)
    x, dout = randn(T, d), randn(T, d)
    layer(x)
    want = {n: t.clone() for n, t in layer.backward(x, dout).items()}
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    try:
        moe.moe_set_wait_limit_ns(1_000_000)
        moe.moe_debug_inject_wait_timeout(True)
        layer.backward(x, dout)
        status = moe.moe_last_device_error(raise_on_error=False)
    finally:
        moe.moe_debug_inject_wait_timeout(False)
        moe.moe_set_wait_limit_ns(0)
    assert status == moe.MOE_ERR_DEVICE_TIMEOUT
    got = layer.backward(x, dout)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    for n in want:
        assert torch.equal(got[n], want[n]), n
