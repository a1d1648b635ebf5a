"""moe_clip_grad_norm where squares leave fp32's range while the norm does not:
the tolerances of tests/test_gpu_clip.py hold there too, as the powers of two
that are taken out of such squares are exact."""
import pytest
import torch

from tests.gpu_util import load_moe
from tests.test_gpu_clip import check, clip

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def fill(n, dtype, *values):
    """n elements that take the values in turn, with both signs."""
    t = torch.tensor(values, device="cuda", dtype=torch.float64).repeat(-(-n // len(values)))[:n]
    return (t * (1 - 2 * (torch.arange(n, device="cuda") % 3 == 0).double())).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 7, 300, 16384, 70001])
@pytest.mark.parametrize("values", [
    (1e19,), (3e18,), (1e25,),               # the sum of a few, or one square, past 3e38
    (1e-23,), (1e-25,), (1e-30,),            # squares below fp32's smallest
    (1e19, 1.0, 1e-25, 0.0), (1e-25, 1e-30, 0.0), (1.0, 1e-25),
], ids=str)
def test_values(moe, dtype, n, values):
    g = fill(n, dtype, *values)
    for max_norm in (1.0, 1e-26):
        check(moe, [g], max_norm, [torch.empty_like(g)])


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_ends_of_the_range(moe, dtype):
    big = fill(3, dtype, 1.5e38)             # their norm is 2.6e38
    check(moe, [big], 1.0, [torch.empty_like(big)])
    assert clip(moe, [fill(8, dtype, 3e38)], 1.0, [None]) == float("inf")  # 8.5e38 is not a float
    small = fill(1 << 20, dtype, 1e-40)      # subnormal; their norm is 1e-37
    check(moe, [small], 1.0, [torch.empty_like(small)])


def test_tensors_of_unlike_scales(moe):
    """Each tensor's squares have their own range; the sum across them is fp64."""
    grads = [fill(40000, torch.float32, 1e20), fill(33, torch.bfloat16, 1e-25),
             fill(70000, torch.bfloat16, 0.5), torch.zeros(20000, device="cuda")]
    check(moe, grads, 1.0, [torch.empty_like(g) for g in grads])
    check(moe, grads[1:2] + grads[3:], 1.0, [torch.empty_like(g) for g in grads[1:2] + grads[3:]])


@pytest.mark.parametrize("dtype", DTYPES)
def test_zeros_and_non_finite_values_beside_them(moe, dtype):
    zeros = fill(40000, dtype, 0.0)
    assert clip(moe, [zeros], 1.0, [zeros]) == 0.0 and (zeros == 0).all()
    g = fill(40000, dtype, 1e20, 1e-25)
    g[777] = float("-inf")
    assert clip(moe, [g], 1.0, [None]) == float("inf")
    g[9] = float("nan")
    norm = clip(moe, [g], 1.0, [None])
    assert norm != norm
