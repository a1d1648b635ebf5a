"""Lists as long as the table of a launch, and around it: every tensor is stepped once."""
import pytest
import torch

from tests.gpu_util import load_moe
from tests.test_gpu_adamw import BF, F32, HYPER, copy, entry, run, verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return load_moe()


@pytest.mark.parametrize("n", [301, 346, 347, 348, 694, 695])
def test_lists_around_a_launch(moe, n):
    es = [entry(1 + (i * 37) % 600, i, p=BF if i % 3 else F32, g=BF, bits=8 if i % 5 == 4 else 32,
                master=i % 3 == 1) for i in range(n)]
    before = [copy(e) for e in es]
    run(moe, es)
    for b, a in zip(before, es):
        verify(b, a, HYPER)
