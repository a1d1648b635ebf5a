"""moe_clip_grad_norm against a 64-bit norm.

Tolerances: within 16384 elements a thread adds 64 squares in fp32 and the
rest is fp64, so the sum of squares (all terms positive) is within 66 u32 of
itself, its root within 33 u32, rounded once: 34 u32 relative (u32 = 2^-24).
The scale max_norm / (norm + 1e-6) adds two roundings, the product one, and
the output's own rounding (u32 or, for bf16, 2^-8)."""
import pytest
import torch

from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu
U32, UB = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def clip(moe, grads, max_norm, outs):
    ws = torch.full((moe.moe_clip_grad_norm_workspace_size(),), 255, dtype=torch.uint8, device="cuda")
    norm = torch.full((1,), float("nan"), device="cuda")
    moe.moe_clip_grad_norm(moe.grad_list(grads, outs), max_norm, norm, ws)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    return float(norm)


def check(moe, grads, max_norm, outs):
    inputs = [g.clone() for g in grads]
    want = float(sum((g.double() ** 2).sum() for g in inputs)) ** 0.5 if inputs else 0.0
    norm = clip(moe, grads, max_norm, outs)
    assert abs(norm - want) <= 34 * U32 * want
    coef = min(1.0, max_norm / (want + 1e-6))
    for g, o in zip(inputs, outs):
        if o is None:
            continue
        ref = g.double() * coef
        tol = 40 * U32 * ref.abs() + (UB if g.dtype == torch.bfloat16 else U32) * ref.abs() + 2.0 ** -149
        if g.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -133
        assert ((o.double() - ref).abs() <= tol).all()
        if coef == 1.0:
            assert torch.equal(o, g)


def tensors(sizes, dtypes, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(t) for n, t in zip(sizes, dtypes)]


MIX = [torch.bfloat16, torch.float32, torch.bfloat16]


@pytest.mark.parametrize("max_norm", [0.0, 1e-3, 1.0, 1e6])
@pytest.mark.parametrize("sizes", [[1], [7, 8, 9], [16383, 16384, 16385], [100000, 1, 33000],
                                   [0, 5, 0, 70000]], ids=str)
def test_sizes(moe, sizes, max_norm):
    dtypes = [MIX[i % 3] for i in range(len(sizes))]
    grads = tensors(sizes, dtypes, len(sizes))
    check(moe, grads, max_norm, [torch.full_like(g, 9.0) for g in grads])


@pytest.mark.parametrize("n", [511, 512, 513, 1400])
def test_many_tensors(moe, n):
    sizes = [1 + (37 * i) % 900 for i in range(n)]
    grads = tensors(sizes, [MIX[i % 3] for i in range(n)], n)
    check(moe, grads, 0.5, [torch.empty_like(g) for g in grads])


def test_in_place_and_norm_only(moe):
    grads = tensors([5000, 123, 70001], MIX, 4)
    keep = grads[1].clone()
    check(moe, grads, 2.0, [grads[0], None, grads[2]])
    assert torch.equal(grads[1], keep)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("a,b", [(0, 0), (1, 1), (3, 3), (1, 2), (5, 0), (0, 7)])
def test_offsets_into_a_flat_buffer(moe, dtype, a, b):
    """Sources and copies at every alignment of their element type."""
    n = 40000
    g = torch.Generator(device="cuda").manual_seed(a * 8 + b)
    src = torch.randn(n + 16, generator=g, device="cuda").to(dtype)
    dst = torch.full((n + 16,), 7.0, device="cuda", dtype=dtype)
    check(moe, [src[a:a + n]], 1.0, [dst[b:b + n]])
    assert (dst[:b] == 7.0).all() and (dst[b + n:] == 7.0).all()


def test_no_tensors_and_no_elements(moe):
    assert clip(moe, [], 1.0, []) == 0.0
    empty = [torch.empty(0, device="cuda"), torch.empty(0, device="cuda", dtype=torch.bfloat16)]
    assert clip(moe, empty, 1.0, empty) == 0.0


def test_infinite_and_nan_gradients(moe):
    """The formula is followed: an infinite norm scales finite gradients to
    zero (and inf * 0 is NaN), a NaN norm makes every gradient NaN."""
    a, b = tensors([100, 20000], [torch.float32, torch.bfloat16], 3)
    b[777] = float("inf")
    outs = [torch.empty_like(a), torch.empty_like(b)]
    assert clip(moe, [a, b], 1.0, outs) == float("inf")
    assert (outs[0] == 0).all() and torch.isnan(outs[1][777]) and (outs[1][:777] == 0).all()
    a[5] = float("nan")
    norm = clip(moe, [a, b], 1.0, outs)
    assert norm != norm and torch.isnan(outs[0]).all() and torch.isnan(outs[1].float()).all()


def test_large_and_tiny_values(moe):
    """Squares across tensors are added in fp64: no overflow of the sum while
    single squares fit fp32, and small tensors count beside large ones."""
    big = torch.full((1 << 20,), 1e18, device="cuda")
    check(moe, [big], 1.0, [torch.empty_like(big)])
    small = tensors([1000], [torch.float32], 9, std=1e-15)
    check(moe, small, 1.0, [torch.empty_like(small[0])])


def test_repeats_bit_for_bit(moe):
    grads = tensors([3_000_001, 17, 999_999], MIX, 5)
    outs = [[torch.empty_like(g) for g in grads] for _ in range(2)]
    norms = [clip(moe, grads, 1.0, o) for o in outs]
    assert norms[0] == norms[1]
    for a, b in zip(*outs):
        assert torch.equal(a, b)
