"""GPU checks of moe_balance_loss_grad where its scale, grad_loss coef num_experts / (tokens sum
counts), leaves fp32's range and the gradient does not."""

import pytest
import torch

from tests import mxfp4_ops as ref
from tests.test_gpu_balance import _grad, _logits
from tests.test_gpu_expert_ops import _gen, _normal, _say

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    yield
    torch.cuda.synchronize()


def _check(z, counts, tokens, coef, g=None, add=None):
    out = _grad(z, None, counts, tokens, coef=coef, g=g, add=add).double()
    want, tol = ref.balance_grad(z, None, counts, int(tokens), torch.tensor(coef, dtype=F32).item(),
                                 1.0 if g is None else float(g), add)
    assert bool(want.isfinite().all()) and bool((want != 0).any())
    # half a step of the value, and below a type's smallest normal number half of its smallest step:
    # BF16's steps are 2^-126 * 2^-7 there, fp32's 2^-126 * 2^-23
    half, least = (ref.BF16_HALF_STEP, 2.0 ** -134) if z.dtype == BF16 else (ref.F32_HALF_STEP, 2.0 ** -150)
    assert bool(((out - want).abs() <= tol + half * 1.001 * (want.abs() + tol) + least).all())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E", [12, 60, 200, 896, 4096])
def test_gradient_whose_scale_leaves_fp32s_range(E, bf16):
    """A scale beyond the largest or below the smallest fp32 number, where the
    gradient itself is neither."""
    _say(f"balance gradient scales E={E} bf16={bf16}")
    T, g = 5, _gen(E)
    z = _normal(g, T, E, std=0.1, dtype=F32).to(BF16 if bf16 else F32)
    one = torch.ones(1, dtype=I32, device="cuda")
    counts = torch.zeros(E, dtype=I32, device="cuda")
    counts[E // 2] = 1
    _check(z, counts, one, 1e38)                               # coef E is infinite in fp32
    _check(z, counts, one, 1e38, g=torch.tensor([-0.5], device="cuda"))
    _check(z, counts, one, 1e30, g=torch.tensor([1e8], device="cuda"))
    many = torch.full((1,), 1 << 21, dtype=I32, device="cuda")
    counts = torch.randint(1 << 20, 1 << 26, (E,), generator=g, device="cuda").to(I32)
    _check(z, counts, many, 1e-36, g=torch.tensor([1e30], device="cuda"))
    _check(z, counts, many, 1e-30)
    add = _normal(g, T, E, std=1e-30, dtype=F32).to(z.dtype)
    _check(z, counts, many, 1e-36, g=torch.tensor([1e25], device="cuda"), add=add)


@pytest.mark.parametrize("E", [12, 896])
def test_equal_counts_have_no_gradient_under_any_scale(E):
    _say(f"balance equal counts, large scale E={E}")
    z = _logits(_gen(E), 6, E, False)
    counts, one = torch.ones(E, dtype=I32, device="cuda"), torch.ones(1, dtype=I32, device="cuda")
    for coef, g in ((3.3e38, None), (1e38, 1e30), (-1e38, 1e-30)):
        g = None if g is None else torch.tensor([g], device="cuda")
        assert torch.equal(_grad(z, None, counts, one, coef=coef, g=g), torch.zeros_like(z))


@pytest.mark.parametrize("E", [16, 64, 896, 4096])
def test_large_counts_that_cancel_under_a_large_scale(E):
    """Half of the experts share every row and every count: sum p c is their count, the gradient 0, and
    the sum on the way to it many times as large as one count."""
    _say(f"balance cancelling counts, large scale E={E}")
    z = torch.full((5, E), -float("inf"), device="cuda")
    z[:, : E // 2] = 1.25
    counts = torch.zeros(E, dtype=I32, device="cuda")
    counts[: E // 2] = 1 << 30                         # centred: 2^29 and -2^29
    one = torch.ones(1, dtype=I32, device="cuda")
    for coef, g in ((3e38, 1e38), (3e38, 1e30), (1e30, 1e20)):
        out = _grad(z, None, counts, one, coef=coef, g=torch.tensor([g], device="cuda"))
        assert torch.equal(out, torch.zeros_like(z))
