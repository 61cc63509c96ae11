"""GPU checks of how exact the router's probabilities are in moe_balance_loss and
moe_balance_loss_grad.

A probability is exp(x) over a row's sum, x = z - max rounded once.  exp(x) itself is off by one step
of the exponential (two half steps) and the rounding of its correction; the correction's own error and
square are below a hundredth of a half step.  So nothing grows with |x| but the rounding of x, which
is exact where the largest logit is 0."""

import pytest
import torch

from tests import mxfp4_ops as ref
from tests.test_gpu_balance import _grad, _loss
from tests.test_gpu_expert_ops import _gen, _say

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
HALF = ref.F32_HALF_STEP
EXP = 3.02                            # half steps of exp(x) for an exact x


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    yield
    torch.cuda.synchronize()


def softmax64(z):
    """In 64 bits, written out: the library's softmax of more than 1024 doubles a row has fp32's errors."""
    e = torch.exp(z.double() - z.double().amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _far_row(g, T, E, bf16):
    """Rows with one logit of 0 and the others 28 to 86 below it: 4096 of those sum to less than a
    tenth of a half step of 1, so the row's sum is 1 exactly and p is exp(x) as it was computed."""
    z = torch.empty((T, E), device="cuda").uniform_(-86, -28, generator=g).to(BF16 if bf16 else F32)
    top = torch.randint(0, E, (T,), generator=g, device="cuda")
    z[torch.arange(T, device="cuda"), top] = 0.0
    return z, top


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E", [7, 16, 50, 64, 200, 501, 896, 1501, 2048, 4096])
def test_probabilities_far_below_the_largest(E, bf16):
    _say(f"balance far E={E} bf16={bf16}")
    for seed in range(4):
        z, _ = _far_row(_gen(E + seed), 1, E, bf16)
        _, sums, _, _ = _loss(z, torch.zeros((1, 1), dtype=I32, device="cuda"), None)
        want = softmax64(z)[0]
        assert bool(((sums.double() - want).abs() <= (EXP + 0.1) * HALF * want).all())


def test_probabilities_of_two():
    """p = e / (1 + e) and 1 / (1 + e): e's half steps, the sum's, the quotient's and the product's."""
    _say("balance pairs")
    ids = torch.zeros((1, 1), dtype=I32, device="cuda")
    for d in torch.linspace(-9, 4.9, 70).exp2().tolist():
        z = torch.tensor([[0.0, -d]], device="cuda")
        _, sums, _, _ = _loss(z, ids, None)
        want = softmax64(z)[0]
        assert bool(((sums.double() - want).abs() <= (2 * EXP + 3) * HALF * want).all()), d


@pytest.mark.parametrize("E", [7, 64, 200, 501, 896, 1501, 4096])
def test_gradient_far_below_the_largest(E):
    """The row's sum is 1, so sum p c is the count of its largest logit but for a tenth of a half step
    of the largest one.  Roundings: the centred counts, the scale, its product with exp(x), the
    difference of the counts, the last product."""
    _say(f"balance far gradient E={E}")
    T, g = 60, _gen(E)
    z, top = _far_row(g, T, E, False)
    counts = torch.randint(0, 1000, (E,), generator=g, device="cuda").to(I32)
    routed = int(counts.sum())
    coef = torch.tensor(T * routed / E, dtype=F32).item()      # a scale near 1: no result underflows
    tokens = torch.tensor([T], dtype=I32, device="cuda")
    out = _grad(z, None, counts, tokens, coef=coef).double()
    p, c = softmax64(z), counts.double()
    f, d = coef * E / (T * routed), c - c.mean()
    dot = (p * d).sum(1, keepdim=True)
    want = f * p * (d - dot)
    off = HALF * (d.abs() + d[top][:, None].abs() + 0.2 * d.abs().amax())
    tol = f * p * ((d - dot).abs() * (EXP + 0.1 + 4) * HALF + off)
    assert bool(((out - want).abs() <= 1.001 * tol + 2.0 ** -149).all())
