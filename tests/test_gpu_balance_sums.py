"""GPU checks of the router's sums over rows (moe_balance_loss): bounds that count the roundings of
the launch that a call makes, and sums in which every row shows."""

import math

import pytest
import torch

from tests import mxfp4_ops as ref
from tests.test_gpu_balance import _logits, _loss, _mask, _picks
from tests.test_gpu_balance_exact import EXP, HALF, softmax64
from tests.test_gpu_expert_ops import _gen, _say

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    yield
    torch.cuda.synchronize()


# rows of lanes, registers and workgroups of every kind, one launch and two
SIZES = [(1, 1), (3, 5), (129, 16), (1025, 16), (30000, 8), (1 << 20, 13), (33, 64), (257, 40), (70001, 33),
         (5, 256), (64, 130), (65, 130), (6001, 256), (300, 512), (20000, 300), (64, 896), (65, 896),
         (4099, 896), (16384, 1024), (32, 1500), (33, 1500), (9000, 2048), (8, 4095), (5000, 4096)]


def _launch(T, E):
    """(additions of a sum over rows, additions of a row's sum)."""
    waves, slots = (16, 8) if E <= 1024 else (8, 2)
    per_wave = 16 if E <= 16 else 4 if E <= 64 else 1
    rows, most = waves * per_wave, 256 if E <= 1024 else 512
    G = 1 if T <= 4 * rows else min((T + rows - 1) // rows, most)
    # a lane's rows, the rows of a wavefront, the wavefronts by their places and these, the rounding
    # behind the sum in doubles
    over = (T + G * rows - 1) // (G * rows) + int(math.log2(per_wave)) + waves // slots - 1 + slots - 1 + (G > 1)
    values = next(v for v, n in ((4, 256), (8, 512), (16, 1024), (32, 2048), (64, 4096)) if E <= n)
    return over, values - 1 + int(math.log2(64 // per_wave))


@pytest.mark.parametrize("mask", ["none", "bool"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E", SIZES)
def test_sums_within_the_roundings_of_their_launch(T, E, bf16, mask):
    """Tight enough for one row more or less to lie outside, up to some 10^5 rows."""
    _say(f"balance sums T={T} E={E} bf16={bf16} mask={mask}")
    g = _gen(T + E)
    z, m, k = _logits(g, T, E, bf16), _mask(g, T, mask), min(3, E)
    ids = _picks(g, T, E, k)
    counts, sums, tokens, loss = _loss(z, ids, m, coef=0.37)
    over, inside = _launch(T, E)
    x = z.double() - z.double().amax(1, keepdim=True)
    p = softmax64(z)
    own = EXP + x.abs()
    rel = HALF * (own + (p * own).sum(1, keepdim=True) + inside + 1)    # and the quotient's rounding
    if m is not None:
        p = torch.where(m[:, None], p, 0.0)
    want = p.sum(0)
    tol = 1.001 * ((rel * p).sum(0) + over * HALF * want) + T * 2.0 ** -126
    assert bool(((sums.double() - want).abs() <= tol).all())
    if 1000 < T < 100000:
        assert bool((tol < 0.5 * want / T).all())      # half of an expert's mean probability
    c, _, _, n, value, _ = ref.balance(z, ids, m, 0.37)
    assert torch.equal(counts.long(), c) and int(tokens) == n
    f = 0.37 * E / (max(1, n) * max(1, int(c.sum())))
    # in doubles; coef itself is rounded to fp32
    assert abs(float(loss) - value) <= f * float((c.double() * tol).sum()) + 2.5 * HALF * abs(value)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E", SIZES)
def test_every_row_counts_once(T, E, bf16, masked):
    """Rows that can take one expert only, each its own: their sums are whole numbers."""
    _say(f"balance one-hot T={T} E={E} bf16={bf16} masked={masked}")
    g = _gen(T + 2 * E)
    to = (torch.randperm(T, generator=g, device="cuda") % E).view(T, 1)
    z = torch.full((T, E), -INF, dtype=BF16 if bf16 else F32, device="cuda")
    z.scatter_(1, to, 2.5)
    m = _mask(g, T, "bytes" if masked else "none")
    counts, sums, tokens, loss = _loss(z, to.to(I32), m)
    live = to[:, 0] if m is None else to[m != 0, 0]
    want = torch.bincount(live, minlength=E)
    assert torch.equal(sums.double(), want.double()) and torch.equal(counts.long(), want)
    assert int(tokens) == live.numel()
