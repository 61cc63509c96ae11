"""GPU checks of the router's balance loss, its counts and its gradient (moe_balance_loss,
moe_balance_loss_grad) against their definitions in 64 bits (tests/mxfp4_ops.py), within the bounds
derived there; whole numbers exactly."""

import pytest
import torch

import routed_moe_layer_amd as rm
from tests import mxfp4_ops as ref
from tests.test_gpu_expert_ops import _gen, _guarded, _intact, _normal, _say

pytestmark = pytest.mark.gpu

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
INF, NAN = float("inf"), float("nan")
COEF = 0.37


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    yield
    torch.cuda.synchronize()


def _logits(g, T, E, bf16, std=1.5):
    return (_normal(g, T, E, std=std, dtype=F32) + _normal(g, E, dtype=F32)).to(BF16 if bf16 else F32)


def _picks(g, T, E, k):
    """Ids with repeats, and some that are no expert."""
    u = torch.empty(T * k, device="cuda").uniform_(0, 1, generator=g)
    ids = (u.square() * (E + 1)).long()
    ids[u > 0.97] = -1
    return torch.where(u < 0.02, 2 ** 31 - 1, ids).to(I32).view(T, k)


def _mask(g, T, kind):
    if kind == "none":
        return None
    if kind == "all":
        return torch.zeros(T, dtype=torch.bool, device="cuda")
    m = torch.empty(T, device="cuda").uniform_(0, 1, generator=g) < 0.7
    return m if kind == "bool" else m.to(U8) * 200


def _loss(z, ids, mask, coef=COEF, stream=None, ws=None):
    T, E = z.shape
    k = ids.shape[1]
    outs = [_guarded(E, dtype=F32), _guarded(E, dtype=F32), _guarded(1, dtype=F32), _guarded(1, dtype=F32)]
    counts, tokens = outs[0][0].view(I32), outs[2][0].view(I32)
    size = rm.moe_balance_workspace_size(T, E)
    if ws is None:
        ws = torch.full((size + 512,), 0x55, dtype=U8, device="cuda")
    torch.cuda.synchronize()
    rm.moe_balance_loss(T, E, k, z, ids, coef, counts, outs[1][0], tokens, outs[3][0], ws,
                        token_mask=mask, logits_bf16=z.dtype == BF16, workspace_bytes=size,
                        stream=stream)
    torch.cuda.synchronize()
    assert all(_intact(g) for _, g in outs)
    assert bool((ws[size:] == 0x55).all())
    return counts, outs[1][0], tokens, outs[3][0]


def _check_loss(z, ids, mask, coef=COEF):
    counts, sums, tokens, loss = _loss(z, ids, mask, coef)
    c, s, tol, n, value, vtol = ref.balance(z, ids, mask, coef)
    assert torch.equal(counts.long(), c) and int(tokens) == n
    assert bool(((sums.double() - s).abs() <= tol).all())
    assert abs(float(loss) - value) <= vtol
    return counts, sums, tokens, loss


def _grad(z, mask, counts, tokens, coef=COEF, g=None, add=None, out=None, stream=None):
    T, E = z.shape
    guard = None
    if out is None:
        out, guard = _guarded(T, E, dtype=z.dtype)
    rm.moe_balance_loss_grad(T, E, z, counts, tokens, coef, out, grad_loss=g, token_mask=mask, add=add,
                             logits_bf16=z.dtype == BF16, stream=stream)
    torch.cuda.synchronize()
    assert guard is None or _intact(guard)
    return out


def _check_grad(z, mask, counts, tokens, coef=COEF, g=None, add=None):
    out = _grad(z, mask, counts, tokens, coef, g, add)
    want, tol = ref.balance_grad(z, mask, counts, int(tokens), coef, 1.0 if g is None else float(g), add)
    half = ref.BF16_HALF_STEP if z.dtype == BF16 else ref.F32_HALF_STEP
    assert bool(((out.double() - want).abs() <= tol + half * 1.001 * (want.abs() + tol)).all())
    return out


SIZES = [(1, 1, 1), (1, 2, 1), (3, 5, 2), (5, 16, 4), (40, 13, 3), (129, 16, 1), (700, 17, 5),
         (33, 64, 8), (3000, 60, 2), (1, 130, 4), (9, 256, 64), (211, 250, 7), (17, 257, 16),
         (1000, 512, 8), (64, 896, 16), (4099, 896, 16), (5, 1001, 3), (300, 1024, 2),
         (77, 1500, 6), (10, 2048, 1), (600, 4096, 16), (8, 4095, 5), (30000, 8, 2), (70001, 33, 1)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("mask", ["none", "bool", "bytes"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_loss_and_gradient(T, E, k, mask, bf16):
    _say(f"balance T={T} E={E} k={k} mask={mask} bf16={bf16}")
    g = _gen(T + 3 * E + k)
    z, ids, m = _logits(g, T, E, bf16), _picks(g, T, E, k), _mask(g, T, mask)
    counts, _, tokens, _ = _check_loss(z, ids, m)
    _check_grad(z, m, counts, tokens)
    scale = torch.tensor([-3.5], device="cuda")
    size = max(1e-30, float(_grad(z, m, counts, tokens).double().std(unbiased=False)))
    add = _normal(g, T, E, std=size, dtype=F32).to(z.dtype)
    want = _check_grad(z, m, counts, tokens, g=scale, add=add)
    # in the place of what was added, and of the logits
    assert torch.equal(_grad(z, m, counts, tokens, g=scale, add=add, out=add.clone()), want)
    again = add.clone()
    assert torch.equal(_grad(z, m, counts, tokens, g=scale, add=again, out=again), want)
    over = z.clone()
    assert torch.equal(_grad(over, m, counts, tokens, g=scale, add=add, out=over), want)


@pytest.mark.parametrize("E", [130, 896, 4096])
def test_rows_that_are_not_aligned(E):
    """Tensors that begin inside another one: any multiple of their values' size."""
    _say(f"balance unaligned E={E}")
    g = _gen(E)
    T = 50
    ids = _picks(g, T, E, 4)
    for bf16 in (False, True):
        z = _logits(g, T, E, bf16)
        counts, sums, tokens, loss = _check_loss(z, ids, None)
        want = _check_grad(z, None, counts, tokens)
        moved = torch.empty(T * E + 1, dtype=z.dtype, device="cuda")[1:].view(T, E)
        moved.copy_(z)
        c2, s2, t2, l2 = _check_loss(moved, ids, None)
        assert torch.equal(c2, counts)
        _check_grad(moved, None, counts, tokens)
        out = torch.zeros(T * E + 1, dtype=z.dtype, device="cuda")
        _grad(z, None, counts, tokens, out=out[1:].view(T, E))
        want64, tol = ref.balance_grad(z, None, counts, int(tokens), COEF, 1.0, None)
        half = ref.BF16_HALF_STEP if bf16 else ref.F32_HALF_STEP
        assert bool(((out[1:].view(T, E).double() - want64).abs() <= tol + half * 1.001 * (want64.abs() + tol)).all())
        assert float(out[0]) == 0.0 and want.shape == (T, E)


@pytest.mark.parametrize("T,E", [(6, 10), (40, 896), (3000, 130)])
def test_nothing_counted(T, E):
    _say(f"balance nothing T={T} E={E}")
    g = _gen(1)
    z, ids = _logits(g, T, E, False), _picks(g, T, E, 3)
    add = _normal(g, T, E, dtype=F32)
    none = _mask(g, T, "all")
    counts, sums, tokens, loss = _loss(torch.full_like(z, NAN), ids, none)
    assert not bool(counts.any()) and not bool(sums.any()) and int(tokens) == 0 and float(loss) == 0
    assert not bool(_grad(torch.full_like(z, NAN), none, counts, tokens).any())
    assert torch.equal(_grad(z, none, counts, tokens, add=add), add)
    # tokens, but no id that counts
    counts, sums, tokens, loss = _check_loss(z, torch.full_like(ids, E), None)
    assert float(loss) == 0 and int(tokens) == T and not bool(counts.any())
    assert not bool(_grad(z, None, counts, tokens).any())
    assert torch.equal(_grad(z, None, counts, tokens, add=add), add)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E", [(6, 10), (40, 896), (300, 130)])
def test_nothing_counted_in_rows_of_nan(T, E, bf16):
    """The loss is 0 and its gradient what is added, whatever the probabilities are."""
    _say(f"balance nothing of NaN T={T} E={E} bf16={bf16}")
    g = _gen(9)
    z = _logits(g, T, E, bf16)
    z[::2, 1], z[1, 2] = NAN, INF
    add = _normal(g, T, E, dtype=z.dtype)
    ids = torch.full((T, 3), -1, dtype=I32, device="cuda")
    counts, sums, tokens, loss = _loss(z, ids, None)
    assert float(loss) == 0 and int(tokens) == T and not bool(counts.any())
    assert not bool(_grad(z, None, counts, tokens).any())
    assert torch.equal(_grad(z, None, counts, tokens, add=add), add)


@pytest.mark.parametrize("T,E", [(20, 12), (20, 50), (100, 896), (9, 4096)])
def test_experts_that_a_token_cannot_take(T, E):
    """Logits of -inf and of the type's lowest value; a row of nothing else; a NaN and a +inf."""
    _say(f"balance -inf T={T} E={E}")
    g = _gen(2)
    lowest = torch.finfo(F32).min
    z, ids = _logits(g, T, E, False), _picks(g, T, E, 3)
    z[1, : E - 1] = -INF
    z[2, ::2] = -INF
    z[3, 1:] = lowest
    z[5] = lowest                                      # equal logits
    z[6] = -INF                                        # no expert at all: p = 0
    counts, sums, tokens, _ = _check_loss(z, ids, None)
    grad = _check_grad(z, None, counts, tokens)
    assert not bool(grad[6].any()) and not bool(grad[2, ::2].any())
    clean = grad.clone()
    z[4, E // 2], z[7, 0] = NAN, INF
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    bad = _grad(z, None, counts, tokens)
    assert bool(bad[[4, 7]].isnan().all())
    others = [t for t in range(T) if t not in (4, 7)]
    assert torch.equal(bad[others], clean[others])
    _, s, _, loss = _loss(z, ids, None)
    assert bool(s.isnan().all()) and bool(loss.isnan())
    # what a mask hides is not looked at
    mask[[4, 7]] = False
    c, _, n, _ = _check_loss(torch.where(mask[:, None], z, 0.0), ids, mask)
    c2, s2, n2, l2 = _loss(z, ids, mask)
    assert torch.equal(c, c2) and int(n) == int(n2) == T - 2 and bool(s2.isfinite().all())
    assert not bool(_grad(z, mask, c2, n2)[[4, 7]].any())


def test_equal_counts_have_no_gradient_and_nearly_equal_ones_a_precise_one():
    _say("balance equal counts")
    T, E = 300, 896
    z = _logits(_gen(3), T, E, False)
    counts = torch.full((E,), 7_000_001, dtype=I32, device="cuda")
    tokens = torch.tensor([T], dtype=I32, device="cuda")
    assert not bool(_grad(z, None, counts, tokens).any())
    counts[5] += 1
    _check_grad(z, None, counts, tokens)
    # a load that is even: the loss is the coefficient
    ids = torch.arange(T * 16, device="cuda").remainder(8).to(I32).view(T, 16)
    loss = _check_loss(_logits(_gen(4), T, 8, False), ids, None)[3]
    assert abs(float(loss) - COEF) <= 1e-5 * COEF


def test_counts_of_many_ranks():
    """Counts and tokens summed over ranks, past 2^31 in all."""
    _say("balance many ranks")
    T, E = 64, 40
    z = _logits(_gen(6), T, E, False)
    counts = torch.randint(1 << 28, 1 << 30, (E,), generator=_gen(7), device="cuda").to(I32)
    tokens = torch.tensor([1 << 30], dtype=I32, device="cuda")
    _check_grad(z, None, counts, tokens)


def test_steep_logits():
    _say("balance steep")
    for std in (0.0, 1e-3, 30.0, 1e4, 1e30):
        z, ids = _normal(_gen(8), 100, 200, std=std, dtype=F32), _picks(_gen(9), 100, 200, 4)
        counts, _, tokens, _ = _check_loss(z, ids, None)
        _check_grad(z, None, counts, tokens)


@pytest.mark.parametrize("T,E,k", [(50, 896, 16), (5000, 896, 8), (40, 12, 2), (9000, 40, 3)])
def test_graph_and_repeats_bit_for_bit(T, E, k):
    """Two graphs and eager calls in turn on one workspace give the first call's bits."""
    _say(f"balance graph T={T} E={E}")
    g = _gen(T)
    z, ids, mask = _logits(g, T, E, False), _picks(g, T, E, k), _mask(g, T, "bool")
    e = lambda *shape, dtype=F32: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    ws = torch.full((rm.moe_balance_workspace_size(T, E),), 0xFF, dtype=U8, device="cuda")
    outs = [e(E, dtype=I32), e(E), e(1, dtype=I32), e(1), e(T, E)]

    def run(stream=None):
        rm.moe_balance_loss(T, E, k, z, ids, COEF, *outs[:4], ws, token_mask=mask, stream=stream)
        rm.moe_balance_loss_grad(T, E, z, outs[0], outs[2], COEF, outs[4], grad_loss=outs[3],
                                 token_mask=mask, stream=stream)

    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side, graphs = torch.cuda.Stream(), []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            run(stream=side)
    for i in range(4):
        for again in (graphs[0].replay, run, graphs[1].replay):
            for t in outs:
                t.zero_()
            again()
            torch.cuda.synchronize()
            for t, w in zip(outs, want):
                assert torch.equal(t, w)


def test_rows_past_32_bit_offsets():
    _say("balance large")
    T, E = 1 << 20, 4096                               # 4.3e9 logits
    z = torch.zeros((T, E), dtype=BF16, device="cuda")
    z[T - 3:] = _logits(_gen(1), 3, E, True)
    ids = torch.zeros((T, 1), dtype=I32, device="cuda")
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[T - 3:] = True
    ids[T - 3:, 0] = torch.tensor([7, 4095, 7], dtype=I32)
    counts, sums, tokens, loss = _loss(z, ids, mask)
    c, s, tol, n, value, vtol = ref.balance(z[T - 3:], ids[T - 3:], None, COEF)
    assert torch.equal(counts.long(), c) and int(tokens) == 3
    assert bool(((sums.double() - s).abs() <= tol).all()) and abs(float(loss) - value) <= vtol
    out = _grad(z, mask, counts, tokens, out=torch.full_like(z, 1.0))
    want, tol = ref.balance_grad(z[T - 3:], None, counts, 3, COEF, 1.0, None)
    assert bool(((out[T - 3:].double() - want).abs() <= tol + 2.0 ** -8 * 1.001 * (want.abs() + tol)).all())
    assert not bool(out[:T - 3].any())


def test_binding_refuses_wrong_tensors():
    _say("balance binding refusals")
    z = torch.zeros((4, 8), device="cuda")
    ids, e = torch.zeros((4, 2), dtype=I32, device="cuda"), torch.zeros(8, device="cuda")
    c, one = torch.zeros(8, dtype=I32, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    ws = torch.zeros(rm.moe_balance_workspace_size(4, 8), dtype=U8, device="cuda")
    with pytest.raises(ValueError, match="token_mask holds 3 elements, not 4"):
        rm.moe_balance_loss(4, 8, 2, z, ids, COEF, c, e, one, e[:1], ws,
                            token_mask=torch.ones(3, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError, match="logits is not contiguous"):
        rm.moe_balance_loss_grad(4, 8, z.view(8, 4).t(), c, one, COEF, z)
