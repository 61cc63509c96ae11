"""GPU checks of every kernel of moe_grouped_gemm_mxfp4 (tests/mxfp4_kernels.py names the problems that
reach them): products, rows without a source, captured and replayed calls, bad scales, rows that no
expert owns, prefix sums that are no prefix sums."""

import pytest
import torch

from tests import mxfp4_ops as ref
from tests.mxfp4_kernels import PROBLEMS, ROW_DIV, WIDE_ROWS, WIDE_WEIGHTS, sizes
from tests.test_gpu_expert_ops import _gen, _guarded, _intact, _say
from tests.test_gpu_mxfp4 import _call, _check, _problem, _random_rows

pytestmark = pytest.mark.gpu

U8, I32 = torch.uint8, torch.int32
NAMES = {k: "x".join(map(str, k[:3])) + ("-wide" if k[3] else "") + "-" + k[4]
         for k in (*PROBLEMS, *WIDE_WEIGHTS)}
each_kernel = pytest.mark.parametrize("kernel", PROBLEMS, ids=[NAMES[k] for k in PROBLEMS])
with_activation = pytest.mark.parametrize("situ", [False, True])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    yield
    torch.cuda.synchronize()


def _make(kernel, situ, kind="uniform", seed=0):
    """The problem, and the one that the definition in 64 bits is worked out on: the same rows, which
    are few of many where their codes take more than 4 GB."""
    R, E, N, K, x_rows = sizes(kernel, situ)
    gathered = kernel[4] != "plain"
    p = _problem(R, E, N, K, situ, gathered, kind, seed)
    assert p["row_div"] == (ROW_DIV if gathered else 1)
    if not kernel[3]:
        assert p["x_rows"] == x_rows
        return p, p
    x = torch.zeros((WIDE_ROWS, K // 2), dtype=U8, device="cuda")
    xs = torch.zeros((WIDE_ROWS, ref.stride(K)), dtype=U8, device="cuda")
    to = torch.randperm(WIDE_ROWS, generator=_gen(seed), device="cuda")[:p["x_rows"]]
    to[0], to[-1] = WIDE_ROWS - 1, WIDE_ROWS - 2
    x[to], xs[to] = p["x"], p["xs"]
    src = p["row_idx"].long()
    wide = dict(p, x=x, xs=xs, x_rows=WIDE_ROWS, to=to,
                row_idx=(to[src // ROW_DIV] * ROW_DIV + src % ROW_DIV).to(I32))
    return wide, p


def _run(p, R, N):
    out, guard = _guarded(R, N)
    _call(p, out)
    torch.cuda.synchronize()
    assert _intact(guard)
    return out


@with_activation
@each_kernel
def test_products_and_rows_without_a_source(kernel, situ):
    _say(f"mxfp4 kernel {NAMES[kernel]} situ={situ}")
    p, plain = _make(kernel, situ, "zipf")
    R, N = p["R"], p["N"]
    _check(plain, _run(p, R, N))
    if kernel[4] == "plain":
        return
    gone = sorted({0, R // 2, R - 1})
    past = {id(q): torch.tensor([-1, ROW_DIV * q["x_rows"], 2 ** 31 - 1], dtype=I32, device="cuda")
            for q in (p, plain)}
    for q in {id(q): q for q in (p, plain)}.values():
        q["row_idx"][gone] = past[id(q)]
    out = _run(p, R, N)
    _check(plain, out)
    assert not bool(out[gone].any())


@with_activation
@each_kernel
def test_graphs_repeat_bit_for_bit(kernel, situ):
    """Two graphs of one call and eager calls in turn."""
    _say(f"mxfp4 kernel graph {NAMES[kernel]} situ={situ}")
    p, plain = _make(kernel, situ, seed=1)
    out, guard = _guarded(p["R"], p["N"])
    _call(p, out)
    torch.cuda.synchronize()
    _check(plain, out)
    want, side, graphs = out.clone(), torch.cuda.Stream(), []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            _call(p, out, stream=side)
    for _ in range(3):
        for again in (graphs[0].replay, lambda: _call(p, out), graphs[1].replay):
            out.zero_()
            again()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    assert _intact(guard)


@with_activation
@each_kernel
def test_bad_scales_stay_in_their_rows_and_columns(kernel, situ):
    """A byte of 255 in one row's scales and one in one expert's weights, first, middle and last block."""
    _say(f"mxfp4 kernel NaN {NAMES[kernel]} situ={situ}")
    p, _ = _make(kernel, situ, "zipf", seed=2)
    R, N, K, E = p["R"], p["N"], p["K"], p["E"]
    clean = _run(p, R, N)
    assert bool(clean.isfinite().all())
    ends = p["cumsum"].tolist()
    src = torch.arange(R, device="cuda") if p["row_idx"] is None else p["row_idx"].long() // p["row_div"]
    # the row behind the middle one, and its expert's weights; each in its own block
    row = R // 2
    expert = next(e for e in range(E) if ends[e] > row)
    for block in sorted({0, K // 64, K // 32 - 1}):
        n = (7 + 31 * block) % N
        at, w_at = (int(src[row]), block), (expert, n + (N if situ and block % 2 else 0), K // 32 - 1 - block)
        kept, w_kept = p["xs"][at].item(), p["ws"][w_at].item()
        p["xs"][at], p["ws"][w_at] = 255, 255
        out = _run(p, R, N)
        nan = (src == at[0])[:, None].repeat(1, N)
        nan[ends[expert - 1] if expert else 0:ends[expert], n] = True
        assert torch.equal(out.isnan(), nan)
        assert torch.equal(out[~nan], clean[~nan])
        p["xs"][at], p["ws"][w_at] = kept, w_kept
    assert torch.equal(_run(p, R, N), clean)


@with_activation
@each_kernel
def test_rows_behind_the_last_expert_stay(kernel, situ):
    """Prefix sums that end before the last row, at none, and inside a tile."""
    _say(f"mxfp4 kernel rows behind {NAMES[kernel]} situ={situ}")
    p, plain = _make(kernel, situ, seed=3)
    R, N = p["R"], p["N"]
    full = p["cumsum"]
    for kept in (0, 1, R // 2 + 1, R - 1):
        p["cumsum"] = plain["cumsum"] = full.clamp(max=kept)
        out = _run(p, R, N)
        _check(plain, out)
        assert bool((out[kept:].view(torch.int16) == 0x55).all())


@with_activation
@each_kernel
def test_prefix_sums_that_are_none(kernel, situ):
    """Below 0, past R, falling: whatever they say, a call ends and stays inside its buffers.  A row
    that some expert claims gets one of its claimants' products, all others stay."""
    _say(f"mxfp4 kernel prefix sums {NAMES[kernel]} situ={situ}")
    p, _ = _make(kernel, situ, seed=4)
    R, E, N = p["R"], p["E"], p["N"]
    odd = torch.randint(-R, 2 * R, (E,), generator=_gen(E), device="cuda").to(I32)
    fall = torch.tensor([R, 0], dtype=I32, device="cuda").repeat(E // 2 + 1)[:E]
    down = (R - torch.arange(E, device="cuda") * (R // E + 1)).clamp(min=-5).to(I32)
    for cumsum in (odd, fall, down, torch.full_like(odd, -3), torch.full_like(odd, 2 ** 31 - 1)):
        p["cumsum"] = cumsum
        out = _run(p, R, N)
        hi = cumsum.long().clamp(0, R)
        lo = torch.cat((hi.new_zeros(1), hi[:-1]))
        mark = torch.zeros(R + 1, dtype=torch.long, device="cuda")
        mark.index_add_(0, lo, (hi > lo).long())
        mark.index_add_(0, hi, -(hi > lo).long())
        claimed = mark.cumsum(0)[:R] > 0
        assert bool((out[~claimed].view(torch.int16) == 0x55).all())
        if cumsum is not odd and cumsum is not fall:   # one claimant a row: nothing is left out
            assert bool((out[claimed].view(torch.int16) != 0x55).any(1).all())


@pytest.mark.parametrize("kernel", WIDE_WEIGHTS, ids=[NAMES[k] for k in WIDE_WEIGHTS])
def test_weights_past_32_bits_with_a_bad_scale_and_rows_behind(kernel):
    _say(f"mxfp4 kernel {NAMES[kernel]}")
    R, E, N, K = WIDE_WEIGHTS[kernel]
    g = _gen(R)
    x, xs = _random_rows(g, R, K, -6)
    w = torch.zeros((2 * N, K // 2), dtype=U8, device="cuda")
    ws = torch.full((2 * N, K // 32), 127, dtype=U8, device="cuda")
    cols = torch.tensor([0, 1, 777, N - 2, N - 1], device="cuda")
    rows = torch.cat((cols, cols + N))
    w[rows], ws[rows] = _random_rows(g, rows.numel(), K, -6)
    p = {"R": R, "E": E, "N": N, "K": K, "situ": True, "x_rows": R, "row_div": 1, "row_idx": None,
         "beta": None, "lam": None, "x": x, "xs": xs, "w": w.view(1, 2 * N, -1), "ws": ws.view(1, 2 * N, -1)}
    for kept in (R, R - 1, 0):
        p["cumsum"] = torch.tensor([kept], dtype=I32, device="cuda")
        out = _run(p, R, N)
        assert bool((out[kept:].view(torch.int16) == 0x55).all())
        if not kept:
            continue
        want, tol, _ = ref.grouped(ref.decode(x, xs), torch.arange(R, device="cuda"), p["cumsum"],
                                   lambda e: ref.decode(w[rows], ws[rows]), cols.numel(),
                                   torch.full((1,), 4.0), torch.full((1,), 25.0), True)
        assert bool(((out[:kept, cols].double() - want[:kept]).abs() <= tol[:kept]).all())
    p["cumsum"] = torch.tensor([R], dtype=I32, device="cuda")
    clean = _run(p, R, N)
    p["xs"][R // 2, 900], ws[2 * N - 1, 2047] = 255, 255
    out, nan = _run(p, R, N), torch.zeros((R, N), dtype=torch.bool, device="cuda")
    nan[R // 2], nan[:, N - 1] = True, True
    assert torch.equal(out.isnan(), nan) and torch.equal(out[~nan], clean[~nan])
