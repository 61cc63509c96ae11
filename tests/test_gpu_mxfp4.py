"""GPU checks of the microscaled FP4 operators (moe_quantize_mxfp4, moe_dequantize_mxfp4,
moe_grouped_gemm_mxfp4) against their definitions in 64 bits (tests/mxfp4_ops.py): codes, scales
and decoded values exactly, products within the bound derived there."""

import pytest
import torch

import routed_moe_layer_amd as rm
from tests import mxfp4_ops as ref
from tests.test_gpu_expert_ops import _gen, _guarded, _intact, _normal, _say

pytestmark = pytest.mark.gpu

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    yield
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------------------
# Rows.
# ---------------------------------------------------------------------------------------
def _rows_check(x):
    rows, K = x.shape
    codes, guard_c = _guarded(rows, K // 2, dtype=U8)
    scales, guard_s = _guarded(rows, ref.stride(K), dtype=U8)
    rm.moe_quantize_mxfp4(x, rows, K, codes, scales)
    torch.cuda.synchronize()
    assert _intact(guard_c) and _intact(guard_s)
    want_c, want_s = ref.quantize(x)
    assert torch.equal(scales, want_s)
    assert torch.equal(codes, want_c)
    out, guard_o = _guarded(rows, K)
    rm.moe_dequantize_mxfp4(codes, scales, rows, K, out)
    torch.cuda.synchronize()
    assert _intact(guard_o)
    want = ref.decode(codes, scales).to(BF16)
    nan = want.isnan()
    assert torch.equal(out.isnan(), nan)
    assert torch.equal(out.view(torch.int16)[~nan], want.view(torch.int16)[~nan])
    return codes, scales


@pytest.mark.parametrize("rows,K", [(1, 32), (1, 96), (3, 64), (2, 128), (7, 160), (37, 2912),
                                    (64, 3584), (5, 7168), (1000, 288), (3, 65536), (4099, 416),
                                    (70001, 32), (2050, 4096)])
def test_rows(rows, K):
    _say(f"mxfp4 rows {rows} x {K}")
    x = _normal(_gen(rows + K), rows, K)
    x *= torch.exp2(torch.randint(-12, 12, (rows, 1), generator=_gen(K), device="cuda").float()).to(BF16)
    _rows_check(x)


def test_rows_of_every_bf16_value():
    """Every BF16 pattern as a block's largest value, and as the small one beside others."""
    _say("mxfp4 every value")
    bits = torch.arange(65536, device="cuda", dtype=I32).to(torch.int16)
    x = torch.zeros((65536, 32), dtype=torch.int16, device="cuda")
    x[:, 5] = bits
    _rows_check(x.view(BF16))
    # shuffled: neighbours of any size, every pattern somewhere
    order = torch.randperm(65536, generator=_gen(3), device="cuda")
    _rows_check(bits[order].view(BF16).view(512, 128))
    finite = bits[bits.view(BF16).isfinite()]
    order = torch.randperm(finite.numel(), generator=_gen(4), device="cuda")[:65024]
    _rows_check(finite[order].view(BF16).view(32, 2032)[:, :2016].contiguous())


@pytest.mark.parametrize("exp", [-133, -127, -126, -125, -124, -60, 0, 90, 125, 126, 127])
def test_rows_on_the_borders_of_the_codes(exp):
    """Multiples of 1/32 up to 8 under one scale: every border between two codes and its
    neighbours, from BF16's subnormals to its largest values."""
    _say(f"mxfp4 borders 2^{exp}")
    v = torch.arange(0, 256, device="cuda").double() / 32
    v = torch.stack((v, -v)).view(-1, 16)
    v = torch.cat((torch.full((32, 1), 4.0, device="cuda", dtype=torch.float64), v,
                   torch.zeros((32, 15), device="cuda", dtype=torch.float64)), 1)
    _rows_check((v * 2.0 ** (exp - 2)).to(BF16))


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_rows_with_a_bad_value_mark_its_block_only(bad):
    _say(f"mxfp4 {bad}")
    x = _normal(_gen(8), 5, 224)
    x[3, 100] = bad
    codes, scales = _rows_check(x)
    assert int(scales[3, 3]) == 255 and not bool(codes[3, 48:64].any())
    assert int((scales == 255).sum()) == 1


def test_rows_of_every_scale_decode():
    _say("mxfp4 every scale")
    codes = torch.randint(0, 256, (256, 16), generator=_gen(2), device="cuda").to(U8)
    scales = torch.zeros((256, 4), dtype=U8, device="cuda")
    scales[:, 0] = torch.arange(256, device="cuda")
    scales[:, 1:] = 255                                # past K / 32: not read as scales
    out = torch.empty((256, 32), dtype=BF16, device="cuda")
    rm.moe_dequantize_mxfp4(codes, scales, 256, 32, out)
    want = ref.decode(codes, scales).to(BF16)
    assert torch.equal(out.isnan(), want.isnan()) and bool(want[255].isnan().all())
    assert torch.equal(out[:255].view(torch.int16), want[:255].view(torch.int16))


def test_rows_past_32_bit_offsets():
    _say("mxfp4 large rows")
    rows, K = 1100000, 4096                            # 4.5e9 values
    x = torch.zeros((rows, K), dtype=BF16, device="cuda")
    x[rows - 3:] = _normal(_gen(4), 3, K)
    codes = torch.empty((rows, K // 2), dtype=U8, device="cuda")
    scales = torch.empty((rows, K // 32), dtype=U8, device="cuda")
    rm.moe_quantize_mxfp4(x, rows, K, codes, scales)
    want = ref.quantize(x[rows - 3:])
    assert torch.equal(codes[rows - 3:], want[0]) and torch.equal(scales[rows - 3:], want[1])
    assert not bool(codes[:rows - 3].any()) and not bool(scales[:rows - 3].any())
    rm.moe_dequantize_mxfp4(codes, scales, rows, K, x)
    assert torch.equal(x[rows - 3:].double(), ref.decode(*want))


# ---------------------------------------------------------------------------------------
# Products by expert.
# ---------------------------------------------------------------------------------------
def _counts(kind, R, E, g):
    if kind == "one":
        c = torch.zeros(E, dtype=torch.long)
        c[E // 2] = R
        return c
    p = 1.0 / torch.arange(1, E + 1) if kind == "zipf" else torch.ones(E)
    picks = torch.multinomial(p, R, replacement=True, generator=torch.Generator().manual_seed(R + E))
    return torch.bincount(picks, minlength=E)


def _random_rows(g, rows, K, mid):
    """Random codes, scales around 2^mid; bytes past K / 32 are no scales and hold anything."""
    codes = torch.randint(0, 256, (rows, K // 2), generator=g, device="cuda").to(U8)
    scales = torch.randint(127 + mid - 3, 127 + mid + 4, (rows, ref.stride(K)), generator=g,
                           device="cuda").to(U8)
    return codes, scales


def _problem(R, E, N, K, situ, gather, kind="uniform", seed=0):
    g = _gen(seed + 7 * R + E + N + K)
    Nw, k = N * (2 if situ else 1), 3 if gather else 1
    x_rows = (R + k - 1) // k if gather else R
    # scales whose products have a standard deviation of a few units
    mid = -round((3 + 0.5 * torch.tensor(float(K)).log2().item()) / 2)
    p = {"R": R, "E": E, "N": N, "K": K, "situ": situ, "x_rows": x_rows, "row_div": k,
         "row_idx": None, "beta": None, "lam": None}
    p["x"], p["xs"] = _random_rows(g, x_rows, K, mid)
    w, ws = _random_rows(g, E * Nw, K, mid)
    p["w"], p["ws"] = w.view(E, Nw, -1), ws.view(E, Nw, -1)
    if gather:
        p["row_idx"] = torch.randperm(x_rows * k, generator=g, device="cuda")[:R].to(I32)
    p["cumsum"] = _counts(kind, R, E, g).cumsum(0).to(I32).cuda()
    if situ:
        p["beta"] = torch.empty(E, device="cuda").uniform_(3, 5, generator=g)
        p["lam"] = torch.empty(E, device="cuda").uniform_(20, 30, generator=g)
    return p


def _call(p, out, **kw):
    rm.moe_grouped_gemm_mxfp4(p["R"], p["N"], p["K"], p["E"], p["x"], p["xs"], p["cumsum"], p["w"],
                              p["ws"], out, x_rows=p["x_rows"], row_idx=p["row_idx"],
                              row_div=p["row_div"], situ=p["situ"], situ_beta=p["beta"],
                              situ_linear_beta=p["lam"], **kw)


def _want(p):
    if p["row_idx"] is None:
        src = torch.arange(p["R"], device="cuda")
    else:
        src = p["row_idx"].long().div(p["row_div"], rounding_mode="floor")
    src = torch.where((src >= 0) & (src < p["x_rows"]), src, -1)
    return ref.grouped(ref.decode(p["x"], p["xs"]), src, p["cumsum"],
                       lambda e: ref.decode(p["w"][e], p["ws"][e]), p["N"], p["beta"], p["lam"],
                       p["situ"])


def _check(p, out):
    want, tol, written = _want(p)
    bad = (out.double() - want).abs() > tol
    bad |= ~out.isfinite()
    bad[~written] = False
    assert not bool(bad.any()), f"{int(bad.sum())} outputs outside the bound"
    untouched = out.view(torch.int16)[~written]
    assert bool((untouched == 0x55).all()), "a row behind the last expert's was written"


GROUPED = [
    # R, E, N, K, counts
    (1, 1, 1, 32, "uniform"), (1, 5, 33, 64, "uniform"), (7, 3, 17, 96, "uniform"),
    (16, 1, 64, 256, "one"), (40, 16, 96, 800, "uniform"), (64, 4, 130, 2080, "zipf"),
    (65, 2, 64, 512, "one"), (200, 900, 40, 288, "uniform"), (333, 7, 257, 1056, "zipf"),
    (1000, 9, 128, 1024, "one"), (2500, 20, 384, 2048, "zipf"), (700, 3, 1000, 544, "uniform"),
    (3000, 2, 256, 4096, "uniform"), (129, 1, 36, 7200, "one"), (50, 10240, 16, 64, "uniform"),
    # every tile size, with items enough and too few, ragged N and K and odd chunk counts
    (33, 1, 1100, 4128, "one"), (600, 1, 5000, 544, "one"), (20000, 3, 1031, 800, "zipf"),
    (9000, 16, 3000, 288, "zipf"), (5000, 600, 2051, 288, "zipf"), (70000, 2500, 24, 128, "uniform"),
    (300000, 5000, 40, 64, "zipf"), (60, 10240, 17, 4128, "uniform"), (31000, 65, 96, 96, "uniform"),
    (1000, 1, 20000, 2080, "one"), (2, 1, 7181, 7168, "one"), (17, 1, 300, 65536, "one"),
    (260, 1, 520, 768, "one"), (5000, 1, 2048, 1280, "one"), (12000, 8, 1500, 640, "zipf"),
]


@pytest.mark.parametrize("situ,gather", [(False, False), (True, True), (False, True), (True, False)])
@pytest.mark.parametrize("R,E,N,K,kind", GROUPED)
def test_grouped(R, E, N, K, kind, situ, gather):
    _say(f"mxfp4 grouped R={R} E={E} N={N} K={K} {kind} situ={situ} gather={gather}")
    p = _problem(R, E, N, K, situ, gather, kind)
    out, guard = _guarded(R, N)
    _call(p, out)
    torch.cuda.synchronize()
    assert _intact(guard)
    _check(p, out)


@pytest.mark.parametrize("K", list(range(32, 1056, 32)))
def test_grouped_lengths(K):
    """Every count of blocks around the chunks that the kernels take, with few rows and many."""
    _say(f"mxfp4 grouped K={K}")
    for R, E, N in ((5, 2, 40), (100, 2, 40), (700, 1, 300), (3000, 1, 4096)):
        p = _problem(R, E, N, K, False, False)
        out, guard = _guarded(R, N)
        _call(p, out)
        assert _intact(guard)
        _check(p, out)


def test_grouped_leaves_rows_behind_the_last_expert():
    _say("mxfp4 grouped rows behind")
    for R, kept in ((300, 171), (40, 0), (9000, 4100)):
        p = _problem(R, 6, 100, 512, False, True, seed=4)
        p["cumsum"] = p["cumsum"].clamp(max=kept)
        out, guard = _guarded(R, 100)
        _call(p, out)
        assert _intact(guard)
        _check(p, out)


def test_grouped_prefix_sums_and_indices_out_of_range():
    """Prefix sums past R or falling ones stay inside the buffers; a source row outside x is a
    row of zeros."""
    _say("mxfp4 grouped out of range")
    p = _problem(96, 5, 70, 320, False, True, seed=8)
    p["row_idx"][[3, 50]] = -1
    p["row_idx"][[7, 90]] = 3 * p["x_rows"] + 5
    out, guard = _guarded(96, 70)
    _call(p, out)
    _check(p, out)
    assert not bool(out[[3, 7, 50, 90]].any())
    p["cumsum"] = torch.tensor([-5, 30, 20, 500, 96], dtype=I32, device="cuda")
    _call(p, out)
    torch.cuda.synchronize()
    assert _intact(guard)


def test_grouped_prefix_sums_that_fall_make_no_more_tiles():
    _say("mxfp4 grouped falling")
    R, E, N, K = 200000, 10240, 64, 64
    p = _problem(R, 4, N, K, False, False, seed=9)
    p["E"] = E
    p["w"], p["ws"] = p["w"][:1].repeat(E, 1, 1), p["ws"][:1].repeat(E, 1, 1)
    p["cumsum"] = torch.tensor([R, 0] * (E // 2), dtype=I32, device="cuda")
    out, guard = _guarded(R, N)
    _call(p, out)
    torch.cuda.synchronize()
    assert _intact(guard)


def test_grouped_default_situ_parameters_and_wide_ones():
    _say("mxfp4 grouped SiTU parameters")
    p = _problem(60, 4, 64, 512, True, False, seed=2)
    out, _ = _guarded(60, 64)
    p["beta"] = p["lam"] = None
    _call(p, out)
    _check(dict(p, beta=torch.full((4,), 4.0), lam=torch.full((4,), 25.0)), out)
    p["beta"], p["lam"] = torch.full((4,), 1e5, device="cuda"), torch.full((4,), 1e6, device="cuda")
    _call(p, out)
    _check(p, out)


@pytest.mark.parametrize("rows,N", [(20, 80), (600, 80), (3000, 1024)])
def test_grouped_bad_scales_stay_in_their_row_and_column(rows, N):
    _say(f"mxfp4 grouped NaN rows={rows} N={N}")
    p = _problem(rows, 1, N, 1024, False, False, seed=6)
    out, _ = _guarded(rows, N)
    _call(p, out)
    clean = out.clone()
    p["xs"][11, 17] = 255
    p["ws"][0, 33, 31] = 255
    p["x"][11, 17 * 16:18 * 16] = 0                    # NaN times codes of 0
    _call(p, out)
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[11], nan[:, 33] = True, True
    assert torch.equal(out.isnan(), nan)
    assert torch.equal(out[~nan], clean[~nan])


def test_grouped_sums_keep_small_blocks_beside_large_ones():
    """Blocks of 2^20 that cancel leave the sum of the blocks of 1: scales and sums hold 24 bits."""
    _say("mxfp4 grouped precision")
    R, N, K = 40, 48, 128
    code = torch.full((R, K // 2), 0x22, dtype=U8, device="cuda")          # all ones
    xs = torch.full((R, 4), 127, dtype=U8, device="cuda")
    xs[:, 0] = xs[:, 2] = 127 + 16
    w, ws = torch.full((N, K // 2), 0x22, dtype=U8, device="cuda"), torch.full((N, 4), 127, dtype=U8, device="cuda")
    w[:, 32:48] = 0xAA                                                      # block 2: minus one
    out = torch.empty((R, N), dtype=BF16, device="cuda")
    cum = torch.tensor([R], dtype=I32, device="cuda")
    rm.moe_grouped_gemm_mxfp4(R, N, K, 1, code, xs, cum, w, ws, out)
    assert bool((out == 64).all())


@pytest.mark.parametrize("sx,sw", [(0, 254), (254, 0), (60, 70), (10, 120), (127, 250), (200, 40)])
def test_grouped_scales_of_the_whole_range(sx, sw):
    _say(f"mxfp4 grouped scales {sx} {sw}")
    p = _problem(33, 1, 40, 96, False, False, seed=5)
    p["xs"].fill_(sx)
    p["ws"].fill_(sw)
    out, _ = _guarded(33, 40)
    _call(p, out)
    want, tol, _ = _want(p)
    # The bound holds for sums in fp32's range: any partial sum is at most the magnitudes' sum, so
    # where that stays below the largest BF16 no partial sum is infinite (96 products of up to 36
    # at 2^123 pass it: 2^123 * 2^11.7, and then two blocks may be infinite before a third
    # brings the sum back).
    mag = ref.ref.product(ref.decode(p["x"], p["xs"]), ref.decode(p["w"][0], p["ws"][0]))[1]
    inside = mag < 3.38e38
    assert sx + sw > 360 or bool(inside.all())
    assert bool(((out.double() - want).abs() <= tol + 2.0 ** -133)[inside].all())
    assert not bool(out[inside].isnan().any())
    assert not bool(out[want.abs() > 3.41e38].isfinite().any())


def test_grouped_weights_and_outputs_past_32_bit_offsets():
    _say("mxfp4 grouped large")
    E, N, K = 1200, 1000, 8192                         # 4.9e9 bytes of codes
    g = _gen(1)
    w, ws = torch.zeros((E, N, K // 2), dtype=U8, device="cuda"), torch.zeros((E, N, K // 32), dtype=U8, device="cuda")
    p = _problem(35, 1, N, K, False, False)
    w[E - 1], ws[E - 1] = p["w"][0], p["ws"][0]
    p.update(E=E, w=w, ws=ws, cumsum=torch.tensor([5] * (E - 1) + [35], dtype=I32, device="cuda"))
    out, guard = _guarded(35, N)
    _call(p, out)
    assert _intact(guard)
    _check(p, out)
    assert not bool(out[:5].any())
    del w, ws, p
    R, N, K = 300000, 8192, 64                         # 2.5e9 outputs
    x, xs = _random_rows(g, R, K, -2)
    w, ws = _random_rows(g, 2 * N, K, -2)
    out = torch.empty((R, N), dtype=BF16, device="cuda")
    cum = torch.tensor([R - 150, R], dtype=I32, device="cuda")
    rm.moe_grouped_gemm_mxfp4(R, N, K, 2, x, xs, cum, w.view(2, N, -1), ws.view(2, N, -1), out)
    for rows, e in ((slice(R - 300, R - 150), 0), (slice(R - 150, R), 1)):
        want, mag = ref.ref.product(ref.decode(x[rows], xs[rows]),
                                    ref.decode(w[e * N:(e + 1) * N], ws[e * N:(e + 1) * N]))
        tol = ref.BF16_HALF_STEP * 1.001 * want.abs() + 6 * 2.0 ** -23 * mag
        assert bool(((out[rows].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("R,N,situ", [(5, 100, False), (40, 700, True), (300, 9000, False),
                                      (2100, 1500, True), (4096, 3600, False), (4200, 1900, True)])
def test_grouped_token_rows_past_32_bit_offsets(R, N, situ):
    """Gathered rows of more than 4 GB of codes, on every tile size; some of them missing."""
    _say(f"mxfp4 grouped wide rows R={R} N={N} situ={situ}")
    K, x_rows = 16384, 530000                          # 4.3e9 bytes of codes
    g = _gen(R)
    x = torch.zeros((x_rows, K // 2), dtype=U8, device="cuda")
    xs = torch.zeros((x_rows, K // 32), dtype=U8, device="cuda")
    idx = torch.randint(0, x_rows, (R,), generator=g, device="cuda")
    idx[-1], idx[R // 2] = x_rows - 1, x_rows - 2
    p = _problem(R, 1, N, K, situ, False)
    x[idx], xs[idx] = p["x"], p["xs"]
    sub = dict(p, x=x[idx], xs=xs[idx])               # (where two rows share a source: what it holds)
    gone = torch.zeros(R, dtype=torch.bool, device="cuda")
    gone[1] = True
    sub["row_idx"] = torch.where(gone, -1, torch.arange(R, device="cuda")).to(I32)
    out, guard = _guarded(R, N)
    idx = torch.where(gone, -1, idx).to(I32)
    _call(dict(p, x=x, xs=xs, x_rows=x_rows, row_idx=idx), out)
    torch.cuda.synchronize()
    assert _intact(guard) and not bool(out[1].any())
    _check(sub, out)


@pytest.mark.parametrize("R", [3, 200])
def test_grouped_weights_of_one_expert_past_32_bit_offsets(R):
    _say(f"mxfp4 grouped wide weights R={R}")
    N, K = 65536, 65536                                # 4.3e9 bytes of codes with SiTU
    g = _gen(R)
    x, xs = _random_rows(g, R, K, -6)
    w, ws = torch.zeros((2 * N, K // 2), dtype=U8, device="cuda"), torch.full((2 * N, K // 32), 127, dtype=U8, device="cuda")
    cols = torch.tensor([0, 1, 777, N - 2, N - 1], device="cuda")
    rows = torch.cat((cols, cols + N))
    w[rows], ws[rows] = _random_rows(g, rows.numel(), K, -6)
    out, guard = _guarded(R, N)
    cum = torch.tensor([R], dtype=I32, device="cuda")
    beta, lam = torch.full((1,), 4.0), torch.full((1,), 25.0)
    rm.moe_grouped_gemm_mxfp4(R, N, K, 1, x, xs, cum, w, ws, out, situ=True)
    torch.cuda.synchronize()
    assert _intact(guard)
    want, tol, _ = ref.grouped(ref.decode(x, xs), torch.arange(R, device="cuda"), cum,
                               lambda e: ref.decode(w[rows], ws[rows]), cols.numel(), beta, lam, True)
    assert bool(((out[:, cols].double() - want).abs() <= tol).all())
    others = torch.ones(N, dtype=torch.bool, device="cuda")
    others[cols] = False
    assert not bool(out[:, others].any())


# one problem for each tile size and ring that the launch rule chooses between
KERNELS = [(40, 1, 1100, 4128), (40, 4, 300, 544), (600, 1, 5000, 544), (9000, 16, 3000, 288),
           (20000, 3, 2000, 800), (20000, 3, 2000, 2080), (1, 1, 900, 2048), (3000, 600, 512, 384)]


@pytest.mark.parametrize("situ", [False, True])
@pytest.mark.parametrize("R,E,N,K", KERNELS)
def test_grouped_in_a_graph_repeats_bit_for_bit(R, E, N, K, situ):
    _say(f"mxfp4 grouped graph R={R} E={E} N={N} K={K} situ={situ}")
    p = _problem(R, E, N, K, situ, True, "zipf", seed=12)
    out, guard = _guarded(R, N)
    _call(p, out)
    _check(p, out)
    want = out.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        _call(p, out, stream=side)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.zero_()
        _call(p, out)
        assert torch.equal(out, want)
    assert _intact(guard)


@pytest.mark.parametrize("R,E,N,K", KERNELS)
def test_grouped_zero_rows_with_the_activation(R, E, N, K):
    _say(f"mxfp4 grouped missing sources R={R}")
    p = _problem(R, E, N, K, True, True, seed=13)
    gone = sorted({0, R // 2, R - 1})
    p["row_idx"][gone] = torch.tensor([-1, 3 * p["x_rows"], 2 ** 31 - 1], dtype=I32,
                                      device="cuda")[:len(gone)]
    p["xs"][0] = 255                                   # NaN in the row that stands in
    out, guard = _guarded(R, N)
    _call(p, out)
    torch.cuda.synchronize()
    assert _intact(guard) and not bool(out[gone].any())


def test_a_rows_result_does_not_depend_on_the_others_positions():
    """The same rows under one expert, in other places of a tile: the same sums."""
    _say("mxfp4 grouped order")
    p = _problem(300, 1, 520, 1056, False, False, seed=3)
    out, _ = _guarded(300, 520)
    _call(p, out)
    order = torch.randperm(300, generator=_gen(1), device="cuda")
    q = dict(p, x=p["x"][order].contiguous(), xs=p["xs"][order].contiguous())
    again, _ = _guarded(300, 520)
    _call(q, again)
    assert torch.equal(again, out[order])


# ---------------------------------------------------------------------------------------
# The layer in 4 bits.
# ---------------------------------------------------------------------------------------
def _layer(T, H, I, E, k, seed=0):
    """Inputs and buffers of one expert layer on MXFP4 weights and rows, and its stages."""
    g = _gen(seed + T)
    R, d = T * k, rm.MoeDims(H, I, E, k)
    e = lambda *shape, dtype=BF16: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    s = {"x": _normal(g, T, H), "res": _normal(g, T, H), "gate": _normal(g, E, H, std=0.05),
         "nw": (1 + 0.1 * _normal(g, H, dtype=F32)).to(BF16)}
    for name, Nw, K in (("w13", 2 * I, H), ("w2", H, I)):
        s[name], s[name + "s"] = e(E, Nw, K // 2, dtype=U8), e(E, Nw, ref.stride(K), dtype=U8)
        rm.moe_quantize_mxfp4(_normal(g, E * Nw, K, std=0.05), E * Nw, K, s[name], s[name + "s"])
    s["gq"] = (448.0 * 6.0 / s["gate"].float().abs().amax()).reshape(1)
    s["galpha"] = 1.0 / s["gq"]
    s["gcodes"], s["gscales"] = e(E, H // 2, dtype=U8), e(E, H // 16, dtype=U8)
    rm.moe_quantize_nvfp4(s["gate"], 1, E, H, s["gq"], s["gcodes"], s["gscales"])
    s.update(res_out=e(T, H), y=e(T, H), logits=e(T, E, dtype=F32), ids=e(T, k, dtype=I32),
             rw=e(T, k), srow=e(R, dtype=I32), map=e(R, dtype=I32), cum=e(E, dtype=I32), ex=e(R, H),
             yc=e(T, H // 2, dtype=U8), ys=e(T, ref.stride(H), dtype=U8), act=e(R, I),
             ac=e(R, I // 2, dtype=U8), acs=e(R, ref.stride(I), dtype=U8), rows=e(R, H), out=e(T, H),
             counts=e(E, dtype=I32), sums=e(E, dtype=F32), tokens=e(1, dtype=I32),
             loss=e(1, dtype=F32), grad=e(T, E, dtype=F32),
             ws=e(rm.moe_workspace_size(d, T, rm.MOE_QUANT_NONE), dtype=U8),
             bws=e(rm.moe_balance_workspace_size(T, E), dtype=U8))

    def run(stream=None):
        kw = {"stream": stream}
        rm.moe_rmsnorm(T, H, s["x"], s["res"], s["nw"], 1e-6, rm.MOE_QUANT_NONE, s["res_out"],
                       s["y"], None, None, **kw)
        rm.moe_matvec_nvfp4(T, E, H, s["y"], s["gcodes"], s["gscales"], s["galpha"], s["logits"],
                            out_f32=True, **kw)
        rm.moe_topk_softmax(T, E, k, s["logits"], s["ids"], s["rw"], **kw)
        rm.moe_balance_loss(T, E, k, s["logits"], s["ids"], 0.01, s["counts"], s["sums"],
                            s["tokens"], s["loss"], s["bws"], **kw)
        rm.moe_balance_loss_grad(T, E, s["logits"], s["counts"], s["tokens"], 0.01, s["grad"], **kw)
        rm.moe_route(d, T, s["y"], s["ids"], rm.MOE_QUANT_NONE, None, None, s["srow"], s["map"],
                     s["cum"], s["ex"], None, s["ws"], **kw)
        rm.moe_quantize_mxfp4(s["y"], T, H, s["yc"], s["ys"], **kw)
        rm.moe_grouped_gemm_mxfp4(R, I, H, E, s["yc"], s["ys"], s["cum"], s["w13"], s["w13s"],
                                  s["act"], x_rows=T, row_idx=s["srow"], row_div=k, situ=True, **kw)
        rm.moe_quantize_mxfp4(s["act"], R, I, s["ac"], s["acs"], **kw)
        rm.moe_grouped_gemm_mxfp4(R, H, I, E, s["ac"], s["acs"], s["cum"], s["w2"], s["w2s"],
                                  s["rows"], **kw)
        rm.moe_combine(T, H, k, R, s["rows"], s["map"], s["rw"], s["res_out"], s["out"], **kw)

    return s, run


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 64, 16, 4), (33, 512, 192, 24, 3),
                                       (64, 384, 96, 8, 2), (20, 2912, 160, 40, 8)])
def test_the_layer_in_four_bits(T, H, I, E, k):
    """Every stage against its definition on what the stage before it left."""
    _say(f"mxfp4 layer T={T} H={H} I={I} E={E} k={k}")
    s, run = _layer(T, H, I, E, k)
    run()
    torch.cuda.synchronize()
    # the counts are the routing's
    cum = s["cum"].long()
    assert torch.equal(s["counts"].long(), cum - torch.cat((cum.new_zeros(1), cum[:-1])))
    counts, sums, tol, tokens, loss, ltol = ref.balance(s["logits"], s["ids"], None, 0.01)
    assert int(s["tokens"]) == tokens == T and torch.equal(s["counts"].long(), counts)
    assert bool(((s["sums"].double() - sums).abs() <= tol).all())
    assert abs(float(s["loss"]) - loss) <= ltol
    grad, gtol = ref.balance_grad(s["logits"], None, counts, tokens, 0.01, 1.0, None)
    assert bool(((s["grad"].double() - grad).abs() <= gtol + ref.F32_HALF_STEP * grad.abs()).all())
    for rows, codes, scales in ((s["y"], s["yc"], s["ys"]), (s["act"], s["ac"], s["acs"])):
        want = ref.quantize(rows)
        assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    four, wide = torch.full((E,), 4.0), torch.full((E,), 25.0)
    want, tol, _ = ref.grouped(ref.decode(s["yc"], s["ys"]), s["srow"].long() // k, s["cum"],
                               lambda e: ref.decode(s["w13"][e], s["w13s"][e]), I, four, wide, True)
    assert bool(((s["act"].double() - want).abs() <= tol).all())
    want, tol, _ = ref.grouped(ref.decode(s["ac"], s["acs"]), torch.arange(T * k, device="cuda"),
                               s["cum"], lambda e: ref.decode(s["w2"][e], s["w2s"][e]), H)
    assert bool(((s["rows"].double() - want).abs() <= tol).all())
    want, tol = ref.ref.combine(s["rows"], s["map"], s["rw"], s["res_out"])
    assert bool(((s["out"].double() - want).abs() <= tol).all())


def test_the_layer_in_a_graph_and_beside_eager_work():
    _say("mxfp4 layer graph")
    T, H, I, E, k = 24, 512, 128, 32, 4
    s, run = _layer(T, H, I, E, k, seed=3)
    run()
    torch.cuda.synchronize()
    names = ("yc", "ys", "act", "ac", "acs", "rows", "out", "counts", "sums", "tokens", "loss", "grad")
    keep = {n: s[n].clone() for n in names}
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(stream=side)
    for _ in range(4):
        for n in keep:
            s[n].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, v in keep.items():
            assert torch.equal(s[n].view(U8), v.view(U8)), n
        run()
        torch.cuda.synchronize()
    s["x"].copy_(_normal(_gen(77), T, H))
    graph.replay()
    torch.cuda.synchronize()
    replayed = {n: s[n].clone() for n in names}
    run()
    torch.cuda.synchronize()
    for n, v in replayed.items():
        assert torch.equal(s[n].view(U8), v.view(U8)), n
    assert not torch.equal(replayed["out"], keep["out"])


def test_two_streams_at_once_give_the_same_results():
    _say("mxfp4 layer two streams")
    a, run_a = _layer(40, 512, 128, 32, 4, seed=5)
    b, run_b = _layer(17, 768, 64, 16, 2, seed=6)
    run_a()
    run_b()
    torch.cuda.synchronize()
    names = ("out", "loss", "grad")
    want = [{n: s[n].clone() for n in names} for s in (a, b)]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for s in (a, b):
            for n in names:
                s[n].zero_()
        torch.cuda.synchronize()
        run_a(stream=sa)
        run_b(stream=sb)
        torch.cuda.synchronize()
        for s, w in zip((a, b), want):
            for n in names:
                assert torch.equal(s[n], w[n]), n


def test_binding_refuses_wrong_tensors():
    _say("mxfp4 binding refusals")
    x = torch.zeros((4, 64), dtype=BF16, device="cuda")
    codes, scales = torch.zeros((4, 32), dtype=U8, device="cuda"), torch.zeros((4, 4), dtype=U8, device="cuda")
    with pytest.raises(ValueError, match="src is not contiguous"):
        rm.moe_quantize_mxfp4(x.view(8, 32).t(), 8, 32, codes, scales)
    with pytest.raises(ValueError, match="scales holds 8 elements, not 16"):
        rm.moe_quantize_mxfp4(x, 4, 64, codes, scales[:2])
    with pytest.raises(ValueError, match="codes holds"):
        rm.moe_dequantize_mxfp4(codes[:3], scales, 4, 64, x)
