"""GPU checks of the expert-stage operators (moe_rmsnorm, moe_matvec_nvfp4, moe_grouped_gemm,
moe_combine) against their definitions in 64 bits (tests/expert_ops.py), within the bounds
derived there."""

import sys

import pytest
import torch

import routed_moe_layer_amd as rm
from tests import expert_ops as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
QUANT = {"none": rm.MOE_QUANT_NONE, "bf16": rm.MOE_QUANT_NONE,
         "int8": rm.MOE_QUANT_INT8_ROW_DYNAMIC, "e4m3": rm.MOE_QUANT_E4M3_ROW_DYNAMIC}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    yield
    torch.cuda.synchronize()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _guarded(*shape, dtype=BF16):
    """A buffer of the shape with 512 elements behind it that no call may write."""
    n = 1
    for s in shape:
        n *= s
    full = torch.zeros(n + 512, dtype=torch.int32 if dtype == F32 else torch.int16 if dtype == BF16
                       else torch.uint8, device="cuda")
    full.fill_(0x55)
    t = full[:n].view(dtype).view(shape)
    return t, full[n:]


def _intact(guard):
    return bool((guard == 0x55).all())


# ---------------------------------------------------------------------------------------
# moe_rmsnorm
# ---------------------------------------------------------------------------------------
def _norm_check(T, H, q, residual, with_y, x=None, eps=1e-6, seed=0):
    g = _gen(seed + 31 * T + H)
    x = _normal(g, T, H) if x is None else x
    res = _normal(g, T, H, std=2.0) if residual else None
    w = (1 + 0.1 * _normal(g, H, dtype=F32)).to(BF16)
    h, y = ref.rmsnorm(x, res, w, eps)
    rel = ref.norm_rel(H)
    res_out, guard_r = _guarded(T, H)
    out, guard_y = _guarded(T, H)
    codes, guard_c = _guarded(T, H, dtype=torch.uint8)
    scales, guard_s = _guarded(T, dtype=F32)
    quant = q != "none"
    rm.moe_rmsnorm(T, H, x, res, w, eps, QUANT[q], res_out if residual else None,
                   out if with_y else None, codes if quant else None, scales if quant else None)
    torch.cuda.synchronize()
    assert all(map(_intact, (guard_r, guard_y, guard_c, guard_s)))
    if residual:
        assert bool(((res_out.double() - h).abs() <= ref.BF16_HALF_STEP * 1.001 * h.abs()).all())
    if with_y:
        assert bool(((out.double() - y).abs() <= (ref.BF16_HALF_STEP + 2 * rel) * y.abs() + 1e-38).all())
    if quant:
        top = ref.CODE_MAX[q]
        want = y.abs().amax(1) / top
        assert bool(((scales.double() - want).abs() <= 2 * rel * want).all())
        v = torch.where(want[:, None] == 0, 0.0, y / want.clamp(min=1e-300)[:, None])
        got = codes.view(CODE[q]).double()
        slack = top * 4 * rel + top * 3 * ref.F32_HALF_STEP      # y, scale and quotient
        if q == "int8":
            assert bool(((got - v).abs() <= 0.5 + slack).all())
            nearest = torch.round(v)
        else:
            near = ref.e4m3_nearest(v)
            assert bool(((got - v).abs() <= (near - v).abs() + 2 * slack).all())
            nearest = near
        # next to a border between two codes the kernel may take either one; only there
        differ = got != nearest
        assert float(differ.double().mean()) <= 0.01 or T * H < 1000
    return res_out, out, codes, scales


@pytest.mark.parametrize("q,residual,with_y", [("none", True, True), ("none", False, True),
                                               ("int8", True, False), ("int8", False, True),
                                               ("e4m3", True, True), ("e4m3", False, False)])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 72), (1, 3584), (130, 512), (37, 520), (300, 3584),
                                 (5, 7168), (2, 8200), (9, 16384), (2, 65536)])
def test_rmsnorm(T, H, q, residual, with_y):
    _say(f"rmsnorm T={T} H={H} {q} residual={residual} y={with_y}")
    _norm_check(T, H, q, residual, with_y)


def test_rmsnorm_many_rows():
    _say("rmsnorm 5000 x 1024")
    _norm_check(5000, 1024, "int8", True, True)


def test_rmsnorm_zero_rows_and_outliers():
    _say("rmsnorm zero rows")
    x = _normal(_gen(5), 6, 256)
    x[1] = 0
    x[4] = 0
    x[2, 7] = 3e4
    for q in ("int8", "e4m3"):
        _, y, codes, scales = _norm_check(6, 256, q, False, True, x=x, eps=0.5)
        assert float(scales[1]) == 0 and float(scales[4]) == 0
        assert not bool(codes[1].any()) and not bool(y[4].any())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rmsnorm_a_bad_row_is_marked_and_leaves_the_others(bad):
    _say(f"rmsnorm {bad}")
    g = _gen(6)
    x, w = _normal(g, 9, 1000), torch.ones(1000, dtype=BF16, device="cuda")
    want = [torch.empty((9, 1000), dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda")]
    rm.moe_rmsnorm(9, 1000, x, None, w, 1e-6, QUANT["int8"], None, None, *want)
    y, got = x.clone(), [torch.empty_like(t) for t in want]
    x[4, 333] = bad
    rm.moe_rmsnorm(9, 1000, x, None, w, 1e-6, QUANT["int8"], None, y, *got)
    others = [i for i in range(9) if i != 4]
    assert torch.equal(got[0][others], want[0][others]) and torch.equal(got[1][others], want[1][others])
    assert bool(got[1][4].isnan()) and bool(y[4, 333].isnan()) and not bool(y[others].isnan().any())


def test_rmsnorm_in_place():
    _say("rmsnorm in place")
    g = _gen(7)
    for T, H in ((3, 3584), (700, 256), (2, 20000)):
        x, r, w = _normal(g, T, H), _normal(g, T, H), _normal(g, H)
        y, ro = torch.empty_like(x), torch.empty_like(x)
        rm.moe_rmsnorm(T, H, x, r, w, 1e-5, 0, ro, y, None, None)
        rm.moe_rmsnorm(T, H, x, r, w, 1e-5, 0, r, x, None, None)
        assert torch.equal(x, y) and torch.equal(r, ro)


# ---------------------------------------------------------------------------------------
# moe_matvec_nvfp4
# ---------------------------------------------------------------------------------------
def _matvec_check(T, N, K, f32, seed=0):
    g = _gen(seed + T + 7 * N + K)
    x = _normal(g, T, K)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(0, 0x7F, (N, K // 16), generator=g, device="cuda", dtype=torch.uint8)
    alpha = torch.tensor([0.0173], device="cuda")
    y, guard = _guarded(T, N, dtype=F32 if f32 else BF16)
    rm.moe_matvec_nvfp4(T, N, K, x, codes, scales, alpha, y, out_f32=f32)
    torch.cuda.synchronize()
    assert _intact(guard)
    want, mag = ref.product(x, ref.nvfp4_weights(codes, scales))
    want, mag = want * alpha.double(), mag * alpha.double()
    tol = (32 + K / 8) * ref.F32_HALF_STEP * mag + (0 if f32 else ref.BF16_HALF_STEP * 1.001) * want.abs()
    assert bool(((y.double() - want).abs() <= tol).all())
    return x, codes, scales, alpha, y


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 896, 3584), (1, 17, 48), (2, 300, 1040),
                                   (3, 64, 2064), (4, 5, 4096), (5, 129, 272), (8, 100, 512),
                                   (16, 333, 3600), (17, 31, 1024), (33, 48, 656), (64, 257, 1008),
                                   (1, 2051, 65536), (2, 77, 32768), (2, 2100, 512),
                                   (64, 40, 16384), (12, 14500, 160), (40, 7300, 208)])
def test_matvec_nvfp4(T, N, K, f32):
    _say(f"matvec T={T} N={N} K={K} f32={f32}")
    _matvec_check(T, N, K, f32)


def test_matvec_takes_the_librarys_quantized_weights():
    _say("matvec with moe_quantize_nvfp4")
    g = _gen(9)
    N, K, T = 200, 768, 3
    w, x = _normal(g, N, K, std=0.02), _normal(g, T, K)
    q = (448.0 * 6.0 / w.float().abs().amax()).reshape(1)
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((N, K // 16), dtype=torch.uint8, device="cuda")
    rm.moe_quantize_nvfp4(w, 1, N, K, q, codes, scales)
    y = torch.empty((T, N), device="cuda")
    rm.moe_matvec_nvfp4(T, N, K, x, codes, scales, 1.0 / q, y, out_f32=True)
    want, mag = ref.product(x, ref.nvfp4_weights(codes, scales) / q.double())
    assert bool(((y.double() - want).abs() <= (34 + K / 8) * ref.F32_HALF_STEP * mag).all())
    # and it is the projection: each weight is off by at most 1/4 of its block's maximum
    full, _ = ref.product(x, w)
    assert float((want - full).norm() / full.norm()) < 0.25


@pytest.mark.parametrize("T", [1, 2, 3, 20])
def test_matvec_bad_values_stay_in_their_token(T):
    _say(f"matvec NaN T={T}")
    x, codes, scales, alpha, y = _matvec_check(T, 50, 512, True, seed=3)
    x[T - 1, 100] = float("nan")
    got = torch.empty_like(y)
    rm.moe_matvec_nvfp4(T, 50, 512, x, codes, scales, alpha, got, out_f32=True)
    assert bool(got[T - 1].isnan().all()) and torch.equal(got[:T - 1], y[:T - 1])
    x[T - 1, 100] = float("inf")
    rm.moe_matvec_nvfp4(T, 50, 512, x, codes, scales, alpha, got, out_f32=True)
    assert not bool(got[T - 1].isfinite().any()) and torch.equal(got[:T - 1], y[:T - 1])


# ---------------------------------------------------------------------------------------
# moe_grouped_gemm
# ---------------------------------------------------------------------------------------
def _counts(kind, R, E, g):
    if kind == "one":                                   # every row to one expert
        c = torch.zeros(E, dtype=torch.long)
        c[E // 2] = R
        return c
    p = torch.ones(E) if kind == "uniform" else 1.0 / torch.arange(1, E + 1)
    ids = torch.multinomial(p.cuda(), R, replacement=True, generator=g)
    return torch.bincount(ids, minlength=E).cpu()


def _operand(g, q, *shape, std):
    """(rows, scales or None) of the type."""
    v = _normal(g, *shape, std=std, dtype=F32)
    if q == "bf16":
        return v.to(BF16), None
    scale = v.abs().amax(-1) / ref.CODE_MAX[q]
    u = v / scale[..., None]
    return (u.round() if q == "int8" else u).to(CODE[q]), scale


def _grouped_problem(R, E, N, K, q, situ, gather, kind, seed=0):
    g = _gen(seed + R + 3 * E + 5 * N + 7 * K)
    Nw = 2 * N if situ else N
    k = 3 if gather else 1
    x_rows = (R + k - 1) // k if gather else R
    p = {"R": R, "E": E, "N": N, "K": K, "q": q, "situ": situ, "x_rows": x_rows, "row_div": k}
    p["x"], p["x_scale"] = _operand(g, q, x_rows, K, std=1.0)
    p["w"], p["w_scale"] = _operand(g, q, E, Nw, K, std=0.5)
    p["row_idx"] = (torch.randperm(x_rows * k, generator=g, device="cuda")[:R].to(torch.int32)
                    if gather else None)
    p["cumsum"] = _counts(kind, R, E, g).cumsum(0).to(torch.int32).cuda()
    p["beta"] = torch.empty(E, device="cuda").uniform_(3, 5, generator=g) if situ else None
    p["lam"] = torch.empty(E, device="cuda").uniform_(20, 30, generator=g) if situ else None
    return p


def _call(p, out, **kw):
    rm.moe_grouped_gemm(p["R"], p["N"], p["K"], p["E"], p["x"], p["cumsum"], p["w"], out,
                        quant=QUANT[p["q"]], x_scale=p["x_scale"], w_scale=p["w_scale"],
                        x_rows=p["x_rows"], row_idx=p["row_idx"], row_div=p["row_div"],
                        situ=p["situ"], situ_beta=p["beta"], situ_linear_beta=p["lam"], **kw)


def _want(p):
    if p["row_idx"] is None:
        src = torch.arange(p["R"], device="cuda")
    else:
        src = p["row_idx"].long().div(p["row_div"], rounding_mode="floor")
    src = torch.where((src >= 0) & (src < p["x_rows"]), src, -1)
    return ref.grouped(p["x"], p["x_scale"], src, p["cumsum"], p["w"], p["w_scale"], p["N"],
                       p["beta"], p["lam"], p["situ"])


def _check_grouped(p, out):
    want, tol, written = _want(p)
    bad = (out.double() - want).abs() > tol
    bad |= ~out.isfinite()
    bad[~written] = False
    assert not bool(bad.any()), f"{int(bad.sum())} outputs outside the bound"
    untouched = out.view(torch.int16)[~written]
    assert bool((untouched == 0x55).all()), "a row behind the last expert's was written"


GROUPED = [
    # R, E, N, K (K is divided by 2 for BF16 where it must be), counts
    (1, 1, 1, 16, "uniform"), (1, 5, 33, 64, "uniform"), (7, 3, 17, 48, "uniform"),
    (16, 1, 64, 128, "one"), (40, 16, 96, 400, "uniform"), (64, 4, 130, 1040, "zipf"),
    (65, 2, 64, 256, "one"), (200, 900, 40, 144, "uniform"), (333, 7, 257, 528, "zipf"),
    (1000, 9, 128, 512, "one"), (2500, 20, 384, 1024, "zipf"), (700, 3, 1000, 272, "uniform"),
    (3000, 2, 256, 2048, "uniform"), (129, 1, 36, 3600, "one"), (50, 10240, 16, 32, "uniform"),
    # every tile size, with items enough and too few, ragged N and K and odd chunk counts
    (33, 1, 1100, 2064, "one"), (600, 1, 5000, 272, "one"), (20000, 3, 1031, 400, "zipf"),
    (9000, 16, 3000, 144, "zipf"), (5000, 600, 2051, 144, "zipf"), (70000, 2500, 24, 64, "uniform"),
    (300000, 5000, 40, 32, "zipf"), (60, 10240, 17, 2064, "uniform"), (31000, 65, 96, 48, "uniform"), (1000, 1, 20000, 1040, "one"),
]


@pytest.mark.parametrize("q", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("situ,gather", [(False, False), (True, True), (False, True)])
@pytest.mark.parametrize("R,E,N,K,kind", GROUPED)
def test_grouped_gemm(R, E, N, K, kind, situ, gather, q):
    _say(f"grouped R={R} E={E} N={N} K={K} {kind} {q} situ={situ} gather={gather}")
    p = _grouped_problem(R, E, N, K, q, situ, gather, kind)
    out, guard = _guarded(R, N)
    _call(p, out)
    torch.cuda.synchronize()
    assert _intact(guard)
    _check_grouped(p, out)


@pytest.mark.parametrize("K", [8, 24, 72, 120, 136])
def test_grouped_gemm_bf16_lengths_between_the_8_bit_ones(K):
    _say(f"grouped BF16 K={K}")
    p = _grouped_problem(100, 3, 50, K, "bf16", False, False, "uniform")
    out, guard = _guarded(100, 50)
    _call(p, out)
    assert _intact(guard)
    _check_grouped(p, out)


@pytest.mark.parametrize("q", ["bf16", "int8", "e4m3"])
def test_grouped_gemm_leaves_rows_behind_the_last_expert(q):
    _say(f"grouped rows behind {q}")
    for R, kept in ((300, 171), (40, 0), (9000, 4100)):
        p = _grouped_problem(R, 6, 100, 256, q, False, True, "uniform", seed=4)
        p["cumsum"] = p["cumsum"].clamp(max=kept)
        out, guard = _guarded(R, 100)
        _call(p, out)
        assert _intact(guard)
        _check_grouped(p, out)


@pytest.mark.parametrize("q", ["bf16", "int8", "e4m3"])
def test_grouped_gemm_prefix_sums_and_indices_out_of_range(q):
    """Prefix sums past R or falling ones stay inside the buffers; a source row outside x is a
    row of zeros."""
    _say(f"grouped out of range {q}")
    p = _grouped_problem(96, 5, 70, 160, q, False, True, "uniform", seed=8)
    p["row_idx"][[3, 50]] = -1
    p["row_idx"][[7, 90]] = 3 * p["x_rows"] + 5
    out, guard = _guarded(96, 70)
    _call(p, out)
    _check_grouped(p, out)
    assert not bool(out[[3, 7, 50, 90]].any())
    p["cumsum"] = torch.tensor([-5, 30, 20, 500, 96], dtype=torch.int32, device="cuda")
    _call(p, out)
    torch.cuda.synchronize()
    assert _intact(guard)


def test_grouped_gemm_default_situ_parameters_and_wide_ones():
    _say("grouped SiTU parameters")
    p = _grouped_problem(60, 4, 64, 256, "bf16", True, False, "uniform", seed=2)
    out, _ = _guarded(60, 64)
    p["beta"] = p["lam"] = None
    _call(p, out)
    want = dict(p, beta=torch.full((4,), 4.0), lam=torch.full((4,), 25.0))
    _check_grouped(want, out)
    # nearly linear: tanh(v / beta) * beta with arguments near zero keeps its relative precision
    p["beta"], p["lam"] = torch.full((4,), 1e5, device="cuda"), torch.full((4,), 1e6, device="cuda")
    _call(p, out)
    _check_grouped(p, out)


@pytest.mark.parametrize("rows", [20, 600])
def test_grouped_gemm_bad_values_stay_in_their_row(rows):
    _say(f"grouped NaN rows={rows}")
    p = _grouped_problem(rows, 3, 80, 512, "bf16", False, False, "uniform", seed=6)
    out, _ = _guarded(rows, 80)
    _call(p, out)
    clean = out.clone()
    p["x"][11, 500] = float("nan")
    p["x"][17, 3] = float("inf")
    _call(p, out)
    others = [i for i in range(rows) if i not in (11, 17)]
    assert torch.equal(out[others], clean[others])
    assert bool(out[11].isnan().all()) and not bool(out[17].isfinite().any())


def test_grouped_gemm_weights_past_32_bit_offsets():
    _say("grouped large weights")
    E, N, K = 700, 1000, 4096                        # 2.9e9 bytes of int8 weights
    g = _gen(1)
    w = torch.zeros((E, N, K), dtype=torch.int8, device="cuda")
    w[E - 1] = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.full((E, N), 0.01, device="cuda")
    R = 35
    x = torch.randint(-127, 128, (R, K), generator=g, device="cuda", dtype=torch.int8)
    p = {"R": R, "E": E, "N": N, "K": K, "q": "int8", "situ": False, "x_rows": R, "row_div": 1,
         "x": x, "x_scale": torch.full((R,), 0.02, device="cuda"), "w": w, "w_scale": ws,
         "row_idx": None, "beta": None, "lam": None,
         "cumsum": torch.tensor([5] * (E - 1) + [R], dtype=torch.int32, device="cuda")}
    out, guard = _guarded(R, N)
    _call(p, out)
    assert _intact(guard)
    _check_grouped(p, out)
    assert not bool(out[:5].any())


# one problem for each tile size and ring that the launch rule chooses between
KERNELS = [("int8", 40, 1, 1100, 2064), ("bf16", 40, 4, 300, 272), ("e4m3", 600, 1, 5000, 272),
           ("bf16", 9000, 16, 3000, 144), ("int8", 20000, 3, 2000, 400),
           ("e4m3", 20000, 3, 2000, 1040)]


@pytest.mark.parametrize("q,R,E,N,K", KERNELS)
def test_grouped_gemm_in_a_graph_repeats_bit_for_bit(q, R, E, N, K):
    _say(f"grouped graph {q} R={R} E={E} N={N} K={K}")
    p = _grouped_problem(R, E, N, K, q, False, True, "zipf", seed=12)
    out, guard = _guarded(R, N)
    _call(p, out)
    _check_grouped(p, out)
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


@pytest.mark.parametrize("q,R,E,N,K", KERNELS)
def test_grouped_gemm_zero_rows_with_the_activation(q, R, E, N, K):
    _say(f"grouped missing sources {q} R={R}")
    p = _grouped_problem(R, E, N, K, q, True, True, "uniform", seed=13)
    gone = [0, R // 2, R - 1]
    p["row_idx"][gone] = torch.tensor([-1, 3 * p["x_rows"], 2 ** 31 - 1], dtype=torch.int32,
                                      device="cuda")
    p["x"].view(torch.uint8)[0] = 0x7F                  # NaN (BF16, E4M3) in the row that stands in
    out, guard = _guarded(R, N)
    _call(p, out)
    torch.cuda.synchronize()
    assert _intact(guard) and not bool(out[gone].any())


def test_grouped_gemm_rows_and_outputs_past_32_bit_offsets():
    _say("grouped large rows and outputs")
    R, E, N, K = 300000, 2, 8192, 8192                 # 2.5e9 outputs; x 2.5e9 bytes
    g = _gen(3)
    x = torch.zeros((R, K), dtype=torch.int8, device="cuda")
    last = torch.randint(-127, 128, (300, K), generator=g, device="cuda", dtype=torch.int8)
    x[R - 300:] = last
    w = torch.randint(-127, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    one = torch.full((R,), 0.01, device="cuda")
    cum = torch.tensor([R - 150, R], dtype=torch.int32, device="cuda")
    out = torch.empty((R, N), dtype=BF16, device="cuda")
    rm.moe_grouped_gemm(R, N, K, E, x, cum, w, out, quant=QUANT["int8"], x_scale=one,
                        w_scale=torch.full((E, N), 0.02, device="cuda"))
    assert not bool(out[:R - 300].any())
    for rows, e in ((slice(0, 150), 0), (slice(150, 300), 1)):
        want = ref.product(last[rows], w[e])[0] * (0.01 * 0.02)
        got = out[R - 300:][rows].double()
        assert bool(((got - want).abs() <= (ref.BF16_HALF_STEP + 2.0 ** -20) * want.abs()).all())


# ---------------------------------------------------------------------------------------
# moe_combine
# ---------------------------------------------------------------------------------------
def test_norm_and_combine_past_32_bit_offsets():
    _say("norm and combine large")
    T, H = 600000, 4096                                # 2.5e9 values
    g = _gen(4)
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    x[T - 5:] = _normal(g, 5, H)
    y = torch.empty_like(x)
    codes, scales = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    w = torch.ones(H, dtype=BF16, device="cuda")
    rm.moe_rmsnorm(T, H, x, None, w, 1e-6, QUANT["int8"], None, y, codes, scales)
    want = ref.rmsnorm(x[T - 5:], None, w, 1e-6)[1]
    assert bool(((y[T - 5:].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -16) * want.abs()).all())
    assert not bool(y[:T - 5].any()) and bool((codes[T - 5:].abs().amax(1) == 127).all())
    idx = torch.tensor([T - 1, -1, T - 3, 0], dtype=torch.int32, device="cuda")
    rw = torch.tensor([[0.5, 0.25], [1.0, 2.0]], dtype=BF16, device="cuda")
    out = torch.empty((2, H), dtype=BF16, device="cuda")
    rm.moe_combine(2, H, 2, T, x, idx, rw, None, out)
    want, tol = ref.combine(x, idx, rw, None)
    assert bool(((out.double() - want).abs() <= tol).all()) and bool(out.any(1).all())


def _combine_problem(T, k, H, R, drop, seed=0):
    g = _gen(seed + T + 3 * k + H)
    rows = _normal(g, R, H)
    idx = torch.randint(0, R, (T * k,), generator=g, device="cuda").to(torch.int32)
    if drop:
        u = torch.empty(T * k, device="cuda").uniform_(0, 1, generator=g)
        idx = torch.where(u < 0.3, -1, idx)
        idx = torch.where(u > 0.9, R, idx)
        idx[:k] = -1                                    # a token with no row at all
    w = torch.empty((T, k), device="cuda").normal_(generator=g).softmax(1).to(BF16)
    return rows, idx.to(torch.int32), w, _normal(g, T, H)


@pytest.mark.parametrize("with_add", [False, True])
@pytest.mark.parametrize("T,k,H,R,drop", [
    (1, 1, 8, 1, False), (1, 16, 3584, 16, False), (5, 3, 72, 9, True), (16, 16, 3584, 256, False),
    (300, 7, 520, 2000, True), (2, 64, 4096, 100, True), (3, 9, 65536, 30, False),
    (2000, 2, 128, 4000, True)])
def test_combine(T, k, H, R, drop, with_add):
    _say(f"combine T={T} k={k} H={H} R={R} drop={drop} add={with_add}")
    rows, idx, w, add = _combine_problem(T, k, H, R, drop)
    add = add if with_add else None
    out, guard = _guarded(T, H)
    rm.moe_combine(T, H, k, R, rows, idx, w, add, out)
    torch.cuda.synchronize()
    assert _intact(guard)
    want, tol = ref.combine(rows, idx, w, add)
    assert bool(((out.double() - want).abs() <= tol).all())
    if drop and add is None:
        assert not bool(out[0].any())
    if with_add:
        rm.moe_combine(T, H, k, R, rows, idx, w, add, add)
        assert torch.equal(add, out)


def test_combine_ignores_dropped_rows_contents():
    _say("combine NaN")
    rows, idx, w, _ = _combine_problem(20, 4, 256, 90, False, seed=5)
    idx[idx == 7] = 8
    rows[7] = float("nan")
    out = torch.empty((20, 256), dtype=BF16, device="cuda")
    rm.moe_combine(20, 256, 4, 90, rows, idx, w, None, out)
    assert not bool(out.isnan().any())


# ---------------------------------------------------------------------------------------
# Streams, graphs, and the stages together.
# ---------------------------------------------------------------------------------------
def _layer(T, H, I, E, k, q, seed=0):
    """Inputs and buffers of one expert layer and a function that runs its stages."""
    g = _gen(seed + T)
    R = T * k
    s = {"x": _normal(g, T, H), "res": _normal(g, T, H),
         "nw": (1 + 0.1 * _normal(g, H, dtype=F32)).to(BF16)}
    s["w13"], s["w13s"] = _operand(g, q, E, 2 * I, H, std=0.05)
    s["w2"], s["w2s"] = _operand(g, q, E, H, I, std=0.05)
    gate = _normal(g, E, H, std=0.05)
    s["gq"] = (448.0 * 6.0 / gate.float().abs().amax()).reshape(1)
    s["galpha"] = 1.0 / s["gq"]
    s["gcodes"] = torch.empty((E, H // 2), dtype=torch.uint8, device="cuda")
    s["gscales"] = torch.empty((E, H // 16), dtype=torch.uint8, device="cuda")
    rm.moe_quantize_nvfp4(gate, 1, E, H, s["gq"], s["gcodes"], s["gscales"])
    e = lambda *shape, dtype=BF16: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    i32 = lambda n: e(n, dtype=torch.int32)  # noqa: E731
    d = rm.MoeDims(H, I, E, k)
    s.update(res_out=e(T, H), y=e(T, H), xc=e(T, H, dtype=torch.uint8), xs=e(T, dtype=F32),
             logits=e(T, E, dtype=F32), ids=i32(T * k), rw=e(T, k), sid=i32(R), srow=i32(R),
             map=i32(R), cum=i32(E), ex=e(R, H), act=e(R, I), ac=e(R, I, dtype=torch.uint8),
             acs=e(R, dtype=F32), amap=i32(R), acum=i32(E), rows=e(R, H), out=e(T, H),
             ws=e(max(rm.moe_workspace_size(d, T, rm.MOE_QUANT_NONE),
                      rm.moe_route_workspace_size(R, 1, E)), dtype=torch.uint8))

    def run(stream=None):
        kw = {"stream": stream}
        Q = QUANT[q]
        rm.moe_rmsnorm(T, H, s["x"], s["res"], s["nw"], 1e-6, Q, s["res_out"], s["y"],
                       s["xc"] if Q else None, s["xs"] if Q else None, **kw)
        rm.moe_matvec_nvfp4(T, E, H, s["y"], s["gcodes"], s["gscales"], s["galpha"], s["logits"],
                            out_f32=True, **kw)
        rm.moe_topk_softmax(T, E, k, s["logits"], s["ids"], s["rw"], **kw)
        rm.moe_route(d, T, s["y"], s["ids"], rm.MOE_QUANT_NONE, None, s["sid"], s["srow"], s["map"],
                     s["cum"], s["ex"], None, s["ws"], **kw)
        x, xs = (s["xc"].view(CODE[q]), s["xs"]) if Q else (s["y"], None)
        rm.moe_grouped_gemm(R, I, H, E, x, s["cum"], s["w13"], s["act"], quant=Q, x_scale=xs,
                            w_scale=s["w13s"], x_rows=T, row_idx=s["srow"], row_div=k, situ=True, **kw)
        a, acs = s["act"], None
        if q == "int8":
            # the activation in int8: routing rows that are in expert order already moves
            # nothing and quantizes each row
            rm.moe_route_v2(R, I, E, 1, s["act"], s["sid"], rm.MoeRouteOptions(quant_mode=1),
                            s["ac"], s["amap"], s["acum"], s["acs"], workspace=s["ws"], **kw)
            a, acs = s["ac"].view(torch.int8), s["acs"]
        if q == "e4m3":
            w2, w2s, Q2 = s["w2b"], None, 0
        else:
            w2, w2s, Q2 = s["w2"], s["w2s"], Q
        rm.moe_grouped_gemm(R, H, I, E, a, s["cum"], w2, s["rows"], quant=Q2, x_scale=acs,
                            w_scale=w2s, **kw)
        rm.moe_combine(T, H, k, R, s["rows"], s["map"], s["rw"], s["res_out"], s["out"], **kw)

    if q == "e4m3":                                    # mixed: FC2 in BF16
        s["w2b"] = (s["w2"].float() * s["w2s"][:, :, None]).to(BF16)
    return s, run


def _layer_reference(s, T, H, I, E, k, q):
    """The layer in 64 bits on the expert ids that were picked, with the type's weights but
    nothing else quantized."""
    h, y = ref.rmsnorm(s["x"], s["res"], s["nw"], 1e-6)
    w13, w2 = s["w13"].double(), s["w2"].double()
    if q != "bf16":
        w13, w2 = w13 * s["w13s"].double()[:, :, None], w2 * s["w2s"].double()[:, :, None]
    ids = s["ids"].long().view(T, k)
    logits = ref.product(y, ref.nvfp4_weights(s["gcodes"], s["gscales"]) * s["galpha"].double())[0]
    rw = torch.gather(logits, 1, ids).softmax(1)
    out = h.clone()
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            gu = w13[e] @ y[t]
            a, c = ref.situ_parts(gu[:I], gu[I:], 4.0, 25.0)
            out[t] += rw[t, j] * (w2[e] @ (a * c))
    return h, logits, out


@pytest.mark.parametrize("q,T,H,I,E,k", [("bf16", 1, 256, 64, 16, 4), ("bf16", 33, 512, 192, 24, 3),
                                         ("int8", 7, 256, 64, 16, 4), ("int8", 64, 384, 128, 8, 2),
                                         ("e4m3", 20, 512, 64, 40, 8)])
def test_the_stages_together(q, T, H, I, E, k):
    _say(f"layer {q} T={T} H={H} I={I} E={E} k={k}")
    s, run = _layer(T, H, I, E, k, q)
    run()
    torch.cuda.synchronize()
    h, logits, want = _layer_reference(s, T, H, I, E, k, q)
    # y enters the logits in BF16: each term off by 2^-8 at most
    mag = ref.product(ref.rmsnorm(s["x"], s["res"], s["nw"], 1e-6)[1],
                      ref.nvfp4_weights(s["gcodes"], s["gscales"]) * s["galpha"].double())[1]
    assert bool(((s["logits"].double() - logits).abs() <= (2.0 ** -8 + 2.0 ** -14) * mag).all())
    ids, rw = torch.empty_like(s["ids"]), torch.empty_like(s["rw"])
    rm.moe_topk_softmax(T, E, k, s["logits"], ids, rw)
    assert torch.equal(ids, s["ids"]) and torch.equal(rw, s["rw"])
    # the experts' part of the output, as a whole: a few independent roundings of each term
    # (int8 codes: half a step of 1/127 of the row's largest, about 3.5 times its rms; E4M3:
    # 2^-4) add up like their squares over the sums
    step = {"bf16": 4 * 2.0 ** -8, "int8": 4 * 3.5 / 254, "e4m3": 2 * 2.0 ** -4}[q]
    got = s["out"].double() - h
    rounding = 2.0 ** -8 * want.norm()
    assert float((got - (want - h)).norm()) <= float(step * (want - h).norm() + rounding)


def test_the_stages_in_a_graph_and_beside_eager_work():
    _say("layer graph")
    T, H, I, E, k = 24, 512, 128, 32, 4
    for q in ("bf16", "int8", "e4m3"):
        s, run = _layer(T, H, I, E, k, q, seed=3)
        run()
        torch.cuda.synchronize()
        keep = {n: s[n].clone() for n in ("res_out", "y", "logits", "ids", "rw", "act", "rows", "out")}
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run(stream=side)
        for _ in range(4):
            for n in keep:
                s[n].zero_()
            graph.replay()
            torch.cuda.synchronize()
            for n, v in keep.items():
                assert torch.equal(s[n].view(torch.uint8), v.view(torch.uint8)), (q, n)
            run()
            torch.cuda.synchronize()
        # new inputs at the same addresses
        s["x"].copy_(_normal(_gen(77), T, H))
        graph.replay()
        torch.cuda.synchronize()
        replayed = s["out"].clone()
        run()
        assert torch.equal(replayed, s["out"]) and not torch.equal(replayed, keep["out"])


def test_two_streams_at_once_give_the_same_results():
    _say("layer two streams")
    a, run_a = _layer(40, 512, 128, 32, 4, "int8", seed=5)
    b, run_b = _layer(17, 768, 64, 16, 2, "bf16", seed=6)
    run_a()
    run_b()
    torch.cuda.synchronize()
    want = a["out"].clone(), b["out"].clone()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a["out"].zero_()
        b["out"].zero_()
        torch.cuda.synchronize()
        run_a(stream=sa)
        run_b(stream=sb)
        torch.cuda.synchronize()
        assert torch.equal(a["out"], want[0]) and torch.equal(b["out"], want[1])


def test_binding_refuses_wrong_tensors():
    _say("binding refusals")
    x = torch.zeros((4, 64), dtype=BF16, device="cuda")
    w, y = torch.ones(64, dtype=BF16, device="cuda"), torch.zeros_like(x)
    with pytest.raises(ValueError, match="x is not contiguous"):
        rm.moe_rmsnorm(32, 8, x.view(8, 32).t(), None, w, 1e-6, 0, None, y, None, None)
    with pytest.raises(ValueError, match="x holds"):
        rm.moe_rmsnorm(5, 64, x, None, w, 1e-6, 0, None, y, None, None)
    with pytest.raises(ValueError, match="weight holds"):
        rm.moe_rmsnorm(4, 64, x, None, w.float(), 1e-6, 0, None, y, None, None)
