"""GPU checks of the expert-stage operators at the ends of their ranges (of the types, the sizes
and the prefix sums) and of their stages on more tokens than one call of the logits takes,
against their definitions in 64 bits (tests/expert_ops.py)."""

import pytest
import torch

import routed_moe_layer_amd as rm
import tests.test_gpu_expert_ops as ops
from tests import expert_ops as ref
from tests.test_gpu_expert_ops import (KERNELS, _call, _check_grouped, _gen, _grouped_problem,
                                       _guarded, _intact, _matvec_check, _norm_check, _normal, _say)

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


# ---------------------------------------------------------------------------------------
# moe_rmsnorm: rows whose squares leave fp32's range
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("q", ["int8", "e4m3"])
@pytest.mark.parametrize("exp,eps", [(e, v) for e in (-120, -90, -75, -60, -45)
                                     for v in (0.0, 1e-30, 1e-6)]
                         + [(e, v) for e in (46, 56, 60, 64, 90, 120) for v in (0.0, 1e-6, 1e30)])
@pytest.mark.parametrize("T,H", [(3, 72), (2, 3584), (2, 65536)])
def test_rmsnorm_of_large_and_small_rows(T, H, exp, eps, q):
    _say(f"rmsnorm T={T} H={H} 2^{exp} eps={eps} {q}")
    # y is about 2^exp / sqrt(eps), at least 2^-110: its row scales are normal fp32 numbers
    x = (_normal(_gen(H + exp), T, H, dtype=torch.float32) * 2.0 ** exp).to(BF16)
    # eps is passed as fp32
    _norm_check(T, H, q, False, True, x=x, eps=float(torch.tensor(eps)))


@pytest.mark.parametrize("value", [2.0 ** 60, 2.0 ** 127, -3.3895e38, 2.0 ** -75, 2.0 ** -126,
                                   2.0 ** -133])
def test_rmsnorm_of_rows_of_one_value(value):
    """With eps = 0 and weight 1 the norm of a constant row is its sign, whatever its value."""
    for H in (8, 256, 65536):
        _say(f"rmsnorm constant {value} H={H}")
        x = torch.full((2, H), value, device="cuda").to(BF16)
        assert float(x[0, 0]) != 0
        w, y = torch.ones(H, dtype=BF16, device="cuda"), torch.empty((2, H), dtype=BF16, device="cuda")
        codes = torch.empty((2, H), dtype=torch.int8, device="cuda")
        scales = torch.empty(2, device="cuda")
        rm.moe_rmsnorm(2, H, x, None, w, 0.0, rm.MOE_QUANT_INT8_ROW_DYNAMIC, None, y, codes, scales)
        sign = 1.0 if value > 0 else -1.0
        assert bool((y.float() == sign).all()) and bool((codes == int(127 * sign)).all())
        rel = 2 * ref.norm_rel(H) / 127
        assert bool(((scales.double() - 1 / 127).abs() <= rel).all())


def test_rmsnorm_of_rows_of_very_different_size_in_one_call():
    """Each row by itself, one of them of zeros, one holding both ends of BF16's range."""
    _say("rmsnorm mixed rows")
    H = 1000
    x = _normal(_gen(3), 6, H, dtype=torch.float32)
    x *= torch.tensor([2.0 ** 110, 1.0, 2.0 ** -110, 0.0, 2.0 ** 70, 2.0 ** -70], device="cuda")[:, None]
    x[4, 5], x[4, 6], x[2, 7] = 2.0 ** 127, 2.0 ** -133, 2.0 ** -133
    x = x.to(BF16)
    for q in ("int8", "e4m3"):
        _, y, codes, scales = _norm_check(6, H, q, False, True, x=x, eps=1e-30)
        assert float(scales[3]) == 0 and not bool(codes[3].any()) and not bool(y[3].any())


def test_rmsnorm_of_a_large_row_with_a_residual():
    """The residual's sum is rounded only where it is stored, at any size; a sum past fp32's
    range marks its row."""
    _say("rmsnorm large residual")
    T, H = 3, 512
    x, res = (_normal(_gen(i), T, H, std=2.0 ** 100) for i in (4, 5))
    x[1, 7] = res[1, 7] = 3.3895e38                     # the largest BF16 value
    w = torch.ones(H, dtype=BF16, device="cuda")
    h, y = ref.rmsnorm(x, res, w, 0.0)
    out, res_out = torch.empty_like(x), torch.empty_like(x)
    codes, scales = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    rm.moe_rmsnorm(T, H, x, res, w, 0.0, rm.MOE_QUANT_INT8_ROW_DYNAMIC, res_out, out, codes, scales)
    ok = [0, 2]
    assert bool(((res_out[ok].double() - h[ok]).abs() <= ref.BF16_HALF_STEP * 1.001 * h[ok].abs()).all())
    tol = (ref.BF16_HALF_STEP + 2 * ref.norm_rel(H)) * y[ok].abs()
    assert bool(((out[ok].double() - y[ok]).abs() <= tol).all())
    assert bool(scales[ok].isfinite().all()) and bool(scales[1].isnan())


# ---------------------------------------------------------------------------------------
# moe_grouped_gemm: prefix sums that fall
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("R,E,N,K", [
    (1 << 24, 10240, 16, 16),                           # tiles of 64 rows, 1.3e9 of them uncut
    (245000, 10240, 16, 16), (245000, 10240, 8, 2048),  # tiles of 32 rows, both ring lengths
    ((1 << 20) + 77, 2000, 24, 16),                     # tiles of 128 rows
    (448100, 1000, 40, 16)])                            # tiles of 256 rows
def test_grouped_gemm_prefix_sums_that_fall(R, E, N, K):
    """Every other expert claims all rows: the tiles that are worked on stay as many as rising
    prefix sums could make.  The experts' weights are alike, so that it does not matter which of
    them a row is multiplied with."""
    _say(f"grouped falling prefix sums R={R} E={E} N={N} K={K}")
    g = _gen(R + E)
    x = torch.randint(-127, 128, (R, K), generator=g, device="cuda", dtype=torch.int8)
    w1 = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    w = w1.expand(E, N, K).contiguous()
    cum = torch.zeros(E, dtype=torch.int32, device="cuda")
    cum[::2] = R
    out, guard = _guarded(R, N)
    rm.moe_grouped_gemm(R, N, K, E, x, cum, w, out, quant=rm.MOE_QUANT_INT8_ROW_DYNAMIC,
                        x_scale=torch.full((R,), 0.5, device="cuda"),
                        w_scale=torch.full((E, N), 0.25, device="cuda"))
    torch.cuda.synchronize()
    assert _intact(guard)
    # an exact int32 sum below 2^25 times 1/8: one rounding to fp32 and one to BF16
    for lo in range(0, R, 1 << 20):
        want = ref.product(x[lo:lo + (1 << 20)], w1)[0] / 8
        got = out[lo:lo + (1 << 20)].double()
        assert bool(((got - want).abs() <= (ref.BF16_HALF_STEP + 2.0 ** -20) * want.abs()).all())


# ---------------------------------------------------------------------------------------
# moe_grouped_gemm: SiTU's parameters
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("beta,lam", [(1e20, 1e20), (1e30, 1e9), (1e-3, 1e30), (1e25, 1e-20)])
@pytest.mark.parametrize("q,R,E,N,K", KERNELS)
def test_grouped_gemm_situ_parameters_whose_product_leaves_fp32(q, R, E, N, K, beta, lam):
    _say(f"grouped SiTU beta={beta} lambda={lam} {q} R={R} E={E} N={N} K={K}")
    p = _grouped_problem(R, E, N, K, q, True, True, "uniform", seed=21)
    p["beta"], p["lam"] = torch.full((E,), beta, device="cuda"), torch.full((E,), lam, device="cuda")
    out, guard = _guarded(R, N)
    _call(p, out)
    torch.cuda.synchronize()
    assert _intact(guard)
    _check_grouped(p, out)


# ---------------------------------------------------------------------------------------
# moe_matvec_nvfp4: sizes next to the borders between the shapes of workgroups (in rows per
# CU, of which there are 256), and tokens that fill the LDS they are kept in
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,N,K", [
    (1, 6143, 48), (1, 6144, 48), (2, 6143, 48), (2, 6144, 48),
    (16, 4096, 144), (16, 4097, 144), (3, 8192, 144), (3, 8193, 144), (16, 16385, 144),
    (32, 2048, 144), (32, 2049, 144), (17, 4097, 144), (32, 8193, 144), (64, 1024, 144),
    (64, 1025, 144), (64, 2049, 144), (64, 4097, 144), (48, 8193, 144), (64, 12289, 160),
    (1, 300, 32768), (2, 300, 16384), (1, 300, 32784), (2, 300, 16400)])
def test_matvec_at_the_borders_of_its_shapes(T, N, K):
    _say(f"matvec T={T} N={N} K={K}")
    for f32 in (True, False):
        _matvec_check(T, N, K, f32, seed=5)


@pytest.mark.parametrize("N", [900, 2100, 4100, 8200, 16400])
def test_matvec_of_a_token_does_not_depend_on_the_others(N):
    """From three tokens on every shape adds an output's terms in the same order."""
    _say(f"matvec slices N={N}")
    x, codes, scales, alpha, y = _matvec_check(64, N, 304, True, seed=6)
    for lo, n in ((0, 3), (7, 16), (20, 32), (16, 48)):
        part = torch.empty((n, N), device="cuda")
        rm.moe_matvec_nvfp4(n, N, 304, x[lo:lo + n], codes, scales, alpha, part, out_f32=True)
        assert torch.equal(part, y[lo:lo + n])


# ---------------------------------------------------------------------------------------
# The E4M3 products as a whole, and the stages on more than 64 tokens
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("R,E,N,K", [(40, 1, 1100, 4096), (600, 1, 2000, 4096),
                                     (20000, 3, 1000, 1024), (300, 4, 500, 8192)])
def test_grouped_gemm_e4m3_sums_as_a_whole(R, E, N, K):
    """Over many outputs the errors add like their squares.  A rounding to BF16 is off by at most
    a uniform half step of 2^-7 of the value: rms 2^-7 / sqrt(12).  Seven products of eight are
    cut below 2^-13 of the largest, uniformly and with either sign: rms 2^-13 / sqrt(3) of it,
    whose square is at most the sum of the eight squares; over K / 8 groups that is 2^-13
    sqrt(7 K / 3) of a product's rms, and the output's rms is sqrt(K) of it (the products are
    independent with zero mean).  2% for the finite number of outputs."""
    _say(f"grouped E4M3 rms R={R} E={E} N={N} K={K}")
    p = _grouped_problem(R, E, N, K, "e4m3", False, False, "uniform", seed=31)
    out, _ = _guarded(R, N)
    _call(p, out)
    want = ops._want(p)[0]
    rms = ((2.0 ** -7) ** 2 / 12 + (2.0 ** -13) ** 2 * 7 / 3) ** 0.5
    assert float((out.double() - want).norm() / want.norm()) <= 1.02 * rms


@pytest.mark.parametrize("q,T,H,I,E,k", [("bf16", 150, 256, 64, 16, 4), ("int8", 129, 256, 64, 24, 2),
                                         ("e4m3", 200, 256, 64, 16, 2)])
def test_the_stages_together_on_more_tokens_than_one_call_of_logits(monkeypatch, q, T, H, I, E, k):
    """The logits are made 64 tokens at a time."""
    one = rm.moe_matvec_nvfp4

    def slices(tokens, N, K, x, codes, scales, alpha, y, **kw):
        for lo in range(0, tokens, rm.MOE_MATVEC_MAX_TOKENS):
            part = slice(lo, min(lo + rm.MOE_MATVEC_MAX_TOKENS, tokens))
            one(part.stop - lo, N, K, x[part], codes, scales, alpha, y[part], **kw)

    monkeypatch.setattr(rm, "moe_matvec_nvfp4", slices)
    ops.test_the_stages_together(q, T, H, I, E, k)
