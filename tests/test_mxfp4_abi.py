"""CPU checks of the microscaled FP4 and balance entry points: argument validation (every refusal
returns before any HIP call, so made-up device addresses serve), the binding's look at its tensors,
sizes, and the definitions that the GPU tests compare with."""

import pytest
import torch

import routed_moe_layer_amd as rm
from tests import mxfp4_ops as ref

A = 1 << 20                          # an aligned address that is never used
INVALID, UNSUPPORTED, SMALL = -1, -2, -3
NAN, INF = float("nan"), float("inf")


def _status(fn, *args, **kw):
    with pytest.raises(rm.MoeError) as ei:
        fn(*args, stream=0, **kw)
    return ei.value.status


QUANTIZE = dict(src=A, rows=4, K=64, codes=A, scales=A)
DEQUANTIZE = dict(codes=A, scales=A, rows=4, K=64, out=A)
ROWS = [(dict(rows=0), INVALID), (dict(rows=-3), INVALID), (dict(K=0), INVALID),
        (dict(K=-32), INVALID), (dict(K=48), UNSUPPORTED), (dict(K=65568), UNSUPPORTED),
        (dict(rows=1 << 31), UNSUPPORTED), (dict(rows=1 << 30, K=160), UNSUPPORTED),
        (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(codes=A + 8), INVALID),
        (dict(scales=A + 2), INVALID)]


@pytest.mark.parametrize("change,status", ROWS + [(dict(src=None), INVALID), (dict(src=A + 8), INVALID)])
def test_quantize_refusals(change, status):
    assert _status(rm.moe_quantize_mxfp4, **{**QUANTIZE, **change}) == status


@pytest.mark.parametrize("change,status", ROWS + [(dict(out=None), INVALID), (dict(out=A + 8), INVALID)])
def test_dequantize_refusals(change, status):
    assert _status(rm.moe_dequantize_mxfp4, **{**DEQUANTIZE, **change}) == status


GROUPED = dict(R=8, N=16, K=64, E=4, x_codes=A, x_scales=A, expert_cumsum=A, w_codes=A, w_scales=A,
               out=A, x_rows=8, row_idx=A, row_div=2, situ=True, situ_beta=A, situ_linear_beta=A)


@pytest.mark.parametrize("change,status", [
    (dict(R=0), INVALID), (dict(R=(1 << 24) + 1), UNSUPPORTED), (dict(N=0), INVALID),
    (dict(N=65537), UNSUPPORTED), (dict(K=0), INVALID), (dict(K=48), UNSUPPORTED),
    (dict(K=65568), UNSUPPORTED), (dict(E=0), INVALID), (dict(E=10241), UNSUPPORTED),
    (dict(x_rows=0), INVALID), (dict(x_rows=(1 << 24) + 1), UNSUPPORTED),
    (dict(row_div=0), INVALID), (dict(row_idx=None, x_rows=7), INVALID),
    (dict(situ=False), INVALID), (dict(situ=False, situ_beta=None), INVALID),
    (dict(x_codes=None), INVALID), (dict(x_scales=None), INVALID), (dict(w_codes=None), INVALID),
    (dict(w_scales=None), INVALID), (dict(expert_cumsum=None), INVALID), (dict(out=None), INVALID),
    (dict(x_codes=A + 8), INVALID), (dict(w_codes=A + 8), INVALID), (dict(out=A + 8), INVALID),
    (dict(x_scales=A + 2), INVALID), (dict(w_scales=A + 1), INVALID), (dict(row_idx=A + 2), INVALID),
    (dict(expert_cumsum=A + 1), INVALID), (dict(situ_beta=A + 2), INVALID),
    (dict(situ_linear_beta=A + 2), INVALID)])
def test_grouped_refusals(change, status):
    assert _status(rm.moe_grouped_gemm_mxfp4, **{**GROUPED, **change}) == status


LOSS = dict(T=4, num_experts=8, top_k=2, logits=A, expert_ids=A, coef=0.01, counts=A, prob_sums=A,
            tokens=A, loss=A, workspace=A, token_mask=A, workspace_bytes=1 << 20)
COMMON = [(dict(T=0), INVALID), (dict(T=(1 << 21) + 1), UNSUPPORTED), (dict(num_experts=0), INVALID),
          (dict(num_experts=4097), UNSUPPORTED), (dict(coef=NAN), INVALID), (dict(coef=INF), INVALID),
          (dict(coef=-INF), INVALID), (dict(logits=None), INVALID), (dict(counts=None), INVALID),
          (dict(tokens=None), INVALID), (dict(logits=A + 2), INVALID),
          (dict(logits=A + 1, logits_bf16=True), INVALID), (dict(counts=A + 2), INVALID),
          (dict(tokens=A + 2), INVALID)]


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(top_k=0), INVALID), (dict(top_k=65), UNSUPPORTED), (dict(expert_ids=None), INVALID),
    (dict(prob_sums=None), INVALID), (dict(loss=None), INVALID), (dict(workspace=None), INVALID),
    (dict(expert_ids=A + 2), INVALID), (dict(prob_sums=A + 1), INVALID), (dict(loss=A + 2), INVALID),
    (dict(workspace=A + 64), INVALID), (dict(workspace_bytes=64), SMALL),
    (dict(T=5000, workspace_bytes=rm.moe_balance_workspace_size(5000, 8) - 1), SMALL)])
def test_balance_loss_refusals(change, status):
    assert _status(rm.moe_balance_loss, **{**LOSS, **change}) == status


GRAD = dict(T=4, num_experts=8, logits=A, counts=A, tokens=A, coef=0.01, grad_logits=A, grad_loss=A,
            token_mask=A, add=A)


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(grad_logits=None), INVALID), (dict(grad_logits=A + 2), INVALID),
    (dict(add=A + 2), INVALID), (dict(grad_loss=A + 2), INVALID)])
def test_balance_grad_refusals(change, status):
    assert _status(rm.moe_balance_loss_grad, **{**GRAD, **change}) == status


def test_balance_workspace_size_grows_with_both():
    for Es in ((1, 16, 17, 64, 65, 896, 4096),):
        for T in (1, 7, 8, 9, 31, 32, 33, 127, 129, 1000, 4096, 4097, 70000, 1 << 21):
            row = [rm.moe_balance_workspace_size(T, E) for E in Es]
            assert row == sorted(row)
    for E in (1, 16, 17, 64, 65, 896, 4096):
        col = [rm.moe_balance_workspace_size(T, E) for T in range(1, 9000, 37)]
        assert col == sorted(col)
    for T, E, status in ((0, 4, INVALID), (4, 0, INVALID), (4, 4097, UNSUPPORTED)):
        with pytest.raises(rm.MoeError) as ei:
            rm.moe_balance_workspace_size(T, E)
        assert ei.value.status == status


BF16 = ({torch.bfloat16, torch.int16, torch.uint16}, {torch.float16, torch.float32})
F32 = ({torch.float32}, {torch.int32, torch.float64, torch.bfloat16})
I32 = ({torch.int32}, {torch.float32, torch.int64, torch.uint32})
CODES = ({torch.uint8, torch.int8}, {torch.float8_e4m3fn, torch.bool, torch.int16})
SCALES = ({torch.uint8, torch.float8_e8m0fnu}, {torch.int8, torch.float8_e4m3fn, torch.float32})
MASK = ({torch.bool, torch.uint8}, {torch.int8, torch.int32})
RAW = ({torch.uint8, torch.int8}, {torch.bfloat16, torch.float32})
quantize, dequantize = (rm.moe_quantize_mxfp4, QUANTIZE), (rm.moe_dequantize_mxfp4, DEQUANTIZE)
grouped = (rm.moe_grouped_gemm_mxfp4, GROUPED)
loss, grad = (rm.moe_balance_loss, LOSS), (rm.moe_balance_loss_grad, GRAD)
TYPES = ([(*quantize, {}, "src", BF16), (*dequantize, {}, "out", BF16)]
         + [(*f, {}, "codes", CODES) for f in (quantize, dequantize)]
         + [(*f, {}, "scales", SCALES) for f in (quantize, dequantize)]
         + [(*grouped, {}, n, CODES) for n in ("x_codes", "w_codes")]
         + [(*grouped, {}, n, SCALES) for n in ("x_scales", "w_scales")]
         + [(*grouped, {}, n, I32) for n in ("row_idx", "expert_cumsum")]
         + [(*grouped, {}, n, F32) for n in ("situ_beta", "situ_linear_beta")]
         + [(*grouped, {}, "out", BF16)]
         + [(*loss, {"logits_bf16": b}, "logits", k) for b, k in ((False, F32), (True, BF16))]
         + [(*loss, {}, n, I32) for n in ("expert_ids", "counts", "tokens")]
         + [(*loss, {}, n, F32) for n in ("prob_sums", "loss")]
         + [(*loss, {}, "token_mask", MASK), (*loss, {}, "workspace", RAW)]
         + [(*grad, {"logits_bf16": b}, n, k) for b, k in ((False, F32), (True, BF16))
            for n in ("logits", "add", "grad_logits")]
         + [(*grad, {}, n, I32) for n in ("counts", "tokens")]
         + [(*grad, {}, "grad_loss", F32), (*grad, {}, "token_mask", MASK)])


@pytest.mark.parametrize("fn,args,change,name,kind", TYPES,
                         ids=[f"{f.__name__}-{n}-{c}" for f, _, c, n, _ in TYPES])
def test_types(fn, args, change, name, kind):
    good, bad = kind
    for dtype in good | bad:
        t = torch.zeros(1 << 14, dtype=torch.uint8).view(dtype)
        match = "is not on a GPU" if dtype in good else f"{name} holds {dtype}, not"
        with pytest.raises(ValueError, match=match):
            fn(**{**args, **change, name: t}, stream=0)


def test_the_stride_of_scales_is_the_headers():
    assert [rm.moe_mxfp4_scale_stride(K) for K in (32, 96, 128, 160, 256, 2912, 65536)] == [
        4, 4, 4, 8, 8, 92, 2048]


# ---------------------------------------------------------------------------------------
# The definitions.
# ---------------------------------------------------------------------------------------
def test_quantization_by_hand():
    row = [0.0] * 32
    row[:8] = [6.0, -5.0, 3.5, 2.5, 0.25, -0.25, 0.75, 1.75]
    x = torch.tensor([row, [0.0] * 32, [3.0 * 2.0 ** -100] + [0.0] * 31], dtype=torch.bfloat16)
    codes, scales = ref.quantize(x)
    assert scales.tolist() == [[127, 0, 0, 0], [0, 0, 0, 0], [127 - 100 + 1 - 2, 0, 0, 0]]
    got = ref.decode(codes, scales)
    assert got[0, :8].tolist() == [6.0, -4.0, 4.0, 2.0, 0.0, -0.0, 1.0, 2.0]
    assert codes[0, 2].item() == 0x80 and not codes[1].any()    # 0.25 and -0.25: 0 and -0
    assert got[2, 0].item() == 3.0 * 2.0 ** -100
    x[1, 5], x[2, 9] = NAN, INF
    codes, scales = ref.quantize(x)
    assert scales[1:, 0].tolist() == [255, 255] and not codes[1:].any()
    assert ref.decode(codes, scales)[1:].isnan().all()


def test_quantization_is_the_nearest_value_under_its_scale():
    x = torch.randn((64, 96), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    codes, scales = ref.quantize(x)
    got, s = ref.decode(codes, scales), torch.exp2(scales[:, :3].double() - 127).repeat_interleave(32, 1)
    grid = torch.tensor(ref.ref.E2M1 + tuple(-v for v in ref.ref.E2M1), dtype=torch.float64)
    nearest = (x.double()[:, :, None] - grid * s[:, :, None]).abs().amin(2)
    assert torch.equal((got - x.double()).abs(), nearest)
    top = (x.double().abs() / s).view(64, 3, 32).amax(2)
    assert bool((top >= 4).all()) and bool((top < 8).all())


@pytest.mark.parametrize("masked", [False, True])
def test_balance_gradient_is_the_losss(masked):
    g = torch.Generator().manual_seed(2)
    T, E, k, coef = 6, 5, 2, 0.3
    z = torch.randn((T, E), generator=g, dtype=torch.float64)
    z[1, 3] = -INF
    ids = torch.randint(0, E, (T, k), generator=g)
    mask = torch.tensor([1, 1, 0, 1, 0, 1], dtype=torch.bool) if masked else None
    counts, _, _, tokens, value, _ = ref.balance(z, ids, mask, coef)
    got, _ = ref.balance_grad(z, mask, counts, tokens, coef, 1.0, None)
    at = lambda z: ref.balance(z, ids, mask, coef)[4]  # noqa: E731
    assert value > 0 and counts.sum() == tokens * k
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if torch.isinf(z[t, e]):
                assert got[t, e] == 0
                continue
            step = torch.zeros_like(z)
            step[t, e] = h
            # a central difference of a smooth function: h^2 of its size, and 2^-52 / h
            assert abs((at(z + step) - at(z - step)) / (2 * h) - got[t, e]) < 1e-9
