"""CPU checks of the binding's look at the types of its tensors (moe_rmsnorm, moe_matvec_nvfp4,
moe_grouped_gemm, moe_combine): a type of the right width but the wrong meaning is refused, and
the types a buffer may have get past that check (to the one that wants them on a GPU)."""

import pytest
import torch

import routed_moe_layer_amd as rm
from tests.test_expert_ops_abi import COMBINE, GROUPED, MATVEC, NORM

NONE, INT8, E4M3 = rm.MOE_QUANT_NONE, rm.MOE_QUANT_INT8_ROW_DYNAMIC, rm.MOE_QUANT_E4M3_ROW_DYNAMIC
BF16 = ({torch.bfloat16, torch.int16, torch.uint16}, {torch.float16, torch.float32})
F32 = ({torch.float32}, {torch.int32, torch.uint32, torch.float64, torch.bfloat16})
I32 = ({torch.int32}, {torch.float32, torch.int64, torch.uint32})
ROWS_INT8 = ({torch.int8, torch.uint8}, {torch.float8_e4m3fn, torch.bool, torch.bfloat16})
ROWS_E4M3 = ({torch.float8_e4m3fn, torch.uint8},
             {torch.int8, torch.float8_e5m2, torch.float8_e4m3fnuz, torch.bfloat16})
CODES = ({torch.uint8, torch.int8}, {torch.float8_e4m3fn, torch.bool, torch.int16})
SCALES = ({torch.uint8, torch.float8_e4m3fn}, {torch.int8, torch.float8_e5m2, torch.float32})

norm = (rm.moe_rmsnorm, NORM)
matvec = (rm.moe_matvec_nvfp4, MATVEC)
grouped = (rm.moe_grouped_gemm, GROUPED)
combine = (rm.moe_combine, COMBINE)
CASES = (
    [(*norm, {}, n, BF16) for n in ("x", "residual", "weight", "residual_out", "y")]
    + [(*norm, {}, "scales", F32), (*norm, {"quant": INT8}, "codes", ROWS_INT8),
       (*norm, {"quant": E4M3}, "codes", ROWS_E4M3)]
    + [(*matvec, {}, "x", BF16), (*matvec, {}, "codes", CODES), (*matvec, {}, "scales", SCALES),
       (*matvec, {}, "alpha", F32), (*matvec, {}, "y", BF16), (*matvec, {"out_f32": True}, "y", F32)]
    + [(*grouped, {"quant": q}, n, kind) for q, kind in ((NONE, BF16), (INT8, ROWS_INT8),
                                                         (E4M3, ROWS_E4M3)) for n in ("x", "w")]
    + [(*grouped, {}, n, F32) for n in ("x_scale", "w_scale", "situ_beta", "situ_linear_beta")]
    + [(*grouped, {}, n, I32) for n in ("row_idx", "expert_cumsum")] + [(*grouped, {}, "out", BF16)]
    + [(*combine, {}, n, BF16) for n in ("rows", "route_weights", "add", "out")]
    + [(*combine, {}, "expanded_row_idx", I32)])


@pytest.mark.parametrize("fn,args,change,name,kind", CASES,
                         ids=[f"{f.__name__}-{n}-{c}" for f, _, c, n, _ in CASES])
def test_types(fn, args, change, name, kind):
    good, bad = kind
    for dtype in good | bad:
        t = torch.zeros(1 << 14, dtype=torch.uint8).view(dtype)
        match = "is not on a GPU" if dtype in good else f"{name} holds {dtype}, not"
        with pytest.raises(ValueError, match=match):
            fn(**{**args, **change, name: t}, stream=0)
