"""CPU checks of the expert-stage entry points' argument validation (moe_rmsnorm,
moe_matvec_nvfp4, moe_grouped_gemm, moe_combine): every refusal returns before any HIP call,
so made-up device addresses serve; and of the binding's look at its tensors."""

import pytest
import torch

import routed_moe_layer_amd as rm

A = 1 << 20                          # an aligned address that is never used
INVALID, UNSUPPORTED = -1, -2
NONE, INT8, NVFP4, E4M3 = (rm.MOE_QUANT_NONE, rm.MOE_QUANT_INT8_ROW_DYNAMIC,
                           rm.MOE_QUANT_NVFP4_G16, rm.MOE_QUANT_E4M3_ROW_DYNAMIC)


def _status(fn, *args, **kw):
    with pytest.raises(rm.MoeError) as ei:
        fn(*args, stream=0, **kw)
    return ei.value.status


NORM = dict(T=4, H=64, x=A, residual=A, weight=A, eps=1e-6, quant=INT8, residual_out=A, y=A,
            codes=A, scales=A)


@pytest.mark.parametrize("change,status", [
    (dict(T=0), INVALID), (dict(T=-1), INVALID), (dict(T=(1 << 21) + 1), UNSUPPORTED),
    (dict(H=0), INVALID), (dict(H=12), UNSUPPORTED), (dict(H=65544), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(residual=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(quant=NVFP4), INVALID), (dict(quant=7), INVALID),
    (dict(quant=NONE), INVALID),                                  # codes without a format
    (dict(quant=NONE, codes=None, scales=None, y=None), INVALID),  # nothing to write
    (dict(x=A + 8), INVALID), (dict(residual=A + 2), INVALID), (dict(weight=A + 8), INVALID),
    (dict(residual_out=A + 8), INVALID), (dict(y=A + 8), INVALID), (dict(codes=A + 4), INVALID),
    (dict(scales=A + 2), INVALID)])
def test_rmsnorm_refusals(change, status):
    assert _status(rm.moe_rmsnorm, **{**NORM, **change}) == status


MATVEC = dict(T=2, N=8, K=64, x=A, codes=A, scales=A, alpha=A, y=A)


@pytest.mark.parametrize("change,status", [
    (dict(T=0), INVALID), (dict(T=65), UNSUPPORTED), (dict(N=0), INVALID),
    (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(K=0), INVALID), (dict(K=40), UNSUPPORTED),
    (dict(K=65552), UNSUPPORTED), (dict(x=None), INVALID), (dict(codes=None), INVALID),
    (dict(scales=None), INVALID), (dict(alpha=None), INVALID), (dict(y=None), INVALID),
    (dict(x=A + 8), INVALID), (dict(codes=A + 8), INVALID), (dict(scales=A + 2), INVALID),
    (dict(alpha=A + 2), INVALID), (dict(y=A + 4), INVALID)])
def test_matvec_refusals(change, status):
    assert _status(rm.moe_matvec_nvfp4, **{**MATVEC, **change}) == status


GROUPED = dict(R=8, N=16, K=64, E=4, x=A, expert_cumsum=A, w=A, out=A, quant=INT8, x_scale=A,
               w_scale=A, x_rows=8, row_idx=A, row_div=2, situ=True, situ_beta=A,
               situ_linear_beta=A)


@pytest.mark.parametrize("change,status", [
    (dict(R=0), INVALID), (dict(R=(1 << 24) + 1), UNSUPPORTED), (dict(N=0), INVALID),
    (dict(N=65537), UNSUPPORTED), (dict(K=0), INVALID), (dict(K=24), UNSUPPORTED),
    (dict(K=65552), UNSUPPORTED), (dict(E=0), INVALID), (dict(E=10241), UNSUPPORTED),
    (dict(x_rows=0), INVALID), (dict(x_rows=(1 << 24) + 1), UNSUPPORTED),
    (dict(row_div=0), INVALID), (dict(row_idx=None, x_rows=7), INVALID),
    (dict(quant=NVFP4), INVALID), (dict(quant=9), INVALID),
    (dict(quant=NONE), INVALID),                                  # scales without 8-bit rows
    (dict(quant=NONE, x_scale=None, w_scale=None, K=20), UNSUPPORTED),
    (dict(x_scale=None), INVALID), (dict(w_scale=None), INVALID),
    (dict(situ=False), INVALID), (dict(situ=False, situ_beta=None), INVALID),
    (dict(x=None), INVALID), (dict(expert_cumsum=None), INVALID), (dict(w=None), INVALID),
    (dict(out=None), INVALID), (dict(x=A + 8), INVALID), (dict(w=A + 8), INVALID),
    (dict(out=A + 8), INVALID), (dict(x_scale=A + 2), INVALID), (dict(row_idx=A + 2), INVALID),
    (dict(expert_cumsum=A + 1), INVALID), (dict(situ_beta=A + 2), INVALID)])
def test_grouped_gemm_refusals(change, status):
    assert _status(rm.moe_grouped_gemm, **{**GROUPED, **change}) == status


COMBINE = dict(T=4, H=64, k=2, R=8, rows=A, expanded_row_idx=A, route_weights=A, add=A, out=A)


@pytest.mark.parametrize("change,status", [
    (dict(T=0), INVALID), (dict(T=(1 << 21) + 1), UNSUPPORTED), (dict(H=0), INVALID),
    (dict(H=12), UNSUPPORTED), (dict(H=65544), UNSUPPORTED), (dict(k=0), INVALID),
    (dict(k=65), UNSUPPORTED), (dict(T=1 << 20, k=32), UNSUPPORTED), (dict(R=0), INVALID),
    (dict(R=(1 << 24) + 1), UNSUPPORTED), (dict(rows=None), INVALID),
    (dict(expanded_row_idx=None), INVALID), (dict(route_weights=None), INVALID),
    (dict(out=None), INVALID), (dict(rows=A + 8), INVALID), (dict(add=A + 8), INVALID),
    (dict(out=A + 2), INVALID), (dict(expanded_row_idx=A + 2), INVALID),
    (dict(route_weights=A + 1), INVALID)])
def test_combine_refusals(change, status):
    assert _status(rm.moe_combine, **{**COMBINE, **change}) == status


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x is not on a GPU"):
        rm.moe_rmsnorm(**{**NORM, "x": x}, stream=0)
    with pytest.raises(ValueError, match="codes is not on a GPU"):
        rm.moe_matvec_nvfp4(**{**MATVEC, "codes": torch.zeros((8, 32), dtype=torch.uint8)}, stream=0)
    with pytest.raises(ValueError, match="w is not on a GPU"):
        rm.moe_grouped_gemm(**{**GROUPED, "w": torch.zeros((4, 32, 64), dtype=torch.int8)}, stream=0)
    with pytest.raises(ValueError, match="rows is not on a GPU"):
        rm.moe_combine(**{**COMBINE, "rows": torch.zeros((8, 64), dtype=torch.bfloat16)}, stream=0)


def test_the_e4m3_rows_are_not_a_routing_mode():
    d = rm.MoeDims(64, 64, 4, 2)
    with pytest.raises(rm.MoeError) as ei:
        rm.moe_workspace_size(d, 4, E4M3)
    assert ei.value.status == INVALID
    with pytest.raises(rm.MoeError) as ei:
        rm.moe_route(d, 4, A, A, E4M3, A, A, A, A, A, A, A, A, workspace_bytes=1 << 30, stream=0)
    assert ei.value.status == INVALID
