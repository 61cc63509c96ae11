"""CPU check of the balance's coefficient: any finite number goes, and nothing else."""

import ctypes

import pytest
import torch

import routed_moe_layer_amd as rm
from tests.test_mxfp4_abi import GRAD, INVALID, LOSS, SMALL, _status

LARGEST = torch.finfo(torch.float32).max


@pytest.mark.parametrize("coef", [LARGEST, -LARGEST, 3.401e38, 0.0, -0.0, 2.0 ** -149])
def test_every_finite_coefficient_goes(coef):
    """(The workspace is looked at behind it, so a short one shows that it went.)"""
    assert ctypes.c_float(coef).value == coef or coef == 3.401e38
    assert _status(rm.moe_balance_loss, **{**LOSS, "coef": coef, "workspace_bytes": 64}) == SMALL


@pytest.mark.parametrize("coef", [float("inf"), float("-inf"), float("nan"), 2.0 * LARGEST])
def test_no_other_does(coef):
    assert _status(rm.moe_balance_loss, **{**LOSS, "coef": coef, "workspace_bytes": 64}) == INVALID
    assert _status(rm.moe_balance_loss_grad, **{**GRAD, "coef": coef}) == INVALID
