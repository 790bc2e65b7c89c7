"""Layers sized for a little more than a decode batch, run on fewer tokens: the
shared expert of a separate call takes its small-batch form there."""

import pytest
import torch

from bit_expert_gemm_b200 import MoELayer, abi
from tests.test_gpu_fp8 import _layer_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8_b128"])
@pytest.mark.parametrize("T,T_max", [(3, 17), (7, 20), (16, 40)])
def test_chain_on_fewer_tokens(T, T_max, fmt):
    """The chain of calls gives the same rows in a layer of T_max tokens as in one of T."""
    wl, w, x = _layer_case(T, I=256, seed=T)
    want = MoELayer(w, wl.k, fmt=fmt, T_max=T, fused_decode=False).forward(x)
    got = MoELayer(w, wl.k, fmt=fmt, T_max=T_max, fused_decode=False).forward(x)
    assert torch.isfinite(want).all() and torch.equal(got, want)
    assert abi.moe_device_status() == 0
