"""The one-kernel decode layer on the GPU at the edges of what its calls allow.
Tolerances as in test_gpu_layer_decode and test_gpu_fp8."""

import numpy as np
import pytest
import torch

from bit_expert_gemm_b200 import MoELayer, abi
from tests.helpers import rel_err
from tests.test_gpu_fp8 import _layer_case, _layer_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,T_max", [(1, 1), (3, 20), (16, 16)])
def test_a_layer_too_wide_for_one_kernel_takes_the_chain(T, T_max):
    """I above the one-kernel layer's limit: the default FP8 layer runs all the same
    (16-bit roundings of f, the shared expert and y: 2e-2 normwise)."""
    wl, w, x = _layer_case(T, E=3, k=2, H=128, I=8256, seed=31)
    layer = MoELayer(w, 2, fmt="fp8_b128", T_max=T_max)
    y = layer.forward(x).double().cpu().numpy()
    ref, r = _layer_ref(layer.w, x, 2)
    ok = r["margin"] > 1e-3
    assert ok.any() and rel_err(y[ok], ref[ok]) <= 2e-2
    assert np.isfinite(y).all() and abi.moe_device_status() == 0
