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


@pytest.mark.parametrize("fmt", ["bf16", "fp8_b128"])
@pytest.mark.parametrize("T", [1, 8, 16])
def test_layer_on_its_own_output(T, fmt):
    """forward(forward(x)) reads the layer's output buffer and writes it again; a
    slice of that buffer, which the output covers in part, goes through the chain."""
    wl, w, x = _layer_case(T, norm=True, gate=True, seed=T)
    layer = MoELayer(w, wl.k, fmt=fmt, T_max=20, fused_decode=True)
    assert T in layer.decode_ws
    first = layer.forward(x).clone()
    second = layer.forward(first, y=torch.empty_like(x))
    assert torch.equal(layer.forward(layer.forward(x)), second)
    z = x.clone()
    assert layer.forward(z, y=z) is z and torch.equal(z, first)
    g = layer.capture(z, lambda v: layer.forward(v, y=v))
    z.copy_(x)
    g.replay()
    assert torch.equal(z, first)
    if T > 1:
        chain = MoELayer(w, wl.k, fmt=fmt, T_max=20, fused_decode=False)
        layer.forward(x)
        want = chain.forward(layer.y[1:T].clone()).clone()
        assert torch.equal(layer.forward(layer.y[1:T]), want)
    assert abi.moe_device_status() == 0
