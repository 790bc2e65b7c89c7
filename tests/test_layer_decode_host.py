"""The one-kernel decode layer without a GPU: workspace sizes, limits and the
refusals of the C ABI and of the binding."""

import ctypes

import pytest
import torch

from bit_expert_gemm_b200 import abi

P = ctypes.c_void_p
EPS = ctypes.c_float(1e-6)


def _code(fn, *args):
    return getattr(abi.load(), fn)(*args)


def _bf16(x=P(4096), T=4, H=256, norm=None, gate=None, router=P(4096), E=16, k=2, I=64, gu=P(4096), d=P(4096),
          shgu=None, shd=None, dtype=0, y=P(1 << 20), ws=P(4096), n=1 << 30):
    return _code("moe_layer_decode_bf16", x, T, H, norm, EPS, gate, router, None, E, k, I, gu, d, shgu, shd, dtype, None,
                 None, y, ws, n, None)


def test_workspace_size_and_limits():
    size = abi.load().moe_workspace_size
    need = 16 * 512 * 4 + 160 * 640 * 4 + 16 * 640 * 4 + 160 * 640 * 2 + 160 * 5 * 4
    assert need <= size(abi.MOE_OP_LAYER_DECODE, 16, 2048, 512, 10, 640) <= need + 2048
    assert size(abi.MOE_OP_LAYER_DECODE, 17, 2048, 512, 10, 640) == 0
    assert size(abi.MOE_OP_LAYER_DECODE, 16, 2624, 512, 10, 640) == 0  # T * H > 40960
    assert size(abi.MOE_OP_LAYER_DECODE, 10, 4096, 512, 10, 640) > 0
    assert size(abi.MOE_OP_LAYER_DECODE, 1, 4160, 512, 10, 640) == 0


def test_c_refusals():
    bad, uns, ws = abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED, abi.MOE_ERR_WORKSPACE
    assert _bf16(T=17) == uns and _bf16(H=200) == uns and _bf16(H=4160) == uns and _bf16(T=16, H=2624) == uns
    assert _bf16(I=96) == uns and _bf16(I=8256) == uns and _bf16(k=17, E=32) == uns and _bf16(k=17) == uns
    assert _bf16(k=3, E=2) == uns and _bf16(E=1025) == uns
    assert _bf16(T=-1) == bad and _bf16(k=0) == bad and _bf16(dtype=5) == bad
    assert _bf16(x=None) == bad and _bf16(router=None) == bad and _bf16(gu=None) == bad and _bf16(y=None) == bad
    assert _bf16(x=P(4104)) == bad and _bf16(gu=P(4104)) == bad and _bf16(norm=P(4104)) == bad
    assert _bf16(shgu=P(4096)) == bad and _bf16(gate=P(4096)) == bad  # half a shared expert; a gate without one
    assert _bf16(y=P(4096 + 1024)) == bad and "overlaps" in abi.load().moe_last_error().decode()
    assert _bf16(ws=P(4112)) == ws and _bf16(n=100) == ws
    assert _bf16(T=0, x=None, y=None, ws=None) == abi.MOE_OK
    # FP8: scales are needed
    assert _code("moe_layer_decode_fp8_b128", P(4096), 4, 256, None, EPS, None, P(4096), None, 16, 2, 64, P(4096), None,
                 P(4096), P(4096), None, None, 0, None, None, P(1 << 20), P(4096), 1 << 30, None) == bad


def test_binding_refusals():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    r, gu, d = torch.zeros_like(x[:1]).expand(4, 64), torch.zeros((4, 128, 64)), torch.zeros((4, 64, 64))
    with pytest.raises(ValueError, match="experts"):
        abi.moe_layer_decode_bf16(x, r, None, 2, gu, d)  # FP32 weights
    gu, d = gu.to(x.dtype), d.to(x.dtype)
    with pytest.raises(ValueError, match="experts"):
        abi.moe_layer_decode_bf16(x, r, None, 2, gu, d[:, :32])
    with pytest.raises(ValueError, match="bias"):
        abi.moe_layer_decode_bf16(x, r, torch.zeros(4, dtype=torch.float64), 2, gu, d)
    with pytest.raises(ValueError, match="norm_w"):
        abi.moe_layer_decode_bf16(x, r, None, 2, gu, d, norm_w=torch.zeros(64))
    with pytest.raises(ValueError, match="w_sh_down"):
        abi.moe_layer_decode_bf16(x, r, None, 2, gu, d, w_sh_gate_up=gu[0], w_sh_down=d[0, :32])
    with pytest.raises(ValueError, match="topk_idx"):
        abi.moe_layer_decode_bf16(x, r, None, 2, gu, d, topk_idx=torch.zeros((2, 2), dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        abi.moe_layer_decode_bf16(x, r.contiguous(), None, 2, gu, d)
    from bit_expert_gemm_b200 import MoELayer

    with pytest.raises(ValueError, match="fused_decode"):
        MoELayer({"w_router": r, "w_sh_down": d[0], "w_gu": d, "bias": None}, 2, fmt="nvfp4", T_max=1, fused_decode=True)


def test_negative_or_nan_eps_is_refused():
    b, b2 = P(256), P(1 << 20)
    for eps in (-1.0, float("nan")):
        rc = _code("moe_layer_decode_bf16", b, 4, 128, b, eps, None, b, None, 8, 2, 64, b, b, None, None, 0, None, None,
                   b2, b, 1 << 24, None)
        assert rc == abi.MOE_ERR_INVALID_ARG
        assert "eps" in abi.load().moe_last_error().decode()
