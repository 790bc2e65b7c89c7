"""MoELayer's buffers hold every batch up to T_max, without a GPU."""

import pytest
import torch

from bit_expert_gemm_b200 import MoELayer, abi


@pytest.mark.parametrize("T_max", [17, 20, 130])
def test_workspace_of_the_shared_expert(T_max):
    H, I, E = 256, 192, 2
    w = {"w_router": torch.zeros((E, H), dtype=torch.bfloat16), "bias": None,
         "w_sh_gate_up": torch.zeros((2 * I, H), dtype=torch.bfloat16),
         "w_sh_down": torch.zeros((H, I), dtype=torch.bfloat16),
         "w8_gu": torch.zeros((E, 2 * I, H), dtype=torch.uint8), "w8_d": torch.zeros((E, H, I), dtype=torch.uint8)}
    layer = MoELayer(w, 2, fmt="fp8_b128", T_max=T_max)
    for T in range(1, T_max + 1):
        assert layer.ws_sh.numel() >= abi.moe_workspace_size(abi.MOE_OP_SWIGLU_BF16, T, H, 1, 1, I)
