"""The one-kernel decode layer's limits, without a GPU: the workspace size is 0
for exactly the sizes that the calls refuse, MoELayer leaves those to the chain
of calls, and the output may take the input's place."""

import ctypes

import pytest
import torch

from bit_expert_gemm_b200 import MoELayer, abi

P = ctypes.c_void_p


def _refusal(T, H, E, k, I):
    """The status of a call whose workspace has no bytes: nothing is launched."""
    return abi.load().moe_layer_decode_bf16(P(4096), T, H, None, ctypes.c_float(1e-6), None, P(4096), None, E, k, I,
                                            P(4096), P(4096), None, None, 0, None, None, P(1 << 20), P(4096), 0, None)


@pytest.mark.parametrize("T,H,E,k,I,takes", [
    (1, 64, 1, 1, 64, True), (16, 2560, 1024, 16, 8192, True), (10, 4096, 8, 8, 128, True),
    (17, 64, 8, 2, 64, False), (16, 2624, 8, 2, 64, False), (1, 4160, 8, 2, 64, False), (1, 96, 8, 2, 64, False),
    (1, 64, 8, 2, 8256, False), (1, 64, 8, 2, 96, False), (1, 64, 32, 17, 64, False), (1, 64, 2, 3, 64, False),
    (1, 64, 1025, 2, 64, False)])
def test_workspace_size_is_zero_where_the_call_refuses(T, H, E, k, I, takes):
    assert (abi.moe_workspace_size(abi.MOE_OP_LAYER_DECODE, T, H, E, k, I) > 0) == takes
    assert _refusal(T, H, E, k, I) == (abi.MOE_ERR_WORKSPACE if takes else abi.MOE_ERR_UNSUPPORTED)


@pytest.mark.parametrize("I,sizes", [(8192, list(range(1, 17))), (8256, [])])
def test_layers_outside_the_limits_keep_the_chain(I, sizes):
    H, E = 64, 2
    w = {"w_router": torch.zeros((E, H), dtype=torch.bfloat16), "bias": None,
         "w_sh_gate_up": torch.zeros((2 * I, H), dtype=torch.bfloat16),
         "w_sh_down": torch.zeros((H, I), dtype=torch.bfloat16),
         "w8_gu": torch.zeros((E, 2 * I, H), dtype=torch.uint8), "w8_d": torch.zeros((E, H, I), dtype=torch.uint8)}
    assert sorted(MoELayer(w, 2, fmt="fp8_b128", T_max=20).decode_ws) == sizes


def test_y_may_be_x_but_not_a_part_of_it():
    def call(y):  # no workspace bytes: the last check before a launch refuses
        return abi.load().moe_layer_decode_bf16(P(4096), 4, 256, None, ctypes.c_float(1e-6), None, P(4096), None, 16, 2,
                                                64, P(4096), P(4096), None, None, 0, None, None, P(y), P(4096), 0, None)

    nb = 4 * 256 * 2
    assert call(4096) == call(4096 + nb) == call(4096 - nb) == abi.MOE_ERR_WORKSPACE
    assert call(4096 + 512) == call(4096 + nb - 16) == call(4096 - 512) == abi.MOE_ERR_INVALID_ARG
