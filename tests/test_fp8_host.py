"""FP8 E4M3 with a scale per block of 128, without a GPU: the oracle's pins and
the refusals of the C ABI and of the binding."""

import ctypes

import numpy as np
import pytest
import torch

from bit_expert_gemm_b200 import abi
from oracle import fp8, moe

P = ctypes.c_void_p


def _code(fn, *args):
    return getattr(abi.load(), fn)(*args)


@pytest.mark.parametrize("rows,K,br", [(1, 16, 1), (5, 128, 1), (3, 272, 1), (130, 144, 128), (128, 128, 128)])
def test_oracle_quantise_against_torch(rows, K, br):
    g = torch.Generator().manual_seed(rows + K)
    v = (torch.randn((rows, K), generator=g) * torch.exp(torch.randn((rows, 1), generator=g) * 3)).to(torch.bfloat16)
    codes, scales = fp8.quantize(v.float().numpy(), br)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            b = v[i * br:(i + 1) * br, j * 128:(j + 1) * 128].float()
            a = b.abs().max()
            want = (b * (torch.tensor(448.0) / a)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            assert np.array_equal(codes[i * br:(i + 1) * br, j * 128:(j + 1) * 128], want)
            assert scales[i, j] == (a / torch.tensor(448.0)).item()
    # e4m3 keeps 4 significant bits: half a step is 2^-4 of the value, or half of the smallest step times the scale
    s = np.repeat(np.repeat(scales, br, 0)[:rows], 128, 1)[:, :K]
    err = np.abs(fp8.dequant(codes, scales, br) - v.double().numpy())
    assert np.all(err <= np.maximum(np.abs(v.double().numpy()) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 1e-6))


def test_oracle_zero_block_and_identity():
    codes, scales = fp8.quantize(np.zeros((2, 130)))
    assert not codes.any() and np.all(scales == np.float32(2.0 ** -80) / np.float32(448))
    v = np.array([[448.0, -1.5, 0.0, 2.0 ** -9] + [0.0] * 124])  # on the grid, scale 1
    codes, scales = fp8.quantize(v)
    assert scales[0, 0] == 1 and np.array_equal(fp8.dequant(codes, scales), v)


def test_oracle_expert_is_the_plain_expert_on_the_grid():
    """Where x and h are already on a block's grid, quantising changes nothing."""
    x = np.zeros((1, 128))
    x[0, 0] = 448.0
    wg, wu, wd = np.zeros((64, 128)), np.zeros((64, 128)), np.eye(8, 64)
    wg[:, 0] = 100.0  # silu(g) = g to the last bit
    wu[0, 0], wu[1, 0] = 1.0 / 448, 0.5 / 448
    f, h = fp8.swiglu_expert(x, wg, wu, wd)
    f0, h0 = moe.swiglu_expert(x, wg, wu, wd)
    assert np.allclose(f, f0, rtol=1e-6) and np.array_equal(h, h0)


def test_workspace_sizes():
    size = abi.load().moe_workspace_size
    need = 64 * 2048 + 64 * 16 * 4 + 640 * 640 + 640 * 5 * 4
    assert need <= size(abi.MOE_OP_SWIGLU_FP8_B128, 64, 2048, 512, 10, 640) <= need + 1024
    assert size(abi.MOE_OP_SWIGLU_FP8_B128, 0, 2048, 512, 10, 640) == 0


def test_c_refusals():
    b, m = P(256), P(264)  # never dereferenced: the checks come first
    q = "moe_fp8_quantize_b128"
    assert _code(q, b, 1, 4, 24, 1, 0, b, b, None) == abi.MOE_ERR_UNSUPPORTED  # K % 16
    assert _code(q, b, 1, 4, 32, 64, 0, b, b, None) == abi.MOE_ERR_UNSUPPORTED  # block_rows
    assert _code(q, b, 1, -4, 32, 1, 0, b, b, None) == abi.MOE_ERR_INVALID_ARG
    assert _code(q, b, 1, 4, 32, 1, 7, b, b, None) == abi.MOE_ERR_INVALID_ARG  # dtype
    assert _code(q, None, 1, 4, 32, 1, 0, b, b, None) == abi.MOE_ERR_INVALID_ARG
    assert _code(q, m, 1, 4, 32, 1, 0, b, b, None) == abi.MOE_ERR_INVALID_ARG  # misaligned
    assert _code(q, None, 1, 0, 32, 1, 0, None, None, None) == abi.MOE_OK
    g = "moe_grouped_gemm_fp8_b128"
    assert _code(g, b, b, b, b, 4, 8, 40, 32, 2, b, b, 0, 0, b, None) == abi.MOE_ERR_UNSUPPORTED  # K % 16
    assert _code(g, b, b, b, b, 4, 8, 32, 40, 2, b, b, 0, 0, b, None) == abi.MOE_ERR_UNSUPPORTED  # N % 16
    assert _code(g, b, b, b, b, 4, 8, 32, 32, 1025, b, b, 0, 0, b, None) == abi.MOE_ERR_UNSUPPORTED
    assert _code(g, b, b, b, b, 4, 8, 32, 1 << 22, 1024, b, b, 0, 0, b, None) == abi.MOE_ERR_UNSUPPORTED  # E*N
    assert _code(g, b, b, b, None, 4, 8, 32, 32, 2, b, b, 0, 0, b, None) == abi.MOE_ERR_INVALID_ARG  # no offsets
    assert _code(g, b, b, None, b, 4, 8, 32, 32, 2, b, b, 0, 0, b, None) == abi.MOE_ERR_INVALID_ARG  # rows != T
    assert _code(g, b, b, b, b, 0, 8, 32, 32, 2, b, b, 0, 0, b, None) == abi.MOE_ERR_INVALID_ARG  # no tokens
    assert _code(g, b, b, b, b, 4, 8, 32, 32, 2, m, b, 0, 0, b, None) == abi.MOE_ERR_INVALID_ARG  # misaligned w
    assert _code(g, b, None, b, b, 4, 8, 32, 32, 2, b, b, 0, 0, b, None) == abi.MOE_ERR_INVALID_ARG
    assert _code(g, None, None, None, None, 0, 0, 32, 32, 1, None, None, 0, 0, None, None) == abi.MOE_OK
    s = "moe_grouped_swiglu_fp8_b128"
    assert _code(s, b, b, b, 4, 8, 96, 64, 2, b, b, b, b, 0, 0, b, b, 1 << 20, None) == abi.MOE_ERR_UNSUPPORTED
    assert _code(s, b, b, b, 4, 8, 128, 32, 2, b, b, b, b, 0, 0, b, b, 1 << 20, None) == abi.MOE_ERR_UNSUPPORTED
    assert _code(s, b, b, None, 4, 8, 128, 64, 2, b, b, b, b, 0, 0, b, b, 1 << 20, None) == abi.MOE_ERR_INVALID_ARG
    assert _code(s, b, b, b, 4, 8, 128, 64, 2, b, b, b, b, 0, 0, b, b, 100, None) == abi.MOE_ERR_WORKSPACE
    assert _code(s, b, b, b, 4, 8, 128, 64, 2, b, b, b, b, 0, 0, b, P(272), 1 << 20, None) == abi.MOE_ERR_WORKSPACE
    assert abi.load().moe_last_error().decode()


def test_binding_refusals():
    v = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        abi.moe_fp8_quantize_b128(v)
    with pytest.raises(ValueError, match="v must be"):
        abi.moe_fp8_quantize_b128(v[0])
    with pytest.raises(ValueError, match="scales"):
        abi.moe_fp8_quantize_b128(v, scales=torch.zeros((4, 2)))
    c = torch.zeros((4, 64), dtype=torch.float8_e4m3fn)
    w, s1, sw = c[None], torch.zeros((4, 1)), torch.zeros((1, 1, 1))
    with pytest.raises(ValueError, match="w has K"):
        abi.moe_grouped_gemm_fp8_b128(c, s1, w[..., :32], sw)
    with pytest.raises(ValueError, match="a_scales"):
        abi.moe_grouped_gemm_fp8_b128(c, sw, w, sw)
    with pytest.raises(ValueError, match="codes"):
        abi.moe_grouped_gemm_fp8_b128(v, s1, w, sw)
    with pytest.raises(ValueError, match="expert_offsets"):
        abi.moe_grouped_gemm_fp8_b128(c, s1, w, sw, expert_offsets=torch.zeros(5, dtype=torch.int32))
    x, off = torch.zeros((4, 64), dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    gu, d = torch.zeros((1, 128, 64), dtype=torch.uint8), torch.zeros((1, 64, 64), dtype=torch.uint8)
    with pytest.raises(ValueError, match="sc_gu"):
        abi.moe_grouped_swiglu_fp8_b128(x, None, off, 4, gu, sw, d, sw)
    with pytest.raises(ValueError, match="w_gu must be"):
        abi.moe_grouped_swiglu_fp8_b128(x, None, off, 4, gu, sw, d[:, :32], sw)
