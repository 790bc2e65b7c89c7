"""FP8 E4M3 with one FP32 scale per block of 128: quantisation, dequantisation
and the expert FFN on it.

Test infrastructure (see the package docstring).  The pages describe no FP8
experts; the format is the block-scaled 8-bit checkpoint format (a scale per
128 x 128 weight block, and per token and 128 input features for the
activations).  Per block, every step one float32 IEEE operation, the
precision the kernel uses, so that codes compare bit for bit:

  a = max(amax(|block|), 2^-80),  s = a / 448,  r = 448 / a
  c = e4m3_rn_sat(v * r),         v' = e4m3(c) * s
"""

from __future__ import annotations

import numpy as np

from .formats import e4m3_to_f64, f32_to_e4m3
from .moe import silu

BLOCK = 128
FLOOR = np.float32(2.0 ** -80)


def _n(v: int, b: int) -> int:
    return -(-v // b)


def quantize(v: np.ndarray, block_rows: int = 1):
    """v [rows, K] finite values -> (codes [rows, K] uint8, scales
    [ceil(rows/block_rows), ceil(K/128)] float32)."""
    v = np.asarray(v, np.float32)
    R, K = v.shape
    codes = np.empty((R, K), np.uint8)
    scales = np.empty((_n(R, block_rows), _n(K, BLOCK)), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            sl = np.s_[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            a = np.maximum(np.max(np.abs(v[sl])), FLOOR)
            scales[i, j] = np.float32(a / np.float32(448))
            codes[sl] = f32_to_e4m3(v[sl] * np.float32(np.float32(448) / a))
    return codes, scales


def dequant(codes: np.ndarray, scales: np.ndarray, block_rows: int = 1) -> np.ndarray:
    """v' = e4m3(c) * s, float64 [rows, K]."""
    R, K = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), block_rows, 0)[:R], BLOCK, 1)[:, :K]
    return e4m3_to_f64(codes) * s


def swiglu_expert(x: np.ndarray, w_gate: np.ndarray, w_up: np.ndarray, w_down: np.ndarray):
    """One expert on already dequantised weights: x [n, H] is quantised per
    row and 128 features, h likewise from its float32 value.  -> (f, h before
    its quantisation)."""
    xq = dequant(*quantize(x))
    h = silu(xq @ w_gate.T) * (xq @ w_up.T)
    return dequant(*quantize(h)) @ w_down.T, h


def expert_weights(w_gu, sc_gu, w_d, sc_d):
    """e -> float64 (w_gate, w_up, w_down) of an FP8 bank given as code and
    scale arrays (w_gu [E, 2I, H], sc_gu [E, 2, I/128, H/128], ...)."""
    I = w_gu.shape[1] // 2

    def ew(e):
        return (dequant(w_gu[e, :I], sc_gu[e, 0], BLOCK), dequant(w_gu[e, I:], sc_gu[e, 1], BLOCK),
                dequant(w_d[e], sc_d[e], BLOCK))

    return ew
