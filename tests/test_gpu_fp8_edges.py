"""The FP8 grouped product on the GPU where its tiles meet: several tiles per
thread block, halves of a tile with a single box of 16-bit output columns.
Tolerances as in test_gpu_fp8."""

import pytest
import torch

from bit_expert_gemm_b200 import abi
from oracle import fp8
from tests.test_gpu_fp8 import DEV, HALF, U, _np, _values

pytestmark = pytest.mark.gpu


def _decoded(codes, scales, block_rows):
    return torch.from_numpy(fp8.dequant(_np(codes), _np(scales), block_rows)).to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,N,K", [
    # 128-wide tiles (their bound of 21 x 7 wide tiles does not fill the SMs), 280 of them
    (2560, 1792, 16), (2560, 1792, 128), (2531, 1792, 144),
    # 256-wide tiles whose last one has 64 columns, or 64 in its second half
    (25600, 320, 16), (25600, 320, 128), (19000, 448, 128)])
def test_several_tiles_per_block(rows, N, K, dtype):
    """A warp stages its 16-bit output in two boxes that are copied out while it goes
    on: the next tile's must not take the box that is still being read."""
    w, sw = abi.moe_fp8_quantize_b128(_values((1, N, K), N, spread=0.3).to(DEV), 128)
    wd = _decoded(w[0], sw[0], 128)
    xs = [abi.moe_fp8_quantize_b128(_values((rows, K), seed).to(DEV), 1) for seed in (1, 2)]
    outs = [abi.moe_grouped_gemm_fp8_b128(a, sa, w, sw, out_dtype=dtype) for a, sa in xs for _ in range(3)]
    for i, (a, sa) in enumerate(xs):
        ad = _decoded(a, sa, 1)
        ref, mag = ad @ wd.t(), ad.abs() @ wd.abs().t()
        tol = (K + 3 * (-(-K // 128)) + 3) * U * mag
        tol = tol + HALF[dtype] * (ref.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
        assert ref.abs().min(1).values.max() > 0  # rows of zeros would hide a swap
        for out in outs[3 * i:3 * i + 3]:
            bad = (out.double() - ref).abs() > tol
            assert not bad.any(), int(bad.sum())
    assert abi.moe_device_status() == 0
