"""The FP8 grouped product on the GPU where its tiles meet: several tiles per
thread block, halves of a tile with a single box of 16-bit output columns, and
rows without a token beside weights that are not finite.  Tolerances as in test_gpu_fp8."""

import pytest
import torch

from bit_expert_gemm_b200 import abi
from bit_expert_gemm_b200.layer import prepare_fp8_weights
from oracle import fp8
from tests.test_gpu_fp8 import DEV, HALF, U, _np, _routing, _values

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_without_a_token_are_zero_beside_bad_weights(dtype):
    """Rows whose row_token is out of range are zero where the expert's weights hold
    a NaN code or an infinite scale; rows with a token show them."""
    T, K, N, E = 9, 272, 144, 2
    a, sa = abi.moe_fp8_quantize_b128(_values((T, K), 1).to(DEV), 1)
    wv = _values((E, N, K), 2, spread=0.3)
    wv[0, 3, 5], wv[0, 130, 200], wv[1, 7, 260] = float("nan"), float("inf"), float("-inf")
    w, sw = abi.moe_fp8_quantize_b128(wv.to(DEV), 128)
    row_token = torch.tensor([0, -1, 4, T, 8, -2 ** 31, 2 ** 31 - 1, 3], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    out = abi.moe_grouped_gemm_fp8_b128(a, sa, w, sw, expert_offsets=off, row_token=row_token, out_dtype=dtype)
    gone = (row_token < 0) | (row_token >= T)
    assert (out[gone] == 0).all()
    bad = torch.zeros((2, N), dtype=torch.bool, device=DEV)
    bad[0, 3] = True
    bad[0, 128:] = True  # the scale of rows 128.. and columns 128..255
    bad[1, :128] = True  # the scale of rows ..127 and columns 256..
    want = bad[[0, 0, 1, 1]]
    assert torch.equal(torch.isfinite(out[~gone]), ~want)
    assert abi.moe_device_status() == 0


def test_expert_rows_without_a_token_and_behind_the_last():
    T, H, I, E = 9, 192, 128, 2
    w = prepare_fp8_weights({"w_gate_up": _values((E, 2 * I, H), 5).to(DEV) * H ** -0.5,
                             "w_down": _values((E, H, I), 6).to(DEV) * I ** -0.5})
    args = (w["w8_gu"], w["sc8_gu"], w["w8_d"], w["sc8_d"])
    x = _values((T, H), 4).to(DEV)
    row_token = torch.tensor([0, -1, 4, T, 8, 2 ** 31 - 1, 3, 1, 1], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 4, 7], dtype=torch.int32, device=DEV)
    f = torch.full((9, H), 7.0, dtype=torch.bfloat16, device=DEV)
    abi.moe_grouped_swiglu_fp8_b128(x, row_token, off, 9, *args, f=f)
    assert (f[7:] == 7).all() and (f[[1, 3, 5]] == 0).all()
    # the other rows are those of a batch without the absent ones
    some = torch.tensor([0, 2, 4, 6], device=DEV)
    off2 = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    assert torch.equal(f[some], abi.moe_grouped_swiglu_fp8_b128(x, row_token[some].contiguous(), off2, 4, *args))
    assert abi.moe_device_status() == 0


def test_expert_rows_whatever_the_workspace_holds():
    T, H, I, E, k = 50, 256, 192, 6, 2
    w = prepare_fp8_weights({"w_gate_up": _values((E, 2 * I, H), 5).to(DEV) * H ** -0.5,
                             "w_down": _values((E, H, I), 6).to(DEV) * I ** -0.5})
    args = (w["w8_gu"], w["sc8_gu"], w["w8_d"], w["sc8_d"])
    x = _values((T, H), 4).to(DEV)
    row_token, off, _ = _routing(T, E, k, seed=3)
    want = abi.moe_grouped_swiglu_fp8_b128(x, row_token, off, T * k, *args)
    assert torch.isfinite(want).all()
    ws = abi.workspace(abi.MOE_OP_SWIGLU_FP8_B128, T, H, E, k, I, DEV)
    for fill in (0xff, 0x00, 0x7f):
        ws.fill_(fill)
        assert torch.equal(abi.moe_grouped_swiglu_fp8_b128(x, row_token, off, T * k, *args, ws=ws), want)


def test_quantiser_and_product_captured_on_a_given_stream():
    """A graph of the quantiser and the gathered product replayed with other values
    and other rows, and the same two calls on a stream that is passed."""
    T, K, N, E = 70, 272, 192, 3
    w, sw = abi.moe_fp8_quantize_b128(_values((E, N, K), 2, spread=0.3).to(DEV), 128)
    rows = [_routing(T, E, 2, seed=s)[:2] for s in (1, 2)]
    xs = [_values((T, K), 10 + s).to(DEV) for s in (1, 2)]

    def calls(x, row_token, off, codes, scales, out, stream=None):
        abi.moe_fp8_quantize_b128(x, 1, codes=codes, scales=scales, stream=stream)
        abi.moe_grouped_gemm_fp8_b128(codes, scales, w, sw, expert_offsets=off, row_token=row_token, out=out,
                                      stream=stream)

    def buffers():
        return (torch.empty((T, K), dtype=torch.float8_e4m3fn, device=DEV), torch.empty((T, 3), device=DEV),
                torch.empty((2 * T, N), dtype=torch.float16, device=DEV))

    want = []
    for x, (rt, off) in zip(xs, rows):
        b = buffers()
        calls(x, rt, off, *b)
        want.append(b[2])
    x, rt, off, b = xs[0].clone(), rows[0][0].clone(), rows[0][1].clone(), buffers()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(x, rt, off, *b)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        rt.copy_(rows[i][0])
        off.copy_(rows[i][1])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b[2], want[i])
    s, b2 = torch.cuda.Stream(), buffers()
    torch.cuda.synchronize()
    calls(xs[0], *rows[0], *b2, stream=s)
    s.synchronize()
    assert torch.equal(b2[2], want[0])
