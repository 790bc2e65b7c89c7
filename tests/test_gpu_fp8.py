"""FP8 E4M3 with a scale per block of 128 on the GPU: the quantiser bit for bit,
the grouped product and the expert FFN against float64 element by element,
and the layer built of them.

Tolerances.  A product of two E4M3 values is exact in FP32 and the sums are
FP32: with at most K additions and a scale product per block, each rounded by
at most 2^-23 of the running magnitude, an output is within
(K + 3 ceil(K/128) + 3) 2^-23 of the sum of the terms' magnitudes, plus half
a step of its own type.  Where h is quantised again, a value whose FP32 error
crosses a rounding border moves by one E4M3 step: each element may move by the
difference of the codes of h - u and h + u (u: its error bound), which the
down projection carries into the output."""

import dataclasses

import numpy as np
import pytest
import torch

from bit_expert_gemm_b200 import MoELayer, abi, synth
from bit_expert_gemm_b200.layer import prepare_fp8_weights, slice_layer_weights
from oracle import fp8, moe
from oracle.formats import e4m3_to_f64, f32_to_e4m3
from tests.helpers import f64, rel_err, shared_fn

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -23
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def _np(t):
    t = t.detach().cpu()
    return (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).numpy()


def _values(shape, seed, dtype=torch.bfloat16, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp(spread * torch.randn((*shape[:-1], 1), generator=g))).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,R,K,br", [(1, 1, 16, 1), (1, 1, 128, 1), (1, 37, 272, 1), (3, 5, 2048, 1), (1, 4099, 144, 1),
                                      (1, 1, 16, 128), (2, 130, 272, 128), (3, 257, 128, 128), (1, 128, 640, 128)])
def test_quantise_bit_exact(B, R, K, br, dtype):
    v = _values((B, R, K), B * 100 + K, dtype)
    v[0, 0, :16] = 0
    if K > 144:
        v[0, 0, :128] = 0          # a block of zeros (block_rows = 1)
        v[0, -1, 128:256] = 1e-7   # tiny values: FP16 subnormals
    codes, scales = abi.moe_fp8_quantize_b128(v.to(DEV), br)
    for b in range(B):
        c, s = fp8.quantize(f64(v[b]), br)
        assert np.array_equal(_np(codes[b]), c) and np.array_equal(_np(scales[b]), s)
    if B == 1:  # the same through the two-dimensional call
        c2, s2 = abi.moe_fp8_quantize_b128(v[0].to(DEV), br)
        assert torch.equal(c2.view(torch.uint8), codes[0].view(torch.uint8)) and torch.equal(s2, scales[0])


def test_quantise_inf_nan_and_extremes():
    v = _values((6, 256), 3)
    v[0, 5] = float("inf")
    v[1, 7] = float("nan")
    v[2, :128] = torch.finfo(torch.bfloat16).min  # the type's lowest value
    v[3, :128] = 2.0 ** -120                      # below the floor of the block maximum
    codes, scales = abi.moe_fp8_quantize_b128(v.to(DEV), 1)
    val = codes.float().cpu().double() * scales.cpu().double().repeat_interleave(128, 1)
    assert torch.isnan(val[0, :128]).all() and torch.isfinite(val[0, 128:]).all()
    assert torch.isnan(val[1, 7]) and torch.isfinite(val[1]).sum() == 255
    assert torch.equal(codes[2, :128].float().cpu(), torch.full((128,), -448.0))
    assert not codes[3, :128].float().any() and torch.isfinite(val[2:]).all()


def _routing(T, E, k, seed):
    idx = synth.make_routing(T, E, k, seed=seed)
    p = moe.permute(idx.numpy(), E)
    return (torch.from_numpy(p["row_token"].astype(np.int32)).to(DEV),
            torch.from_numpy(p["offsets"].astype(np.int32)).to(DEV), p)


def _bank(E, N, K, seed):
    c, s = abi.moe_fp8_quantize_b128(_values((E, N, K), seed, spread=0.3).to(DEV), 128)
    return c, s, np.stack([fp8.dequant(_np(c[e]), _np(s[e]), 128) for e in range(E)])


def _check(got, ref, mag, K, dtype):
    tol = (K + 3 * (-(-K // 128)) + 3) * U * mag
    tol = tol + HALF[dtype] * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(got - ref) / tol)))


@pytest.mark.parametrize("T,K,N,E,k,gather,dtype", [
    (1, 16, 16, 1, 1, False, torch.float32), (5, 128, 128, 1, 1, False, torch.float32),
    (129, 272, 144, 1, 1, False, torch.bfloat16), (300, 640, 2048, 1, 1, False, torch.float16),
    (37, 592, 336, 16, 2, True, torch.float32), (37, 592, 336, 16, 2, False, torch.bfloat16),
    (1, 2048, 256, 8, 3, True, torch.float16), (700, 144, 272, 5, 2, True, torch.float32),
    (2500, 256, 768, 3, 1, True, torch.bfloat16), (64, 2560, 48, 64, 4, True, torch.float32)])
def test_grouped_gemm(T, K, N, E, k, gather, dtype):
    row_token, off, p = _routing(T, E, k, seed=T + K)
    rows = T * k
    a, sa = abi.moe_fp8_quantize_b128(_values((T if gather else rows, K), T + N).to(DEV), 1)
    w, sw, wd = _bank(E, N, K, seed=N)
    out = abi.moe_grouped_gemm_fp8_b128(a, sa, w, sw, expert_offsets=off, row_token=row_token if gather else None,
                                        out_dtype=dtype)
    ad = fp8.dequant(_np(a), _np(sa))
    ad = ad[p["row_token"]] if gather else ad
    got = out.double().cpu().numpy()
    for e in range(E):
        lo, hi = p["offsets"][e], p["offsets"][e + 1]
        _check(got[lo:hi], ad[lo:hi] @ wd[e].T, np.abs(ad[lo:hi]) @ np.abs(wd[e]).T, K, dtype)
    if E == 1 and not gather:  # without offsets: one group of all rows
        again = abi.moe_grouped_gemm_fp8_b128(a, sa, w, sw, out_dtype=dtype)
        assert torch.equal(again, out)
    assert abi.moe_device_status() == 0


def test_grouped_gemm_leaves_other_rows_and_zeroes_bad_tokens():
    T, K, N, E = 9, 144, 80, 3
    a, sa = abi.moe_fp8_quantize_b128(_values((T, K), 1).to(DEV), 1)
    w, sw, wd = _bank(E, N, K, seed=2)
    # 12 rows are given, the groups end at 10; expert 1 is empty; rows 2 and 5 have no token
    row_token = torch.tensor([0, 1, -1, 8, 8, T, 3, 3, 4, 2, 7, 7], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 4, 4, 10], dtype=torch.int32, device=DEV)
    out = torch.full((12, N), 7.0, device=DEV)
    abi.moe_grouped_gemm_fp8_b128(a, sa, w, sw, expert_offsets=off, row_token=row_token, out=out)
    ad, got, rt = fp8.dequant(_np(a), _np(sa)), out.double().cpu().numpy(), row_token.cpu().numpy()
    assert (got[10:] == 7).all() and (got[[2, 5]] == 0).all()
    for r in [0, 1, 3, 4, 6, 7, 8, 9]:
        e = 0 if r < 4 else 2
        _check(got[r:r + 1], ad[rt[r]:rt[r] + 1] @ wd[e].T, np.abs(ad[rt[r]:rt[r] + 1]) @ np.abs(wd[e]).T, K,
               torch.float32)


def _swiglu_tol(x, wg, wu, wdn, dtype):
    """float64 reference and elementwise tolerance of one expert (module docstring)."""
    K, I = wg.shape[1], wg.shape[0]
    xq = fp8.dequant(*fp8.quantize(x))
    n1 = (K + 3 * (-(-K // 128)) + 3) * U
    g, u = xq @ wg.T, xq @ wu.T
    dg, du = n1 * (np.abs(xq) @ np.abs(wg).T), n1 * (np.abs(xq) @ np.abs(wu).T)
    h = moe.silu(g) * u
    # |silu'| <= 1.1; the FP32 exponential, division and product: a few steps of the value
    dh = 1.1 * dg * np.abs(u) + (np.abs(moe.silu(g)) + 1.1 * dg) * du + 16 * U * np.abs(h)
    codes, s = fp8.quantize(h)
    hq = fp8.dequant(codes, s)
    blk = np.arange(I) // 128
    amax = np.maximum(s.astype(np.float64) * 448, 2.0 ** -80)[:, blk]
    rel = np.zeros_like(h)
    for b in range(s.shape[1]):
        rel[:, blk == b] = np.max(dh[:, blk == b], axis=1, keepdims=True)
    rel = rel / amax + 4 * U          # the block maximum, and with it the scale
    v = h * 448 / amax
    w = (dh + np.abs(h) * rel) * 448 / amax
    step = e4m3_to_f64(f32_to_e4m3(np.clip(v + w, -448, 448))) - e4m3_to_f64(f32_to_e4m3(np.clip(v - w, -448, 448)))
    dq = step * amax / 448 + np.abs(hq) * rel
    ref = hq @ wdn.T
    n2 = (I + 3 * (-(-I // 128)) + 3) * U
    tol = dq @ np.abs(wdn).T + n2 * ((np.abs(hq) + dq) @ np.abs(wdn).T)
    return ref, tol + HALF[dtype] * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


@pytest.mark.parametrize("T,H,I,E,k,dtype,fp32", [
    (1, 64, 64, 1, 1, torch.bfloat16, False), (1, 2048, 640, 16, 4, torch.bfloat16, False),
    (33, 320, 192, 16, 2, torch.float16, False), (200, 192, 320, 4, 3, torch.bfloat16, True),
    (130, 128, 128, 2, 1, torch.float16, True), (520, 448, 448, 3, 2, torch.bfloat16, False)])
def test_grouped_swiglu(T, H, I, E, k, dtype, fp32):
    row_token, off, p = _routing(T, E, k, seed=I + T)
    x = _values((T, H), T, dtype, spread=0.5)
    gu, sc_gu = abi.moe_fp8_quantize_b128(_values((2 * E, I, H), H, spread=0.2).to(DEV) * H ** -0.5, 128)
    d, sc_d = abi.moe_fp8_quantize_b128(_values((E, H, I), H + 1, spread=0.2).to(DEV) * I ** -0.5, 128)
    gu, sc_gu = gu.view(E, 2 * I, H), sc_gu.view(E, 2, *sc_gu.shape[1:])
    f = abi.moe_grouped_swiglu_fp8_b128(x.to(DEV), row_token, off, T * k, gu, sc_gu, d, sc_d, out_fp32=fp32)
    ew = fp8.expert_weights(_np(gu), _np(sc_gu), _np(d), _np(sc_d))
    got, x64 = f.double().cpu().numpy(), f64(x)
    for e in range(E):
        lo, hi = p["offsets"][e], p["offsets"][e + 1]
        if lo == hi:
            continue
        ref, tol = _swiglu_tol(x64[p["row_token"][lo:hi]], *ew(e), torch.float32 if fp32 else dtype)
        bad = np.abs(got[lo:hi] - ref) > tol
        assert not bad.any(), (e, int(bad.sum()), float(np.max(np.abs(got[lo:hi] - ref) / tol)))
    if E == 1:  # a dense expert: rows in order
        again = abi.moe_grouped_swiglu_fp8_b128(x.to(DEV), None, off, T, gu, sc_gu, d, sc_d, out_fp32=fp32)
        assert torch.equal(again, f)
    assert abi.moe_device_status() == 0


def test_a_bad_token_spoils_only_its_own_rows():
    T, H, I, E, k = 40, 256, 128, 4, 2
    row_token, off, _ = _routing(T, E, k, seed=9)
    x = _values((T, H), 4).to(DEV)
    w = prepare_fp8_weights({"w_gate_up": _values((E, 2 * I, H), 5).to(DEV) * H ** -0.5,
                             "w_down": _values((E, H, I), 6).to(DEV) * I ** -0.5})
    args = (w["w8_gu"], w["sc8_gu"], w["w8_d"], w["sc8_d"])
    clean = abi.moe_grouped_swiglu_fp8_b128(x, row_token, off, T * k, *args)
    x[7, 3], x[20, 200] = float("inf"), float("nan")
    f = abi.moe_grouped_swiglu_fp8_b128(x, row_token, off, T * k, *args)
    hit = (row_token == 7) | (row_token == 20)
    assert torch.isnan(f[hit]).all() and torch.equal(f[~hit], clean[~hit])


def test_two_streams_and_a_graph_give_the_same_rows():
    T, H, I, E, k = 70, 512, 192, 8, 3
    row_token, off, _ = _routing(T, E, k, seed=11)
    xs = [_values((T, H), 20 + i).to(DEV) for i in range(2)]
    w = prepare_fp8_weights({"w_gate_up": _values((E, 2 * I, H), 5).to(DEV) * H ** -0.5,
                             "w_down": _values((E, H, I), 6).to(DEV) * I ** -0.5})

    def call(x, ws=None, f=None):
        return abi.moe_grouped_swiglu_fp8_b128(x, row_token, off, T * k, w["w8_gu"], w["sc8_gu"], w["w8_d"],
                                               w["sc8_d"], ws=ws, f=f)

    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(call(x))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))
    x, f = xs[0].clone(), torch.empty_like(want[0])
    ws = abi.workspace(abi.MOE_OP_SWIGLU_FP8_B128, T, H, E, k, I, DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, ws, f)
    for i in (0, 1, 0):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(f, want[i])


def _layer_case(T, dtype="bf16", norm=False, gate=False, E=16, k=4, H=256, I=192, seed=0):
    wl = dataclasses.replace(synth.WORKLOADS["tiny"], H=H, I=I, I_sh=I, E=E, k=k, act=dtype)
    w = synth.make_weights(wl, seed=seed, device=DEV)
    if norm:
        w["w_norm"] = synth.make_norm_weight(wl, seed, DEV)
    if gate:
        w["w_sh_gate"] = synth.make_shared_gate(wl, seed, DEV)
    return wl, w, synth.make_tokens(wl, T, seed=seed, device=DEV)


def _layer_ref(w, x, k, norm=False, gate=False, dtype="bf16"):
    x64 = f64(x)
    if norm:
        x64 = moe.block_input(x64, f64(w["w_norm"]), dtype=dtype)
    r = moe.route(x64, f64(w["w_router"]), w["bias"].double().cpu().numpy(), k)
    p = moe.permute(r["idx"], w["w_router"].shape[0])
    ew = fp8.expert_weights(*(_np(w[n]) for n in ("w8_gu", "sc8_gu", "w8_d", "sc8_d")))
    f = np.zeros((x64.shape[0] * k, x64.shape[1]))
    for e in range(len(p["offsets"]) - 1):
        lo, hi = p["offsets"][e], p["offsets"][e + 1]
        if hi > lo:
            f[lo:hi] = fp8.swiglu_expert(x64[p["row_token"][lo:hi]], *ew(e))[0]
    sh = moe.swiglu_expert(x64, *shared_fn(w))[0]
    if gate:
        sh = sh * moe.shared_gate(x64, f64(w["w_sh_gate"]))[:, None]
    return moe.combine(f, p["slot_row"], r["w"], sh), r


@pytest.mark.parametrize("T,dtype,norm,gate", [(300, "bf16", False, False), (40, "f16", True, True)])
def test_layer_of_fp8_experts(T, dtype, norm, gate):
    """Routing, FP8 experts, shared expert and combine together, against the
    oracle's layer on the library's own codes (which the first test pins).
    16-bit roundings of f, the shared expert and y: 2e-2 normwise, the bound
    of the 16-bit paths."""
    wl, w, x = _layer_case(T, dtype, norm, gate)
    layer = MoELayer(w, wl.k, fmt="fp8_b128", T_max=T)
    y = layer.forward(x).double().cpu().numpy()
    ref, r = _layer_ref(layer.w, x, wl.k, norm, gate, dtype)
    ok = r["margin"] > 1e-3
    assert ok.mean() > 0.8 and rel_err(y[ok], ref[ok]) <= 2e-2
    g = layer.capture(x)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(layer.y[:T].double().cpu().numpy(), y)


def test_refill_and_slice_of_an_fp8_layer():
    wl, w, x = _layer_case(200, k=3)
    scorer = MoELayer(w, wl.k, fmt="fp8_b128", T_max=200, extra=1)
    s, c = torch.zeros(wl.E, dtype=torch.float64, device=DEV), torch.zeros(wl.E, dtype=torch.int64, device=DEV)
    scorer.refill_pass(x, s, c)
    assert int(c.sum()) == 200 * wl.k and bool((s[c > 0] > 0).all())
    kept, _, _ = abi.razor_select(s, c, 8)
    small = slice_layer_weights(scorer.w, kept)
    ids = kept.long()
    for n in ("w8_gu", "w8_d"):
        assert torch.equal(small[n].view(torch.uint8), scorer.w[n].view(torch.uint8)[ids])
    for n in ("sc8_gu", "sc8_d"):
        assert torch.equal(small[n], scorer.w[n][ids])
    y = MoELayer(small, wl.k, fmt="fp8_b128", T_max=200).forward(x)
    ref, r = _layer_ref(small, x, wl.k)
    ok = r["margin"] > 1e-3
    assert rel_err(y.double().cpu().numpy()[ok], ref[ok]) <= 2e-2


def test_offsets_past_the_rows_are_cut():
    T, K, N, E = 5, 128, 64, 2
    a, sa = abi.moe_fp8_quantize_b128(_values((T, K), 31).to(DEV), 1)
    w, sw, wd = _bank(E, N, K, seed=3)
    buf = torch.full((T + 300, N), 3.0, device=DEV)
    off = torch.tensor([0, 2, 400], dtype=torch.int32, device=DEV)
    abi.moe_grouped_gemm_fp8_b128(a, sa, w, sw, expert_offsets=off, out=buf[:T])
    ad, got = fp8.dequant(_np(a), _np(sa)), buf.double().cpu().numpy()
    assert (got[T:] == 3).all()
    for lo, hi, e in ((0, 2, 0), (2, 5, 1)):
        _check(got[lo:hi], ad[lo:hi] @ wd[e].T, np.abs(ad[lo:hi]) @ np.abs(wd[e]).T, K, torch.float32)


def test_calls_in_a_row_on_one_workspace():
    """Back-to-back FFN calls on the same workspace and stream (the kernels overlap
    their prologues), each read by the next: every result is the first one's."""
    T, H, I, E, k = 300, 256, 256, 6, 2
    row_token, off, _ = _routing(T, E, k, seed=41)
    w = prepare_fp8_weights({"w_gate_up": _values((E, 2 * I, H), 5).to(DEV) * H ** -0.5,
                             "w_down": _values((E, H, I), 6).to(DEV) * I ** -0.5})
    args = (w["w8_gu"], w["sc8_gu"], w["w8_d"], w["sc8_d"])
    ws = abi.workspace(abi.MOE_OP_SWIGLU_FP8_B128, T, H, E, k, I, DEV)
    xs = [_values((T, H), 50 + i).to(DEV) for i in range(3)]
    want = [abi.moe_grouped_swiglu_fp8_b128(x, row_token, off, T * k, *args) for x in xs]
    torch.cuda.synchronize()
    got = [abi.moe_grouped_swiglu_fp8_b128(xs[i % 3], row_token, off, T * k, *args, ws=ws) for i in range(30)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 3]) for i, g in enumerate(got))


def test_1024_groups_most_of_them_empty():
    T, K, N, E = 200, 144, 80, 1024
    w, sw, wd = _bank(E, N, K, seed=5)
    a, sa = abi.moe_fp8_quantize_b128(_values((T, K), 6).to(DEV), 1)
    last = np.sort(np.random.default_rng(7).choice(E, 40, replace=False))
    off = np.searchsorted(last, np.arange(E + 1)) * 5  # five rows for each of the forty
    assert off[0] == 0 and off[-1] == T and (np.diff(off) > 0).sum() == 40
    out = abi.moe_grouped_gemm_fp8_b128(a, sa, w, sw, expert_offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
    ad, got = fp8.dequant(_np(a), _np(sa)), out.double().cpu().numpy()
    for e in last:
        lo, hi = off[e], off[e + 1]
        _check(got[lo:hi], ad[lo:hi] @ wd[e].T, np.abs(ad[lo:hi]) @ np.abs(wd[e]).T, K, out.dtype)


def test_more_than_2_to_the_31_elements():
    """Each row is computed from its own values only, so the rows at the end of a long
    tensor equal the same rows in a short one."""
    rows, K = (1 << 20) + 77, 2064
    tail = _values((300, K), 8).to(DEV)
    v = torch.zeros((rows, K), dtype=torch.bfloat16, device=DEV)
    v[-300:] = tail
    codes, scales = abi.moe_fp8_quantize_b128(v, 1)
    want = abi.moe_fp8_quantize_b128(tail, 1)
    assert torch.equal(codes[-300:].view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(scales[-300:], want[1])
    assert not codes[:-300].view(torch.uint8).any()
    del v, scales
    w, sw, _ = _bank(1, 2064, 32, seed=9)
    a = codes.view(torch.uint8)[:, :32].contiguous()
    sa = torch.ones((rows, 1), device=DEV)
    a[-300:] = want[0].view(torch.uint8)[:, :32]
    for dtype in (torch.bfloat16, torch.float32):
        small = abi.moe_grouped_gemm_fp8_b128(a[-300:].contiguous(), sa[:300], w, sw, out_dtype=dtype)
        big = abi.moe_grouped_gemm_fp8_b128(a, sa, w, sw, out_dtype=dtype)
        assert torch.equal(big[-300:], small) and small.any() and not big[:-300].any()
        del big
