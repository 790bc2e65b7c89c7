"""The one-kernel decode layer on the GPU against float64, element by element.

Tolerances.  16-bit products are exact in FP32 (FP16 products too: 22 bits) and
the sums are FP32, each addition rounded by at most 2^-23 of the running
magnitude.  g and u are sums of H products, h = silu(g) u is kept to 2^-15 of
its value (BF16 in two parts; FP16: 2^-20, or 2^-24 absolutely where the low
part is subnormal), f is a sum of I products, y one of k + 1 terms, rounded
once.  Weights of the selection: FP32 exponentials, a few steps of their
value.  FP8 experts: as in test_gpu_fp8.  The selection itself is compared on
tokens whose logits decide it by more than 1e-3 and must be the oracle's."""

import dataclasses

import numpy as np
import pytest
import torch

from bit_expert_gemm_b200 import MoELayer, abi, synth
from bit_expert_gemm_b200.layer import prepare_fp8_weights
from oracle import fp8, moe
from tests.helpers import f64
from tests.test_gpu_fp8 import HALF, U, _np, _swiglu_tol

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _case(T, H, I, E, k, dtype="bf16", seed=0, norm=False, gate=False, bias_std=1.0):
    wl = dataclasses.replace(synth.WORKLOADS["tiny"], H=H, I=I, I_sh=I, E=E, k=k, act=dtype, bias_std=bias_std)
    w = synth.make_weights(wl, seed=seed, device=DEV)
    for n in ("w_gate_up", "w_down"):
        w[n] = w[n].to(DT[dtype])
    if norm:
        w["w_norm"] = synth.make_norm_weight(wl, seed, DEV)
    if gate:
        w["w_sh_gate"] = synth.make_shared_gate(wl, seed, DEV)
    return w, synth.make_tokens(wl, T, seed=seed, device=DEV)


def _call(w, x, k, fmt, shared=True, **kw):
    rest = dict(w_sh_gate_up=w["w_sh_gate_up"] if shared else None, w_sh_down=w["w_sh_down"] if shared else None,
                norm_w=w.get("w_norm"), w_shared_gate=w.get("w_sh_gate"), **kw)
    if fmt == "fp8":
        return abi.moe_layer_decode_fp8_b128(x, w["w_router"], w["bias"], k, w["w8_gu"], w["sc8_gu"], w["w8_d"],
                                             w["sc8_d"], **rest)
    return abi.moe_layer_decode_bf16(x, w["w_router"], w["bias"], k, w["w_gate_up"], w["w_down"], **rest)


def _swiglu16_tol(x, wg, wu, wdn, small):
    """float64 output of a 16-bit expert and its elementwise FP32 tolerance."""
    H, I = wg.shape[1], wg.shape[0]
    g, u = x @ wg.T, x @ wu.T
    dg, du = (H + 3) * U * (np.abs(x) @ np.abs(wg).T), (H + 3) * U * (np.abs(x) @ np.abs(wu).T)
    h = moe.silu(g) * u
    dh = 1.1 * dg * np.abs(u) + (np.abs(moe.silu(g)) + 1.1 * dg) * du + (16 * U + 2.0 ** -15) * np.abs(h) + small
    ref = h @ wdn.T
    return ref, dh @ np.abs(wdn).T + (2 * I + 3) * U * ((np.abs(h) + dh) @ np.abs(wdn).T)


def _reference(w, x, k, fmt, dtype, shared=True):
    x64 = f64(x)
    if "w_norm" in w:
        x64 = moe.block_input(x64, f64(w["w_norm"]), dtype=dtype)
    bias = None if w["bias"] is None else w["bias"].double().cpu().numpy()
    r = moe.route(x64, f64(w["w_router"]), bias, k)
    small = 2.0 ** -24 if dtype == "f16" else 0.0
    T, H, I = x64.shape[0], x64.shape[1], w["w_sh_down"].shape[1]
    ref, tol = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e, wt = int(r["idx"][t, j]), r["w"][t, j]
            if fmt == "fp8":
                ew = fp8.expert_weights(*(_np(w[n][e:e + 1]) for n in ("w8_gu", "sc8_gu", "w8_d", "sc8_d")))(0)
                f, df = _swiglu_tol(x64[t:t + 1], *ew, torch.float32)
            else:
                gu = f64(w["w_gate_up"][e])
                f, df = _swiglu16_tol(x64[t:t + 1], gu[:I], gu[I:], f64(w["w_down"][e]), small)
            ref[t] += wt * f[0]
            tol[t] += wt * df[0] + 64 * U * np.abs(wt * f[0])
    if shared:
        gu = f64(w["w_sh_gate_up"])
        f, df = _swiglu16_tol(x64, gu[:I], gu[I:], f64(w["w_sh_down"]), small)
        if "w_sh_gate" in w:
            wg = f64(w["w_sh_gate"])
            s = moe.shared_gate(x64, wg)[:, None]
            df = s * df + np.abs(f) * ((H + 3) * U * (np.abs(x64) @ np.abs(wg)) + 16 * U)[:, None]
            f = s * f
        ref += f
        tol += df + 4 * U * np.abs(f)
    tol = tol + HALF[DT[dtype]] * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == "f16" else 0.0)
    return ref, tol, r


def _check(y, ref, tol, r):
    ok = r["set_margin"] > 1e-3
    assert ok.any()
    bad = np.abs(y.double().cpu().numpy() - ref)[ok] > tol[ok]
    assert not bad.any(), (int(bad.sum()), float(np.max((np.abs(y.double().cpu().numpy() - ref) / tol)[ok])))


CASES = [
    # T, H, I, E, k, dtype, norm, gate, shared
    (1, 64, 64, 1, 1, "bf16", False, False, True), (1, 2048, 640, 32, 10, "bf16", False, False, True),
    (2, 192, 128, 16, 16, "f16", True, False, True), (3, 320, 192, 33, 4, "bf16", True, True, True),
    (8, 256, 64, 1024, 2, "bf16", False, True, True), (9, 448, 320, 64, 3, "f16", False, False, False),
    (16, 2560, 128, 40, 5, "f16", True, True, True), (16, 64, 64, 2, 2, "bf16", False, False, True),
    (10, 4096, 64, 24, 3, "bf16", True, False, True), (5, 4096, 448, 8, 2, "f16", False, False, False),
    (16, 128, 1024, 300, 12, "bf16", False, False, True), (13, 1088, 192, 600, 6, "bf16", True, False, True)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H,I,E,k,dtype,norm,gate,shared", CASES)
def test_layer_against_float64(T, H, I, E, k, dtype, norm, gate, shared, fmt):
    w, x = _case(T, H, I, E, k, dtype, seed=T + H, norm=norm, gate=gate)
    if not shared:
        w.pop("w_sh_gate", None)
    if fmt == "fp8":
        w = prepare_fp8_weights(w)
    idx = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    tw = torch.zeros((T, k), device=DEV)
    y = _call(w, x, k, fmt, shared, topk_idx=idx, topk_w=tw)
    ref, tol, r = _reference(w, x, k, fmt, dtype, shared)
    _check(y, ref, tol, r)
    ok = r["margin"] > 1e-3
    assert np.array_equal(_np(idx)[ok], r["idx"][ok])
    # weights: exponentials of FP32 logits (half a step of |l|), a few steps of their own
    lim = (2.0 ** -23 * (np.abs(r["logits"]).max(1) + 16))[:, None] * 2 * r["w"]
    assert np.all(np.abs(_np(tw) - r["w"])[ok] <= lim[ok])
    again = _call(w, x, k, fmt, shared)
    assert torch.equal(again, y)  # the same order of sums every time
    assert abi.moe_device_status() == 0


def test_ties_go_to_the_lower_index_and_all_equal_logits():
    T, H, I, E, k = 4, 128, 64, 200, 7
    w, x = _case(T, H, I, E, k)
    w["w_router"].zero_()
    w["bias"] = torch.zeros(E, device=DEV)
    idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
    _call(w, x, k, "bf16", topk_idx=idx)
    assert torch.equal(idx.cpu(), torch.arange(k, dtype=torch.int32).expand(T, k))
    w["bias"][torch.tensor([150, 3, 77])] = 1.0
    _call(w, x, k, "bf16", topk_idx=idx)
    assert idx[0].tolist() == [3, 77, 150, 0, 1, 2, 4]


def test_masked_experts_and_bad_values():
    """Experts masked by a bias of -inf or of the lowest FP32 number are taken
    last and weigh nothing; NaN logits rank last; weights that are NaN or
    infinite reach only the tokens that select them."""
    T, H, I, E, k = 6, 192, 64, 24, 3
    w, x = _case(T, H, I, E, k, seed=3)
    free = [2, 9, 20]
    bias = torch.full((E,), float("-inf"), device=DEV)
    bias[1::2] = torch.finfo(torch.float32).min
    bias[free] = 0.0
    w["bias"] = bias
    idx, tw = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    y = _call(w, x, k, "bf16", topk_idx=idx, topk_w=tw)
    assert torch.equal(idx.sort(1).values.cpu(), torch.tensor(free, dtype=torch.int32).expand(T, k))
    ref, tol, r = _reference(w, x, k, "bf16", "bf16")
    _check(y, ref, tol, r)
    bias[free[0]] = float("nan")
    _call(w, x, 2, "bf16", topk_idx=idx[:, :2].contiguous(), topk_w=tw[:, :2].contiguous())
    w2, x2 = _case(T, H, I, E, k, seed=4)
    clean = _call(w2, x2, k, "bf16", topk_idx=idx, topk_w=tw)
    e = int(idx[0, 0])
    w2["w_down"][e], w2["w_gate_up"][e, :3] = float("nan"), float("inf")
    y2 = _call(w2, x2, k, "bf16")
    hit = (idx == e).any(1)
    assert hit.any() and torch.isnan(y2[hit]).all() and torch.equal(y2[~hit], clean[~hit])


def test_a_bad_token_spoils_only_itself():
    for fmt in ("bf16", "fp8"):
        w, x = _case(9, 256, 128, 16, 3, seed=6, norm=True)
        w = prepare_fp8_weights(w)
        clean = _call(w, x, 3, fmt)
        x[4, 17] = float("nan")
        y = _call(w, x, 3, fmt)
        keep = torch.arange(9, device=DEV) != 4
        assert torch.isnan(y[4]).all() and torch.equal(y[keep], clean[keep])


def test_all_tokens_on_the_same_experts():
    """16 tokens on 2 experts: more tokens than one 8-column operand per expert."""
    for fmt in ("bf16", "fp8"):
        w, x = _case(16, 512, 192, 8, 2, seed=8)
        w = prepare_fp8_weights(w)
        w["bias"] = torch.zeros(8, device=DEV)
        w["bias"][[1, 6]] = 50.0
        y = _call(w, x, 2, fmt)
        _check(y, *_reference(w, x, 2, fmt, "bf16"))


def test_without_bias_and_zero_tokens():
    w, x = _case(3, 128, 64, 12, 2, seed=5)
    w["bias"] = None
    _check(_call(w, x, 2, "bf16"), *_reference(w, x, 2, "bf16", "bf16"))
    assert _call(w, x[:0], 2, "bf16").shape == (0, 128)


def test_two_streams_graphs_and_a_shared_workspace():
    """Calls on two streams at once (own workspaces), two graphs that share one
    workspace and run one after the other, other weights between them."""
    cases = []
    for s in (0, 1):
        w, x = _case(4 + s, 512, 192, 40, 4, seed=20 + s, norm=True)
        cases.append((prepare_fp8_weights(w), x))
    want = [_call(w, x, 4, fmt) for w, x in cases for fmt in ("bf16", "fp8")]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(6):
        for (w, x), st in zip(cases, streams):
            with torch.cuda.stream(st):
                got += [_call(w, x, 4, fmt) for fmt in ("bf16", "fp8")]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 4]) for i, g in enumerate(got))
    ws = abi.workspace(abi.MOE_OP_LAYER_DECODE, 5, 512, 40, 4, 192, DEV)
    graphs, outs = [], []
    for w, x in cases:
        y = torch.empty_like(x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _call(w, x, 4, "fp8", y=y, ws=ws)
        graphs.append(g)
        outs.append(y)
    for i in (0, 1, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[2 * i + 1])


@pytest.mark.parametrize("fmt", ["bf16", "fp8_b128"])
def test_moe_layer_uses_it(fmt):
    """MoELayer.forward on a decode batch: the one-kernel layer, alone, captured,
    through HostPipeline, and next to the chain of calls for larger batches."""
    from bit_expert_gemm_b200.layer import HostPipeline

    k = 3
    w, x = _case(8, 256, 192, 16, k, seed=12, norm=True, gate=True)
    layer = MoELayer(w, k, fmt=fmt, T_max=40, fused_decode=True)
    kind = "fp8" if fmt == "fp8_b128" else "bf16"
    y = layer.forward(x).clone()
    assert torch.equal(y, _call(layer.w, x, k, kind))
    _check(y, *_reference(layer.w, x, k, kind, "bf16"))
    g = layer.capture(x)
    assert layer.graph_kernels == 1
    layer.y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.y[:8], y)
    pipe = HostPipeline(layer, 8)
    xh, yh = x.cpu().pin_memory(), torch.empty(x.shape, dtype=x.dtype).pin_memory()
    pipe.step(xh, yh)
    pipe.finish()
    torch.cuda.synchronize()
    assert torch.equal(yh, y.cpu())
    # a larger batch takes the chain of calls; both agree to 16-bit roundings of f and the shared expert
    big = x.repeat(5, 1)
    yb = layer.forward(big)
    assert (yb[:8].float() - y.float()).abs().max() <= 2e-2 * y.float().abs().max()
    if fmt == "bf16":
        assert not MoELayer(w, k, fmt=fmt, T_max=8).decode_ws  # the default keeps its path


def test_norm_of_large_and_zero_tokens():
    """Squares beyond FP32's range, and a token of zeros (eps alone)."""
    w, x = _case(3, 256, 64, 12, 2, seed=9, norm=True)
    x[1] *= 1e30
    x[2] = 0
    y = _call(w, x, 2, "bf16")
    ref, tol, r = _reference(w, x, 2, "bf16", "bf16")
    assert torch.isfinite(y).all()
    _check(y, ref, tol, r)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H,I,E,k,dtype,norm,gate,shared", [
    (1, 128, 8192, 2, 2, "bf16", False, False, True), (16, 64, 8192, 3, 1, "f16", True, False, True),
    (16, 64, 64, 1024, 16, "bf16", False, True, True), (4, 4096, 2048, 6, 3, "f16", False, True, True),
    (8, 4096, 1024, 9, 8, "bf16", True, False, False)])
def test_layer_at_its_limits(T, H, I, E, k, dtype, norm, gate, shared, fmt):
    test_layer_against_float64(T, H, I, E, k, dtype, norm, gate, shared, fmt)
