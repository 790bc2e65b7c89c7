"""The one-kernel decode layer on the GPU at the edges of what its calls allow.
Tolerances as in test_gpu_layer_decode and test_gpu_fp8."""

import numpy as np
import pytest
import torch

from bit_expert_gemm_b200 import MoELayer, abi
from bit_expert_gemm_b200.layer import prepare_fp8_weights
from oracle import moe
from tests.helpers import f64, rel_err
from tests.test_gpu_fp8 import HALF, U, _layer_case, _layer_ref
from tests.test_gpu_layer_decode import DEV, _call, _case, _check, _reference

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


def test_norm_of_tiny_and_huge_tokens_without_eps():
    """eps = 0 is allowed: tokens whose squares, or whose reciprocal norm, leave
    FP32's range are normalised from FP64 all the same.  x_norm is pinned bit for
    bit: the layer on it, without its norm, gives the same y."""
    H, k = 512, 3
    w, x = _case(8, H, 64, 24, k, seed=41, norm=True)
    scale = [1.0, 2.0 ** -70, 2.0 ** -100, 2.0 ** -129, 2.0 ** 60, 2.0 ** 126, 2.0 ** -63, 1.0]
    x = (x.double().clamp(-3.9, 3.9) * torch.tensor(scale, device=DEV, dtype=torch.float64)[:, None]).to(x.dtype)
    x[6, ::2] = 0
    x[7, 3:] *= 2.0 ** -90  # three features set the norm, the others all but vanish
    xn = torch.from_numpy(moe.block_input(f64(x), f64(w["w_norm"]), eps=0.0)).to(x.dtype).to(DEV)
    assert torch.isfinite(xn).all() and (xn != 0).any(1).all()
    for fmt in ("bf16", "fp8"):
        w = prepare_fp8_weights(w)
        plain = {n: v for n, v in w.items() if n != "w_norm"}
        assert torch.equal(_call(w, x, k, fmt, eps=0.0), _call(plain, xn, k, fmt))


@pytest.mark.parametrize("E", [24, 200, 900])
def test_selection_among_nan_and_masked_logits(E):
    """A NaN logit counts as the lowest finite number, as in moe_route_topk: behind
    every finite logit above it, tied by index with that mask, before -inf.  With
    the many ties of E = 200 and 900 the selection goes by rounds."""
    T, H, I, low = 5, 192, 64, torch.finfo(torch.float32).min
    w, x = _case(T, H, I, E, 2, seed=E)
    bias = torch.full((E,), float("-inf"), device=DEV)
    bias[[4, 17]] = 0.0
    bias[9] = float("nan")
    bias[[7, 20]] = low
    if E > 24:
        bias[24:] = low
    w["bias"] = bias
    want = {2: [4, 17], 3: [4, 17, 7], 4: [4, 17, 7, 9], 5: [4, 17, 7, 9, 20]}
    if E == 24:  # two more than are left: the first of the -inf ones
        want[7] = [4, 17, 7, 9, 20, 0, 1]
    for k, order in want.items():
        idx, tw = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
        y = _call(w, x, k, "bf16", topk_idx=idx, topk_w=tw)
        ridx, rw, _ = abi.moe_route_topk(x, w["w_router"], bias, k)
        assert torch.equal(idx, ridx)
        assert (idx[:, :2].sort(1).values == torch.tensor([4, 17], device=DEV)).all()
        assert (idx[:, 2:].cpu() == torch.tensor(order[2:], dtype=torch.int32)).all()
        assert (tw[:, 2:] == 0).all() and (tw[:, :2].sum(1) - 1).abs().max() <= 2.0 ** -21
        # the chain's logits: H FP32 additions, each off by 2^-24 of sum |x w| <= 16; half of that in a weight of two
        assert (tw - rw).abs().max() <= H * 2.0 ** -24 * 16 / 2 and torch.isfinite(y).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H", [64, 512, 4096])
def test_selection_at_the_stated_accuracy_of_the_logits(H, dtype):
    """Logits that differ by little more than twice the stated bound, 2^-18 sum |x w|
    and the rounding to FP32, are ranked as the exact ones.  The bias puts the
    exact logits on such a ladder (its own rounding to FP32 is part of them)."""
    E, k = 40, 16
    for seed in range(6):
        w, x = _case(1, H, 64, E, k, dtype, seed=100 * seed + H)
        terms = f64(w["w_router"]) * f64(x)
        dot, mag = terms.sum(1), np.abs(terms).sum(1).max()
        place = np.random.RandomState(seed).permutation(E)
        bound = 2.0 ** -18 * mag + 2.0 ** -24
        ladder = 0.5 - 2.5 * bound * place
        w["bias"] = torch.from_numpy((ladder - dot).astype(np.float32)).to(DEV)
        exact = dot + w["bias"].double().cpu().numpy()
        order = np.argsort(-exact, kind="stable")
        assert np.abs(exact).max() < 1 and np.diff(-exact[order]).min() > 2 * bound
        idx = torch.empty((1, k), dtype=torch.int32, device=DEV)
        _call(w, x, k, "bf16", topk_idx=idx)
        assert idx[0].tolist() == order[:k].tolist()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_h_is_held_in_two_numbers(dtype):
    """Down rows that take the difference of two nearly equal features of h: with h
    rounded once to 16 bits they would be off by 2^-8 (BF16) of it.  The bound is the
    header's for h, the FP32 sums' and y's own rounding."""
    T, H, I = 4, 128, 64
    w, x = _case(T, H, I, 1, 1, dtype, seed=51)
    gu = w["w_gate_up"][0]
    gu[1:I:2] = gu[0:I:2]              # gate features in equal pairs
    gu[I + 1::2] = gu[I::2]            # up features too,
    gu[I + 1::2, 5] *= 1 + 2.0 ** -5   # but for one weight
    wd = torch.zeros_like(w["w_down"][0])
    pairs = torch.arange(H, device=DEV) % (I // 2)
    wd[torch.arange(H), 2 * pairs], wd[torch.arange(H), 2 * pairs + 1] = 1.0, -1.0
    w["w_down"][0] = wd
    y = f64(_call(w, x, 1, "bf16", shared=False))
    x64, wg, wu, wd = f64(x), f64(gu[:I]), f64(gu[I:]), f64(wd)
    g, u = x64 @ wg.T, x64 @ wu.T
    dg, du = (H + 3) * U * (np.abs(x64) @ np.abs(wg).T), (H + 3) * U * (np.abs(x64) @ np.abs(wu).T)
    h = moe.silu(g) * u
    dh = 1.1 * dg * np.abs(u) + (np.abs(moe.silu(g)) + 1.1 * dg) * du + 16 * U * np.abs(h)
    held = 2.0 ** -16 * np.abs(h) if dtype == "bf16" else np.maximum(2.0 ** -22 * np.abs(h), 2.0 ** -25)
    ref = h @ wd.T
    tol = (dh + held + 3 * U * np.abs(h)) @ np.abs(wd).T
    tol = tol + HALF[x.dtype] * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == "f16" else 0.0)
    assert (np.abs(y - ref) <= tol).all()
    once = f64(torch.from_numpy(h).to(x.dtype)) @ wd.T
    assert (np.abs(once - ref) > tol).any()  # the test tells the two apart


def test_an_fp16_h_beyond_its_range_is_infinite():
    T, H, I = 2, 64, 64
    w, x = _case(T, H, I, 1, 1, "f16", seed=52)
    x[1, 0] = 16.0
    w["w_gate_up"][0][:, 0] = 0.0
    w["w_gate_up"][0][0, 0] = w["w_gate_up"][0][I, 0] = 20.0  # g and u of feature 0: about 320 for token 1
    w["w_down"][0][:, 0] = torch.where(torch.arange(H, device=DEV) % 2 == 0, 0.5, -0.5).half()
    x[0, 0] = 0.0
    y = _call(w, x, 1, "bf16", shared=False)
    assert torch.isfinite(y[0]).all()
    assert (y[1, 0::2] == float("inf")).all() and (y[1, 1::2] == float("-inf")).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_same_bits_whatever_the_workspace_holds(fmt):
    """Repeated calls give the same bits, on a workspace of NaNs and after a larger
    batch; a token among others stays within the roundings of its own sums."""
    T, k = 12, 3
    w, x = _case(T, 512, 192, 40, k, seed=61, norm=True, gate=True)
    w = prepare_fp8_weights(w)
    ws = abi.workspace(abi.MOE_OP_LAYER_DECODE, T, 512, 40, k, 192, DEV)
    for t in (1, 3, T):
        want = _call(w, x[:t], k, fmt)
        for fill in (0xff, 0x00, 0x7f):
            ws.fill_(fill)
            assert torch.equal(_call(w, x[:t], k, fmt, ws=ws), want)
        _call(w, x, k, fmt, ws=ws)
        assert torch.equal(_call(w, x[:t], k, fmt, ws=ws), want)
        ref, tol, r = _reference(w, x[:t], k, fmt, "bf16")
        _check(want, ref, tol, r)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_two_host_threads_and_a_given_stream(fmt):
    """Calls from two host threads, each on the stream that it passes."""
    import threading

    k = 3
    w, x = _case(8, 256, 128, 16, k, seed=71, norm=True)
    w = prepare_fp8_weights(w)
    parts = [x[:3].contiguous(), x[3:].contiguous()]
    want = [_call(w, p, k, fmt) for p in parts]
    outs = [[torch.empty_like(p) for _ in range(20)] for p in parts]
    wss = [abi.workspace(abi.MOE_OP_LAYER_DECODE, 8, 256, 16, k, 128, DEV) for _ in parts]
    streams = [torch.cuda.Stream() for _ in parts]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            for y in outs[i]:
                _call(w, parts[i], k, fmt, y=y, ws=wss[i], stream=streams[i])
        except Exception as e:  # reported by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not failed
    assert all(torch.equal(y, want[i]) for i in range(2) for y in outs[i])
