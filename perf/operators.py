"""Cases of the FP8 block-scaled expert products and of the one-kernel decode layer.

Each case is one of four operators:

  quant   moe_fp8_quantize_b128: E4M3 codes with one FP32 scale per 1 x 128 or 128 x 128 block
  gemm    moe_grouped_gemm_fp8_b128: the (grouped) product of two such operands
  swiglu  moe_grouped_swiglu_fp8_b128: the routed experts of a layer with FP8 weights
  layer   moe_layer_decode_bf16 / moe_layer_decode_fp8_b128: a whole MoE layer on at most 16 tokens

The plain forms are elementary torch operations in 32 bits (64 for the norm and the router's logits, which decide a
selection); the quantiser's decisions are FP32 operations by definition.
"""

import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
FLOOR = 2.0 ** -80  # smallest block maximum that a scale is formed from


def listed():
    return [
        # the activations of a prefill batch, quantised in front of the first product
        dict(name="quant_tokens", op="quant", batch=1, rows=8192, K=2048, block_rows=1, dtype="bf16"),
        # an eighth of a 512-expert gate/up bank, quantised once when a checkpoint is loaded
        dict(name="quant_weights", op="quant", batch=64, rows=1280, K=2048, block_rows=128, dtype="bf16"),
        # one dense projection over a prefill batch
        dict(name="gemm_dense", op="gemm", rows=8192, T=8192, K=2048, N=4096, E=1, k=1, gather=False, out="bf16"),
        # the down projection of a 256-expert layer over 16384 tokens x 10 experts
        dict(name="gemm_grouped", op="gemm", rows=163840, T=16384, K=640, N=2048, E=256, k=10, gather=False, out="f16"),
        # a few ragged rows of a small expert bank, gathered; partial blocks along K and N
        dict(name="gemm_ragged", op="gemm", rows=74, T=37, K=592, N=336, E=16, k=2, gather=True, out="f32"),
        # the 512-expert layer's routed experts: prefill, a decode batch of 64, and a tiny odd layer in FP16
        dict(name="swiglu_prefill", op="swiglu", T=8192, H=2048, I=640, E=512, k=10, dtype="bf16"),
        dict(name="swiglu_t64", op="swiglu", T=64, H=2048, I=640, E=512, k=10, dtype="bf16"),
        dict(name="swiglu_tiny", op="swiglu", T=33, H=320, I=192, E=16, k=2, dtype="f16"),
        # whole layers on a few tokens: one token (latency), a small batch with the norm and the shared gate
        dict(name="layer_bf16_t1", op="layer", fmt="bf16", T=1, H=2048, I=640, E=512, k=10, dtype="bf16", norm=False,
             gate=False, shared=True),
        dict(name="layer_f16_t16", op="layer", fmt="bf16", T=16, H=2560, I=640, E=256, k=10, dtype="f16", norm=True,
             gate=True, shared=True),
        dict(name="layer_fp8_t1", op="layer", fmt="fp8", T=1, H=2048, I=640, E=512, k=10, dtype="bf16", norm=False,
             gate=False, shared=True),
        dict(name="layer_fp8_t8", op="layer", fmt="fp8", T=8, H=2048, I=640, E=512, k=10, dtype="bf16", norm=True,
             gate=True, shared=True),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quant", "gemm", "swiglu", "layer", "layer"])
    if op == "quant":
        br = rng.choice([1, 128])
        K = _log(rng, 16, 4096, 16)
        batch = rng.choice([1, 1, rng.randint(2, 16)])
        rows = _log(rng, 1, max(2, (1 << 24) // (K * batch)))
        return dict(op="quant", batch=batch, rows=rows, K=K, block_rows=br, dtype=rng.choice(["bf16", "f16"]))
    if op == "gemm":
        E = rng.choice([1, _log(rng, 2, 128)])
        k = 1 if E == 1 else rng.randint(1, min(E, 8))
        T = _log(rng, 1, 8192 // k)
        K, N = _log(rng, 16, 2560, 16), _log(rng, 16, 2560, 16)
        return dict(op="gemm", rows=T * k, T=T, K=K, N=N, E=E, k=k, gather=E > 1 and rng.random() < 0.5,
                    out=rng.choice(["bf16", "f16", "f32"]))
    if op == "swiglu":
        E = _log(rng, 4, 256)
        k = rng.randint(1, min(E, 10))
        return dict(op="swiglu", T=_log(rng, 1, 4096), H=_log(rng, 64, 2560, 64), I=_log(rng, 64, 1024, 64), E=E, k=k,
                    dtype=rng.choice(["bf16", "f16"]))
    E = _log(rng, 16, 512)
    norm = rng.random() < 0.5
    shared = rng.random() < 0.8
    return dict(op="layer", fmt=rng.choice(["bf16", "fp8"]), T=rng.randint(1, 16), H=_log(rng, 256, 2560, 64),
                I=_log(rng, 64, 768, 64), E=E, k=rng.randint(1, min(E, 12)), dtype=rng.choice(["bf16", "f16"]),
                norm=norm, gate=shared and rng.random() < 0.5, shared=shared)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, shape, std, dtype):
    """N(0, std) in dtype, drawn expert by expert when large."""
    if math.prod(shape) <= 1 << 28:
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 28) * shape[0] // math.prod(shape))
    for a in range(0, shape[0], step):
        b = min(shape[0], a + step)
        out[a:b] = (torch.randn((b - a, *shape[1:]), generator=g, device="cuda") * std).to(dtype)
    return out


def _fp8_weights(g, E, N, K, std):
    """An FP8 checkpoint's tensor: codes [E, N, K] and scales [E, ceil(N/128), ceil(K/128)]."""
    codes = torch.empty((E, N, K), dtype=E4M3, device="cuda")
    scales = torch.empty((E, -(-N // 128), -(-K // 128)), device="cuda")
    step = max(1, (1 << 27) // (N * K))
    for a in range(0, E, step):
        b = min(E, a + step)
        codes[a:b], scales[a:b] = quantize(torch.randn((b - a, N, K), generator=g, device="cuda") * std, 128)
    return codes, scales


def _routed(g, T, E, k):
    """A skewed selection and its permutation by expert: row_token [T*k], offsets [E+1]."""
    logits = torch.randn((T, E), generator=g, device="cuda") + 1.5 * torch.randn((E,), generator=g, device="cuda")
    idx = logits.topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(idx, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(idx, minlength=E).cumsum(0).to(torch.int32)
    return (order // k).to(torch.int32), offsets


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] == "quant":
        # values over several orders of magnitude, one scale per row, and a block of zeros
        v = torch.randn((c["batch"], c["rows"], c["K"]), generator=g, device="cuda")
        v = v * torch.exp(torch.randn((c["batch"], c["rows"], 1), generator=g, device="cuda"))
        s["v"] = v.to(DT[c["dtype"]])
        if c["rows"] > 1:
            s["v"][0, 0, :128] = 0
        return s
    if c["op"] == "gemm":
        x = torch.randn((c["T"] if c["gather"] else c["rows"], c["K"]), generator=g, device="cuda")
        s["a"], s["sa"] = quantize(x, 1)
        s["w"], s["sw"] = _fp8_weights(g, c["E"], c["N"], c["K"], c["K"] ** -0.5)
        row_token, offsets = _routed(g, c["T"], c["E"], c["k"])
        s["offsets"] = offsets
        s["row_token"] = row_token if c["gather"] else None
        return s
    H, I, E, k, dt = c["H"], c["I"], c["E"], c["k"], DT[c["dtype"]]
    s["x"] = _normal(g, (c["T"], H), 1.0, dt)
    if c["op"] == "swiglu":
        s["w_gu"], sc = _fp8_weights(g, 2 * E, I, H, H ** -0.5)
        s["w_gu"], s["sc_gu"] = s["w_gu"].view(E, 2 * I, H), sc.view(E, 2, *sc.shape[1:])
        s["w_d"], s["sc_d"] = _fp8_weights(g, E, H, I, I ** -0.5)
        s["row_token"], s["offsets"] = _routed(g, c["T"], E, k)
        return s
    s["w_router"] = _normal(g, (E, H), H ** -0.5, dt)
    s["bias"] = 1.5 * torch.randn((E,), generator=g, device="cuda")
    if c["fmt"] == "fp8":
        s["w_gu"], sc = _fp8_weights(g, 2 * E, I, H, H ** -0.5)
        s["w_gu"], s["sc_gu"] = s["w_gu"].view(E, 2 * I, H), sc.view(E, 2, *sc.shape[1:])
        s["w_d"], s["sc_d"] = _fp8_weights(g, E, H, I, I ** -0.5)
    else:
        s["w_gu"], s["w_d"] = _normal(g, (E, 2 * I, H), H ** -0.5, dt), _normal(g, (E, H, I), I ** -0.5, dt)
    s["w_sh_gu"] = _normal(g, (2 * I, H), H ** -0.5, dt) if c["shared"] else None
    s["w_sh_d"] = _normal(g, (H, I), I ** -0.5, dt) if c["shared"] else None
    s["norm_w"] = _normal(g, (H,), 0.1, dt) if c["norm"] else None
    s["w_sh_gate"] = _normal(g, (H,), H ** -0.5, dt) if c["gate"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _blocks(v, block_rows):
    """[B, R, K] -> [B, R/br, br, K/128, 128], padded with zeros."""
    B, R, K = v.shape
    v = torch.nn.functional.pad(v, (0, -K % 128, 0, -R % block_rows))
    return v.view(B, (R + block_rows - 1) // block_rows, block_rows, -1, 128)


def quantize(v, block_rows):
    """E4M3 codes and FP32 scales of v [.., R, K]: every step one FP32 operation."""
    shape = v.shape
    v = v.float().reshape(-1, *shape[-2:])
    b = _blocks(v, block_rows)
    a = b.abs().amax(dim=(2, 4), keepdim=True).clamp_min(FLOOR)
    top = torch.full_like(a, 448.0)  # a tensor: a Python number would be divided by its reciprocal, with two roundings
    codes = (b * (top / a)).to(E4M3).float()
    codes = codes.view(b.shape[0], b.shape[1] * block_rows, -1)[:, : shape[-2], : shape[-1]].to(E4M3)
    scales = (a / top)[:, :, 0, :, 0]
    return codes.reshape(shape).contiguous(), scales.reshape(*shape[:-2], *scales.shape[1:]).contiguous()


def dequantize(codes, scales, block_rows):
    R, K = codes.shape[-2:]
    s = scales.repeat_interleave(block_rows, -2)[..., :R, :] if block_rows > 1 else scales
    return codes.float() * s.repeat_interleave(128, -1)[..., :K]


def _per_expert(a, w, offsets):
    """Rows of a [rows, K] (sorted by expert) times their expert's w [E, N, K]: tiles of 128 rows, one expert each."""
    rows, E = a.shape[0], w.shape[0]
    if E == 1:
        return a @ w[0].t()
    tile = 128 if rows > 8 * E else 8
    off = offsets.long()
    count = (off[1:] - off[:-1] + tile - 1) // tile
    start = count.cumsum(0) - count
    t = torch.arange((rows + tile - 1) // tile + min(E, rows), device=a.device)
    e = torch.searchsorted(start + count, t, right=True).clamp_max(E - 1)
    row = (off[e] + (t - start[e]) * tile)[:, None] + torch.arange(tile, device=a.device)
    ok = (row < off[e + 1][:, None]) & (t < start[-1] + count[-1])[:, None]
    # the rows that no tile holds are sent to one spare row behind the result
    r = torch.where(ok, row, rows)
    prod = torch.bmm(a[row.clamp_max(rows - 1)], w[e].transpose(1, 2))
    out = torch.empty((rows + 1, w.shape[1]), device=a.device)
    out[r.reshape(-1)] = prod.view(-1, w.shape[1])
    return out[:rows]


def _silu(v):
    return v / (1 + torch.exp(-v))


def _swiglu_fp8(x, row_token, offsets, w_gu, sc_gu, w_d, sc_d):
    E, I, H = w_gu.shape[0], w_gu.shape[1] // 2, w_gu.shape[2]
    xq = dequantize(*quantize(x, 1), 1)[row_token.long()]
    w = dequantize(w_gu.view(E, 2, I, H), sc_gu, 128).view(E, 2 * I, H)
    gu = _per_expert(xq, w, offsets)
    h = dequantize(*quantize(_silu(gu[:, :I]) * gu[:, I:], 1), 1)
    return _per_expert(h, dequantize(w_d, sc_d, 128), offsets)


def _layer(s):
    c = s["case"]
    T, H, I, k = c["T"], c["H"], c["I"], c["k"]
    x = s["x"]
    if c["norm"]:
        d = x.double()
        d = d / (d.square().mean(1, keepdim=True) + 1e-6).sqrt() * (1 + s["norm_w"].double())
        x = d.to(x.dtype)
    logits = x.double() @ s["w_router"].double().t() + s["bias"].double()
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    p = torch.exp(top - top[:, :1])
    p = (p / p.sum(1, keepdim=True)).float()
    w_gu, w_d, xf = s["w_gu"][idx], s["w_d"][idx], x.float()
    if c["fmt"] == "fp8":
        xf = dequantize(*quantize(x, 1), 1)
        w_gu = dequantize(w_gu.view(T, k, 2, I, H), s["sc_gu"][idx], 128).view(T, k, 2 * I, H)
        w_d = dequantize(w_d, s["sc_d"][idx], 128)
    gu = (w_gu.float() @ xf.view(T, 1, H, 1))[..., 0]
    h = _silu(gu[..., :I]) * gu[..., I:]
    if c["fmt"] == "fp8":
        h = dequantize(*quantize(h, 1), 1)
    y = ((w_d.float() @ h[..., None])[..., 0] * p[..., None]).sum(1)
    if c["shared"]:
        gu = x.float() @ s["w_sh_gu"].float().t()
        sh = (_silu(gu[:, :I]) * gu[:, I:]) @ s["w_sh_d"].float().t()
        if c["gate"]:
            sh = sh / (1 + torch.exp(-(x.float() @ s["w_sh_gate"].float())))[:, None]
        y = y + sh
    return y.to(x.dtype)


def _kept(s, name, make):
    """A buffer that the user's program allocates once and keeps with its weights."""
    if name not in s:
        s[name] = make()
    return s[name]


def _own(s):
    from bit_expert_gemm_b200 import abi

    c = s["case"]
    if c["op"] == "quant":
        return abi.moe_fp8_quantize_b128(s["v"], c["block_rows"])
    if c["op"] == "gemm":
        return abi.moe_grouped_gemm_fp8_b128(s["a"], s["sa"], s["w"], s["sw"], expert_offsets=s["offsets"],
                                             row_token=s["row_token"], out_dtype=DT[c["out"]])
    if c["op"] == "swiglu":
        rows = c["T"] * c["k"]
        ws = _kept(s, "ws", lambda: abi.workspace(abi.MOE_OP_SWIGLU_FP8_B128, c["T"], c["H"], c["E"], c["k"], c["I"],
                                                  s["x"].device))
        return abi.moe_grouped_swiglu_fp8_b128(s["x"], s["row_token"], s["offsets"], rows, s["w_gu"], s["sc_gu"],
                                               s["w_d"], s["sc_d"], ws=ws)
    ws = _kept(s, "ws", lambda: abi.workspace(abi.MOE_OP_LAYER_DECODE, c["T"], c["H"], c["E"], c["k"], c["I"],
                                              s["x"].device))
    rest = dict(w_sh_gate_up=s["w_sh_gu"], w_sh_down=s["w_sh_d"], norm_w=s["norm_w"], w_shared_gate=s["w_sh_gate"],
                ws=ws)
    if c["fmt"] == "fp8":
        return abi.moe_layer_decode_fp8_b128(s["x"], s["w_router"], s["bias"], c["k"], s["w_gu"], s["sc_gu"], s["w_d"],
                                             s["sc_d"], **rest)
    return abi.moe_layer_decode_bf16(s["x"], s["w_router"], s["bias"], c["k"], s["w_gu"], s["w_d"], **rest)


def run(state):
    c = state["case"]
    if c["op"] == "quant":
        codes, scales = _own(state) if own else quantize(state["v"], c["block_rows"])
        return {"codes": codes, "scales": scales}  # codes: E4M3 values
    if own:
        return _own(state)
    if c["op"] == "gemm":
        a = dequantize(state["a"], state["sa"], 1)
        a = a[state["row_token"].long()] if c["gather"] else a
        return _per_expert(a, dequantize(state["w"], state["sw"], 128), state["offsets"]).to(DT[c["out"]])
    if c["op"] == "swiglu":
        f = _swiglu_fp8(state["x"], state["row_token"], state["offsets"], state["w_gu"], state["sc_gu"], state["w_d"],
                        state["sc_d"])
        return f.to(DT[c["dtype"]])
    return _layer(state)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------
def _touched(T, E, k):
    """Experts that a skewed batch of T tokens selects (the distribution of prepare)."""
    r = np.random.RandomState(1)
    logits = r.randn(T, E) + 1.5 * r.randn(E)
    return len(np.unique(np.argsort(-logits, axis=1)[:, :k]))


def work(case):
    c = case
    if c["op"] == "quant":
        n, blocks = c["batch"] * c["rows"] * c["K"], c["batch"] * -(-c["rows"] // c["block_rows"]) * -(-c["K"] // 128)
        return {"bytes": 3 * n + 4 * blocks, "flops": 3 * n}
    if c["op"] == "gemm":
        E = _touched(c["T"], c["E"], c["k"]) if c["E"] > 1 else 1
        src = c["T"] if c["gather"] else c["rows"]
        out = 4 if c["out"] == "f32" else 2
        return {"bytes": src * c["K"] + E * c["N"] * c["K"] + c["rows"] * c["N"] * out,
                "flops": 2 * c["rows"] * c["N"] * c["K"]}
    T, H, I, k = c["T"], c["H"], c["I"], c["k"]
    E = _touched(T, c["E"], k)
    if c["op"] == "swiglu":
        return {"bytes": 2 * T * H + 3 * E * H * I + 2 * T * k * H, "flops": 6 * T * k * H * I}
    each = 1 if c["fmt"] == "fp8" else 2
    n_sh = 1 if c["shared"] else 0
    return {"bytes": 4 * T * H + 2 * c["E"] * H + 3 * H * I * (each * E + 2 * n_sh),
            "flops": 2 * T * c["E"] * H + 6 * T * H * I * (k + n_sh)}


def _q64(v, br=1):
    """The values that quantised rows stand for, in 64 bits (the decisions are FP32 by definition), row blocks of 1."""
    n, K = v.shape
    p = torch.zeros((n, -(-K // 128) * 128), dtype=torch.float32, device=v.device)
    p[:, :K] = v.to(torch.float32)
    p = p.view(n, -1, 128)
    a = torch.maximum(p.abs().max(2, keepdim=True).values, torch.tensor(FLOOR, device=v.device))
    q = torch.mul(p, torch.div(torch.tensor(448.0, device=v.device), a)).to(E4M3).double()
    return (q * torch.div(a, torch.tensor(448.0, device=v.device)).double()).reshape(n, -1)[:, :K]


def _w64(codes, scales):
    """One expert's weight matrix in 64 bits."""
    n, k = codes.shape
    rows, cols = torch.arange(n, device=codes.device) // 128, torch.arange(k, device=codes.device) // 128
    return codes.double() * scales.double()[rows[:, None], cols[None, :]]


def _act64(gu):
    g, u = gu.chunk(2, dim=1)
    return g * torch.sigmoid(g) * u


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quant":
        br, v = c["block_rows"], s["v"].double()
        B, R, K = v.shape
        nr, nk = -(-R // br), -(-K // 128)
        i, j = torch.arange(R, device="cuda") // br, torch.arange(K, device="cuda") // 128
        flat = (i[:, None] * nk + j[None, :]).expand(B, R, K).reshape(B, -1)
        a = torch.zeros((B, nr * nk), dtype=torch.float64, device="cuda")
        a = a.scatter_reduce(1, flat, v.abs().reshape(B, -1), "amax").clamp_min(FLOOR)
        inv = torch.div(torch.tensor(448.0, device="cuda"), a.float()).gather(1, flat).reshape(B, R, K)
        return {"codes": (v.float() * inv).to(E4M3).double(), "scales": (a / 448.0).reshape(B, nr, nk)}
    if c["op"] in ("gemm", "swiglu"):
        off = s["offsets"].tolist()
        n = c["T"] * c["k"]
        out = torch.empty((n, c["N"] if c["op"] == "gemm" else c["H"]), dtype=torch.float64, device="cuda")
        if c["op"] == "gemm":
            a = s["a"].double() * s["sa"].double()[:, torch.arange(c["K"], device="cuda") // 128]
        else:
            a = _q64(s["x"])
        for e in range(c["E"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            r = a[s["row_token"][lo:hi].long()] if s["row_token"] is not None else a[lo:hi]
            if c["op"] == "gemm":
                out[lo:hi] = r @ _w64(s["w"][e], s["sw"][e]).t()
            else:
                I = c["I"]
                gate, up = (_w64(s["w_gu"][e, q * I:(q + 1) * I], s["sc_gu"][e, q]) for q in (0, 1))
                h = _q64(_act64(torch.cat([r @ gate.t(), r @ up.t()], dim=1)))
                out[lo:hi] = h @ _w64(s["w_d"][e], s["sc_d"][e]).t()
        return out
    I, k, x = c["I"], c["k"], s["x"]
    if c["norm"]:
        x64 = x.double()
        x = ((1 + s["norm_w"].double()) * x64 / torch.sqrt((x64 ** 2).sum(1, keepdim=True) / c["H"] + 1e-6)).to(x.dtype)
    x64 = x.double()
    logits = torch.nn.functional.linear(x64, s["w_router"].double(), s["bias"].double()).cpu().numpy()
    y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
    for t in range(c["T"]):
        chosen = np.lexsort((np.arange(c["E"]), -logits[t]))[:k]
        soft = np.exp(logits[t] - logits[t].max())
        weight = soft[chosen] / soft[chosen].sum()
        xe = _q64(x[t:t + 1]) if c["fmt"] == "fp8" else x64[t:t + 1]
        for e, p in zip(chosen.tolist(), weight.tolist()):
            if c["fmt"] == "fp8":
                gate, up = (_w64(s["w_gu"][e, q * I:(q + 1) * I], s["sc_gu"][e, q]) for q in (0, 1))
                h = _q64(_act64(torch.cat([xe @ gate.t(), xe @ up.t()], dim=1)))
                y[t] += p * (h @ _w64(s["w_d"][e], s["sc_d"][e]).t())[0]
            else:
                y[t] += p * (_act64(xe @ s["w_gu"][e].double().t()) @ s["w_d"][e].double().t())[0]
    if c["shared"]:
        sh = _act64(x64 @ s["w_sh_gu"].double().t()) @ s["w_sh_d"].double().t()
        y += sh * (torch.sigmoid(x64 @ s["w_sh_gate"].double())[:, None] if c["gate"] else 1.0)
    return y
