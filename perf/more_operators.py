"""Measured cases of 8-bit activations over MXFP4 weights: norms, products and experts of a decoder block.

MXFP8 (OCP Microscaling, E4M3 elements): 32 consecutive elements of a row share one E8M0 scale 2^(byte - 127)
(byte 255 = NaN); an element is E4M3 (3 bits of mantissa, exponents -6 to 8, subnormal steps of 2^-9, largest 448).
Quantising a block: byte = clamp(exponent(amax) - 8 + 127, 0, 254), 255 when the block holds a NaN or an infinity;
element = E4M3 round-to-nearest-even of x * 2^(127 - byte), saturating at 448.  Weights are MXFP4: E2M1 elements
(magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6, bit 3 = sign) under the same kind of scales.

Operators (``case["op"]``) and what one pass is, q(.) being the rounding to MXFP8:

* ``norm_in``   n = bf16(x / rms(x) * w), and q(n) read back as values
                (moe_norm_in_mxfp8, mxfp8_dequantize)
* ``norm_out``  r' = bf16(r + s * gate * (y / rms(y) * w_post)), n = bf16(r' / rms(r') * w_next), and q(n) read back
                (moe_norm_out_mxfp8, mxfp8_dequantize)
* ``linear``    y = act(q(x) . W^T + bias) + residual                   (mxfp8_quantize, mxfp8_linear)
* ``experts``   the routed experts' SwiGLU FFN from x and a routing to y (mxfp8_quantize, mxfp8_grouped_ffn,
                moe_combine); what is between its two products is rounded to MXFP8 too
* ``layer``     the same with its sigmoid + bias top-k router, as one call for a few tokens (mxfp8_moe_layer)

Packed weights ([N, K], rows padded to 32 and columns to 256 with zeros) are stored as the 32 x 64
operand fragments that a wave loads: codes [G, KK, 4, 64, 16] bytes and scales [G, KK, 64, 4] bytes,
where lane 32 * f + m of row group g, column group c holds row 32 g + rho(m), and its piece s is block
8 c + 4 f + s of that row; rho exchanges bit 2 of m with bits 3-4: rho(8 q + 4 h + j) = 16 h + 4 q + j.
"""

import math

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
RSF = 2.5


# ---------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # after the attention of one decoded token: the residual, and the norm that the experts read in 8 bits
        {"name": "norm_out_token", "op": "norm_out", "T": 1, "H": 6144, "y": "bf16", "gate": "token", "scale": 1.0},
        # the norm before a block over an odd batch cut out of a wider buffer
        {"name": "norm_in_batch", "op": "norm_in", "T": 1999, "H": 2080, "pad": 8},
        # after the block of a prompt: FP32 block output, channel gate, residual, the next block's norm
        {"name": "norm_out_prompt", "op": "norm_out", "T": 8192, "H": 6144, "y": "fp32", "gate": "channel",
         "scale": 0.25},
        # the output projection of one decoded token, added to the residual: the weights' bytes
        {"name": "linear_token", "op": "linear", "T": 1, "K": 6144, "N": 6144, "out": "bf16", "bias": False,
         "act": "none", "residual": "bf16"},
        # a ragged batch through an odd layer with a bias and an activation, FP32 result
        {"name": "linear_ragged_f32", "op": "linear", "T": 77, "K": 2080, "N": 1000, "out": "fp32", "bias": True,
         "act": "gelu", "residual": "none"},
        # a chunk of a prompt, into a narrower layer
        {"name": "linear_chunk", "op": "linear", "T": 509, "K": 6144, "N": 2048, "out": "bf16", "bias": True,
         "act": "silu", "residual": "none"},
        # a prompt through the output projection, added to the residual: the matrix cores
        {"name": "linear_prompt", "op": "linear", "T": 8192, "K": 6144, "N": 6144, "out": "bf16", "bias": True,
         "act": "none", "residual": "bf16"},
        # a chunk of a prompt through 80 experts, top-8: every expert's weights for some 26 rows each
        {"name": "experts_chunk", "op": "experts", "T": 256, "E": 80, "k": 8, "H": 6144, "I": 2048, "skew": 0.5},
        # a prompt through the same experts, some of them much more popular than others
        {"name": "experts_prompt", "op": "experts", "T": 8192, "E": 80, "k": 8, "H": 6144, "I": 2048, "skew": 1.0},
        # the tiny layer: 8 experts, top-2
        {"name": "layer_tiny", "op": "layer", "T": 16, "E": 8, "k": 2, "H": 256, "I": 128, "skew": 0.3},
        # one decoded token through the whole layer: 8 experts' bytes
        {"name": "layer_token", "op": "layer", "T": 1, "E": 80, "k": 8, "H": 6144, "I": 2048, "skew": 0.3},
        # a decode batch through the whole layer: the touched experts' bytes
        {"name": "layer_decode", "op": "layer", "T": 16, "E": 80, "k": 8, "H": 6144, "I": 2048, "skew": 0.3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_in", "norm_out", "linear", "linear", "experts", "layer", "layer"])
    if op == "norm_in":
        return {"op": op, "T": _log(rng, 1, 8192), "H": 32 * _log(rng, 2, 192), "pad": rng.choice([0, 0, 8, 5])}
    if op == "norm_out":
        return {"op": op, "T": _log(rng, 1, 8192), "H": 32 * _log(rng, 2, 192), "y": rng.choice(["bf16", "fp32"]),
                "gate": rng.choice(["none", "token", "channel", "full"]), "scale": rng.choice([1.0, 0.25])}
    if op == "linear":
        return {"op": op, "T": _log(rng, 1, 8192), "K": 32 * _log(rng, 2, 192), "N": _log(rng, 33, 6144),
                "out": rng.choice(["bf16", "bf16", "fp32"]), "bias": rng.random() < 0.5,
                "act": rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"]),
                "residual": rng.choice(["none", "bf16", "fp32"])}
    E = _log(rng, 4, 80)
    sizes = {"E": E, "H": 32 * _log(rng, 8, 192), "I": 32 * _log(rng, 4, 64)}
    if op == "experts":
        return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, min(8, E)), "skew": rng.choice([0.0, 0.5, 1.0]),
                **sizes}
    T = _log(rng, 1, 32)
    return {"op": op, "T": T, "k": rng.randint(1, min(8, E, 128 // T)), "skew": rng.choice([0.0, 0.3, 1.0]), **sizes}


def work(case):
    op = case["op"]
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        size = {"none": 0, "bf16": 2, "fp32": 4}
        return {"bytes": T * K * 2 + N * K * 17 // 32 + T * N * (size[case["out"]] + size[case["residual"]])
                + (2 * N if case["bias"] else 0), "flops": 2 * T * K * N}
    if op in ("experts", "layer"):
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        touched = E * (1.0 - (1.0 - k / E) ** T)  # experts that a token reaches, for an even routing
        router = E * H * 2 if op == "layer" else T * k * 8
        return {"bytes": int(T * H * 4 + touched * 3 * H * I * 17 / 32 + router),
                "flops": 6 * T * k * H * I + (2 * T * E * H if op == "layer" else 0)}
    T, H = case["T"], case["H"]
    values = T * H * 33 // 32 + T * H * 2  # codes with scales, and the values that they stand for
    if op == "norm_in":
        return {"bytes": T * H * 4 + values + H * 2, "flops": 4 * T * H}
    gate = {"none": 0, "token": 2 * T, "channel": 2 * H, "full": 2 * T * H}[case["gate"]]
    return {"bytes": T * H * ((2 if case["y"] == "bf16" else 4) + 4) + values + 4 * H + gate, "flops": 10 * T * H}


# ---------------------------------------------------------------------------------------------
# inputs


def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _activations(rows, cols, pad, dtype, g, device):
    """Activations of a transformer block: normal, with a spread of the channels' sizes."""
    spread = torch.exp(0.6 * torch.randn(cols + pad, generator=g, device=device))
    x = torch.randn(rows, cols + pad, generator=g, device=device).mul_(spread).to(dtype)
    return x[:, :cols]


def _fp4_blocks(x):
    """x FP32 [..., 32] -> MXFP4 scale bytes [...] and codes [..., 32], both uint8 (finite x)."""
    a = x.abs()
    byte = ((a.amax(-1).view(torch.int32) >> 23) - 2).clamp(min=0)
    v = a * ((254 - byte) << 23).view(torch.float32).unsqueeze(-1)
    code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5))
    return byte.to(torch.uint8), code | (torch.signbit(x).to(torch.uint8) << 3)


def _pack_weights(w):
    """FP32 [B, N, K] -> packed codes [B, G, KK, 4, 64, 16], scales [B, G, KK, 64, 4], largest scale byte [B]."""
    B, N, K = w.shape
    G, KK = -(-N // 32), -(-K // 256)
    byte, code = _fp4_blocks(torch.nn.functional.pad(w, (0, 256 * KK - K, 0, 32 * G - N)).view(B, 32 * G, KK * 8, 32))
    pairs = code.view(B, 32 * G, KK * 8, 16, 2)
    packed = pairs[..., 0] | (pairs[..., 1] << 4)
    codes = packed.view(B, G, 2, 4, 4, KK, 2, 4, 16).permute(0, 1, 5, 7, 6, 3, 2, 4, 8).reshape(B, G, KK, 4, 64, 16)
    scales = byte.view(B, G, 2, 4, 4, KK, 2, 4).permute(0, 1, 5, 6, 3, 2, 4, 7).reshape(B, G, KK, 64, 4)
    return codes.contiguous(), scales.contiguous(), byte.view(B, -1).amax(1).to(torch.int32)


def _weights(B, N, K, g, device):
    """Packed MXFP4 weights of B matrices [N, K], a few matrices at a time."""
    parts = []
    step = max(1, (1 << 27) // (N * K))
    for b in range(0, B, step):
        w = torch.randn(min(step, B - b), N, K, generator=g, device=device).mul_(0.7 * K ** -0.5)
        parts.append(_pack_weights(w))
    return tuple(torch.cat(p) for p in zip(*parts))


def _routing(T, E, k, skew, g, device):
    """A top-k routing with its expert-sorted order, and a plan of row tiles that cover each expert's pairs."""
    score = torch.randn(T, E, generator=g, device=device) + skew * torch.randn(E, generator=g, device=device)
    top, ids = score.topk(k, dim=1)
    p = torch.sigmoid(top)
    topk_w = RSF * p / p.sum(1, keepdim=True)
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rows = max(8, min(256, 8 * math.ceil(T * k / E / 8)))
    n = counts.tolist()
    start, tiles, experts = 0, [], []
    for e, c in enumerate(n):
        for a in range(0, c, rows):
            tiles.append((start + a, min(rows, c - a)))
            experts.append(e)
        start += c
    first = torch.tensor([t[0] for t in tiles], device=device).view(-1, 1)
    size = torch.tensor([t[1] for t in tiles], device=device).view(-1, 1)
    at = torch.arange(rows, device=device).view(1, -1)
    pairs = torch.where(at < size, order[(first + at).clamp(max=T * k - 1)], T * k)  # T * k: no pair
    return {"ids": ids, "topk_w": topk_w.to(torch.float32).contiguous(), "offsets": offsets.to(torch.int32),
            "sorted": order.to(torch.int32), "tile_pairs": pairs,
            "tile_expert": torch.tensor(experts, device=device)}


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    g = _gen(seed, device)
    op = case["op"]
    s = {"case": case}
    bf16 = lambda *shape: torch.randn(*shape, generator=g, device=device).to(torch.bfloat16)  # noqa: E731
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        s["x"] = _activations(T, K, 0, torch.bfloat16, g, device)
        codes, scales, _ = _weights(1, N, K, g, device)
        s["w_codes"], s["w_scales"] = codes[0], scales[0]
        s["bias"] = bf16(N) if case["bias"] else None
        r = case["residual"]
        s["residual"] = None if r == "none" else _activations(T, N, 0, DTYPES[r], g, device)
    elif op in ("experts", "layer"):
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        s["x"] = _activations(T, H, 0, torch.bfloat16, g, device)
        s["w13"] = _weights(E, 2 * I, H, g, device)[:2]
        s["w2"] = _weights(E, H, I, g, device)
        if op == "experts":
            s["route"] = _routing(T, E, k, case["skew"], g, device)
        else:
            s["w_router"] = (torch.randn(E, H, generator=g, device=device) * H ** -0.5).to(torch.bfloat16)
            s["bias"] = case["skew"] * torch.randn(E, generator=g, device=device)
    else:
        T, H = case["T"], case["H"]
        weight = lambda: (1.0 + 0.2 * torch.randn(H, generator=g, device=device)).to(torch.bfloat16)  # noqa: E731
        s["w"] = weight()
        if op == "norm_in":
            s["x"] = _activations(T, H, case["pad"], torch.bfloat16, g, device)
        else:
            s["y"] = _activations(T, H, 0, DTYPES[case["y"]], g, device)
            s["r"] = _activations(T, H, 0, torch.bfloat16, g, device)
            s["w_next"] = weight()
            shape = {"none": None, "token": (T, 1), "channel": (1, H), "full": (T, H)}[case["gate"]]
            s["gate"] = None if shape is None else bf16(*shape)
    return s


# ---------------------------------------------------------------------------------------------
# the plain forms


def _power(e):
    """2^e in FP32 for whole e from -126 to 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _rounded(x):
    """The values that the MXFP8 form of x [..., C] stands for, FP32 (every step but the rounding is exact)."""
    blocks = x.to(torch.float32).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = blocks.abs().amax(-1, keepdim=True)
    exponent = top.view(torch.int32) >> 23  # 255 for a NaN or an infinity
    e = (exponent - 8).clamp(0, 246) - 127
    v = blocks * _power(-e)
    step = _power(((v.view(torch.int32) >> 23) & 255).clamp(min=121) - 127 - 3)  # of E4M3 around v
    q = (torch.round(v / step) * step).clamp(-448.0, 448.0)
    q = q * _power(e.clamp(min=-126)) * torch.where(e < -126, 0.5, 1.0)
    return torch.where(exponent == 255, torch.nan, q).view(x.shape)


def _unpacked(codes, scales, N, K):
    """Packed weights [B, ...] -> FP32 values [B, N, K]."""
    B, G, KK = codes.shape[:3]
    half = torch.tensor(LEVELS, device=codes.device)
    levels = torch.cat([half, -half])
    every = torch.arange(256, device=codes.device)
    pair = torch.stack([levels[every & 15], levels[every >> 4]], 1)
    rows = codes.view(B, G, KK, 4, 2, 4, 2, 4, 16).permute(0, 1, 6, 5, 7, 2, 4, 3, 8).reshape(B, 32 * G, KK * 8, 16)
    byte = scales.view(B, G, KK, 2, 4, 2, 4, 4).permute(0, 1, 5, 4, 6, 2, 3, 7).reshape(B, 32 * G, KK * 8)
    values = pair[rows.to(torch.int32)].view(B, 32 * G, KK * 8, 32)
    b = byte.to(torch.int32)
    bits = torch.where(b == 0, 0x00400000, torch.where(b == 255, 0x7FC00000, b << 23)).to(torch.int32)
    values *= bits.view(torch.float32).unsqueeze(-1)
    return values.view(B, 32 * G, KK * 256)[:, :N, :K]


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _activate(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "silu":
        return _silu(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z


def _unit_rms(v):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _plain_linear(s):
    case = s["case"]
    w = _unpacked(s["w_codes"][None], s["w_scales"][None], case["N"], case["K"])[0]
    z = _rounded(s["x"]) @ w.t()
    if s["bias"] is not None:
        z = z + s["bias"].to(torch.float32)
    z = _activate(z, case["act"])
    if s["residual"] is not None:
        z = z + s["residual"].to(torch.float32)
    return z.to(DTYPES[case["out"]])


def _plain_experts(s):
    case = s["case"]
    T, k, H, I = (case[n] for n in ("T", "k", "H", "I"))
    r = s["route"]
    pairs, expert = r["tile_pairs"], r["tile_expert"]
    rows = _rounded(s["x"])[pairs.clamp(max=T * k - 1) // k]
    w = _unpacked(s["w13"][0][expert], s["w13"][1][expert], 2 * I, H)
    gate, up = torch.bmm(rows, w.transpose(1, 2)).split(I, dim=2)
    del w
    h = _rounded(_silu(gate) * up)
    w = _unpacked(s["w2"][0][expert], s["w2"][1][expert], H, I)
    f = torch.bmm(h, w.transpose(1, 2))
    del w
    out = f.new_zeros(T * k + 1, H)
    out[pairs] = f
    return (out[: T * k].view(T, k, H) * r["topk_w"].unsqueeze(-1)).sum(1).to(torch.bfloat16)


def _plain_layer(s):
    case = s["case"]
    T, k, H, I = (case[n] for n in ("T", "k", "H", "I"))
    p = torch.sigmoid(s["x"].double() @ s["w_router"].double().t())  # in 64 bits: it decides which experts
    ids = torch.sort(p + s["bias"].double(), dim=1, descending=True, stable=True)[1][:, :k]
    chosen = p.gather(1, ids)
    topk_w = (RSF * chosen / chosen.sum(1, keepdim=True)).to(torch.float32)
    expert = ids.reshape(-1)
    rows = _rounded(s["x"]).repeat_interleave(k, 0).unsqueeze(2)  # [T k, H, 1]
    w = _unpacked(s["w13"][0][expert], s["w13"][1][expert], 2 * I, H)
    gate, up = torch.bmm(w, rows).squeeze(2).split(I, dim=1)
    del w
    h = _rounded(_silu(gate) * up).unsqueeze(2)
    w = _unpacked(s["w2"][0][expert], s["w2"][1][expert], H, I)
    f = torch.bmm(w, h).view(T, k, H)
    return (f * topk_w.unsqueeze(-1)).sum(1).to(torch.bfloat16), ids.to(torch.int32), topk_w


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "linear":
        return _plain_linear(s)
    if op == "experts":
        return _plain_experts(s)
    if op == "layer":
        return _plain_layer(s)
    if op == "norm_in":
        n = (_unit_rms(s["x"].to(torch.float32)) * s["w"].to(torch.float32)).to(torch.bfloat16)
        return n, _rounded(n).to(torch.bfloat16)
    z = _unit_rms(s["y"].to(torch.float32)) * s["w"].to(torch.float32)
    if s["gate"] is not None:
        z = z * s["gate"].to(torch.float32)
    r = (s["r"].to(torch.float32) + case["scale"] * z).to(torch.bfloat16)
    n = (_unit_rms(r.to(torch.float32)) * s["w_next"].to(torch.float32)).to(torch.bfloat16)
    return r, _rounded(n).to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------
# the framework's operators


def _own(s):
    from nvfp4_w4a4_mixture_amd import ops

    case = s["case"]
    op = case["op"]
    if op == "linear":
        codes, scales = ops.mxfp8_quantize(s["x"])
        act = None if case["act"] == "none" else case["act"]
        return ops.mxfp8_linear(codes, scales, s["w_codes"], s["w_scales"], case["N"], DTYPES[case["out"]],
                                bias=s["bias"], activation=act, residual=s["residual"])
    if op == "experts":
        r = s["route"]
        codes, scales = ops.mxfp8_quantize(s["x"])
        pair_out, pair_scale = ops.mxfp8_grouped_ffn(codes, scales, *s["w13"], *s["w2"], case["H"], case["I"],
                                                     case["k"], r["offsets"], r["sorted"], r["topk_w"])
        return ops.moe_combine(pair_out, pair_scale, case["T"], case["k"])
    if op == "layer":
        return ops.mxfp8_moe_layer(s["x"], s["w_router"], s["bias"], case["k"], RSF, *s["w13"], *s["w2"][:2])
    if op == "norm_in":
        n, codes, scales = ops.moe_norm_in_mxfp8(s["x"], s["w"], EPS)
        return n, ops.mxfp8_dequantize(codes, scales, case["H"])
    r, _, codes, scales = ops.moe_norm_out_mxfp8(s["y"], s["r"], s["w"], s["w_next"], gate=s["gate"],
                                                 residual_scale=case["scale"], eps=EPS, n=False)
    return r, ops.mxfp8_dequantize(codes, scales, case["H"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits


def _grid64(x):
    """MXFP8 rounding of FP64 x [..., C] by the definition: the block's power of two, then the nearest element."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))  # amax = m * 2^e with m in [0.5, 1)
    unit = torch.exp2((e - 9).clamp(-127, 127).to(torch.float64))
    m = b / unit
    _, p = torch.frexp(m.abs())
    step = torch.exp2((p - 1).clamp(min=-6).to(torch.float64) - 3.0)
    return (torch.round(m / step) * step).clamp(-448.0, 448.0).mul(unit).view(x.shape)


def _matrix64(codes, scales, N, K):
    """One packed matrix as FP64 [N, K], element by element from the layout's address formula."""
    r = torch.arange(N, device=codes.device).view(-1, 1)
    c = torch.arange(K, device=codes.device).view(1, -1)
    h, q, j = (r >> 4) & 1, (r >> 2) & 3, r & 3
    block = (c >> 5) & 7
    lane = 32 * (block >> 2) + 8 * q + 4 * h + j
    byte = codes[r >> 5, c >> 8, block & 3, lane, (c & 31) >> 1].to(torch.int32)
    code = torch.where((c & 1) == 1, byte >> 4, byte & 15)
    exponent = scales[r >> 5, c >> 8, lane, block & 3].to(torch.float64) - 127.0
    magnitude = torch.tensor(LEVELS, dtype=torch.float64, device=codes.device)[code & 7]
    return torch.where(code >= 8, -magnitude, magnitude) * torch.exp2(exponent)


def _experts64(s, ids, weight):
    case = s["case"]
    x = _grid64(s["x"].double())
    y = torch.zeros_like(x)
    I = case["I"]
    for e in range(case["E"]):
        t, j = torch.where(ids == e)
        if t.numel() == 0:
            continue
        z = x[t] @ _matrix64(s["w13"][0][e], s["w13"][1][e], 2 * I, case["H"]).t()
        h = _grid64(z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:])
        f = h @ _matrix64(s["w2"][0][e], s["w2"][1][e], case["H"], I).t()
        y.index_add_(0, t, f * weight[t, j].unsqueeze(1))
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        z = _grid64(s["x"].double()) @ _matrix64(s["w_codes"], s["w_scales"], case["N"], case["K"]).t()
        if s["bias"] is not None:
            z = z + s["bias"].double()
        act = case["act"]
        if act == "relu":
            z = torch.maximum(z, torch.zeros_like(z))
        elif act == "silu":
            z = z * torch.sigmoid(z)
        elif act == "gelu":
            z = z * torch.special.ndtr(z)
        elif act == "gelu_tanh":
            z = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
        return z if s["residual"] is None else z + s["residual"].double()
    if op == "experts":
        return _experts64(s, s["route"]["ids"], s["route"]["topk_w"].double())
    if op == "layer":
        z = (s["x"].double().unsqueeze(1) * s["w_router"].double().unsqueeze(0)).sum(-1)
        p = 1.0 / (1.0 + torch.exp(-z))
        score = p + s["bias"].double()
        ahead = (score.unsqueeze(1) > score.unsqueeze(2)).sum(-1)  # experts that a token ranks before this one
        ids = torch.argsort(ahead, dim=1, stable=True)[:, : case["k"]]
        weight = RSF * p.gather(1, ids) / p.gather(1, ids).sum(1, keepdim=True)
        return _experts64(s, ids, weight), ids.to(torch.int32), weight
    rms = lambda v: torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + EPS)  # noqa: E731
    held = lambda v: v.to(torch.bfloat16).double()  # noqa: E731  what the next step reads is kept in BF16
    if op == "norm_in":
        x = s["x"].double()
        n = x / rms(x) * s["w"].double()
        return n, _grid64(held(n))
    y = s["y"].double()
    z = y / rms(y) * s["w"].double()
    if s["gate"] is not None:
        z = z * s["gate"].double()
    r = s["r"].double() + case["scale"] * z
    n = held(r) / rms(held(r)) * s["w_next"].double()
    return r, _grid64(held(n))
