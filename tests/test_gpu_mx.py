"""GPU parity of the MXFP4 operators against oracle/mx.py (float64).

Bitwise: codes, scale bytes, packed weights, read-back values.

Products are checked element by element against bounds that follow from the
arithmetic, u = 2^-24 (FP32) throughout:
* an FP32 sum of K exact products, in any order: (K + 8) u * sum |x||w|;
* h = silu(g) u known to delta = 1.1 |u| err_g + |silu(g)| err_u + (8 + |g|) 2u |h| (|silu'| < 1.1, and the hardware
  exponential and reciprocal are good to an ulp or two, the former on an argument rounded to u |g|), so its
  quantization may move by mx.grid_reach(h, delta), which moves f by reach . |w2|;
  FP32 noise of some 1e-6 crosses a rounding boundary for about one h in 1e5, by a step of some 0.3 of h's size:
  together with the rows' FP16 the relative error in the 2-norm stays near 1e-3 (checked: 4e-3);
* a pair row is FP16 under a power of two: 2^-11 of the value, or half a subnormal step, 2^(E - 25).
BF16 results add half an ulp, 2^-8 of the value."""

import numpy as np
import pytest
import torch

from gpu_cases import dev_bf16, pair_rows, say, to_np
from oracle import mx
from workloads import gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def bf16(a):
    """float array -> (values that BF16 holds, float64; bits)"""
    bits = gen.f32_to_bf16_bits(np.ascontiguousarray(a, dtype=np.float32))
    return gen.bf16_bits_to_f32(bits).astype(np.float64), bits


def draw(rng, rows, cols):
    return rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))


def special(x):
    """Rows and blocks where a quantizer can go wrong, written over x (float32) in place."""
    blocks = x.reshape(x.shape[0], -1, 32)
    pick = [np.zeros(32), np.full(32, -0.0), np.full(32, 2.0 ** -130), np.full(32, 1e-40),
            2.0 ** (np.arange(32) - 16.0), -np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5] * 4),
            np.array([7.99] + [5.0] * 31), np.full(32, 3.3e38), np.full(32, 2.0 ** -126)]
    for i, v in enumerate(pick):
        blocks[i % x.shape[0], (i * 3) % blocks.shape[1]] = v
    blocks[-1, -1, 5] = np.nan
    blocks[x.shape[0] // 2, 0, 31] = np.inf
    return x


@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (1, 6144, 0), (3, 64, 8), (17, 288, 24), (64, 256, 0),
                                           (129, 2080, 32), (5, 8224, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_bitwise(ops, rows, cols, pad, dtype):
    say(f"quantize {rows}x{cols}+{pad} {dtype}")
    rng = np.random.default_rng(rows * cols)
    x = draw(rng, rows, cols + pad).astype(np.float32)
    x[:, :cols] = special(np.ascontiguousarray(x[:, :cols]))
    if dtype == torch.bfloat16:
        v, bits = bf16(x)
        t = dev_bf16(bits)[:, :cols]
    else:
        v, t = x.astype(np.float64), torch.from_numpy(x).cuda()[:, :cols]
    codes, scales = ops.mxfp4_quantize(t)
    oc, ob = mx.quantize(v[:, :cols])
    pc, ps = mx.row_form(oc, ob)
    assert np.array_equal(to_np(scales), ps)
    assert np.array_equal(to_np(codes), pc)
    back = mx.dequantize(oc, ob)
    for out_dtype in (torch.float32, torch.bfloat16):
        got = ops.mxfp4_dequantize(codes, scales, cols, out_dtype)
        assert got.dtype == out_dtype
        assert np.array_equal(to_np(got.float()).astype(np.float64), back, equal_nan=True)
    wide = torch.full((rows, cols + 16), 7.0, dtype=torch.float32, device="cuda")
    ops.mxfp4_dequantize(codes, scales, cols, out=wide[:, :cols])
    assert np.array_equal(to_np(wide[:, :cols]).astype(np.float64), back, equal_nan=True)
    assert bool((wide[:, cols:] == 7.0).all())


def test_quantize_no_rows(ops):
    c, s = ops.mxfp4_quantize(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert tuple(c.shape) == (0, 128) and tuple(s.shape) == (0, 8)
    assert tuple(ops.mxfp4_dequantize(c, s, 64).shape) == (0, 64)


@pytest.mark.parametrize("batch,n,k", [(1, 1, 32), (2, 45, 288), (3, 64, 256), (1, 33, 608)])
def test_weights_packed(ops, batch, n, k):
    rng = np.random.default_rng(n * k)
    v, bits = bf16(special((draw(rng, batch * n, k) * 0.1).astype(np.float32)) if n > 1 else draw(rng, n, k))
    codes, scales, top = ops.mxfp4_quantize_weights(dev_bf16(bits).view(batch, n, k))
    canon_c, canon_s = [], []
    for b in range(batch):
        oc, ob = mx.quantize(v.reshape(batch, n, k)[b])
        pc, ps = mx.pack(oc, ob)
        assert np.array_equal(to_np(codes)[b], pc) and np.array_equal(to_np(scales)[b], ps)
        assert int(top[b]) == ob.max()
        canon_c.append(oc[:, 0::2] | (oc[:, 1::2] << 4))
        canon_s.append(ob)
    cc, cs = np.stack(canon_c).astype(np.uint8), np.stack(canon_s)
    uc, us = ops.mxfp4_unpack_weights(codes, scales, n, k)
    assert np.array_equal(to_np(uc), cc) and np.array_equal(to_np(us), cs)
    pc, ps, pt = ops.mxfp4_pack_weights(torch.from_numpy(cc).cuda(), torch.from_numpy(cs).cuda())
    assert torch.equal(pc, codes) and torch.equal(ps, scales) and torch.equal(pt, top)


def linear_case(seed, T, K, N):
    rng = np.random.default_rng(seed)
    x, xb = bf16(draw(rng, T, K))
    w, wb = bf16(draw(rng, N, K) * 0.05)
    return x, xb, w, wb


def check_linear(got, xq, wq, bf16_out):
    ref = xq @ wq.T
    bound = (xq.shape[1] + 8) * U * (np.abs(xq) @ np.abs(wq).T) + (2.0 ** -8 * np.abs(ref) if bf16_out else 0) + 1e-38
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan)
    worst = np.max(np.where(nan, 0, np.abs(got - ref) / np.where(nan, 1, bound)))
    print(f"  error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0


LINEAR = [(1, 32, 1), (1, 256, 33), (1, 2080, 1000), (2, 64, 31), (3, 6144, 96), (15, 288, 64), (16, 1024, 257),
          (17, 320, 40), (31, 96, 130), (32, 512, 32), (33, 544, 300), (64, 768, 512), (65, 1312, 70), (77, 2080, 1000),
          (128, 256, 256), (129, 800, 260), (255, 288, 511), (256, 1024, 256), (257, 544, 513), (384, 4096, 320),
          (515, 352, 1030), (1031, 288, 289),
          # every tile shape, with ragged last tiles and short and long reductions
          (20, 288, 16420), (400, 288, 4203), (390, 1568, 4200), (900, 320, 6203), (897, 1344, 6200), (1800, 288, 6507),
          (1797, 1888, 6504), (1797, 4128, 6504)]


@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear(ops, T, K, N):
    say(f"linear T={T} K={K} N={N}")
    x, xb, w, wb = linear_case(T * K + N, T, K, N)
    wc, wsc, _ = ops.mxfp4_quantize_weights(dev_bf16(wb)[None])
    codes, scales = ops.mxfp4_quantize(dev_bf16(xb))
    xq, wq = mx.rounded(x), mx.rounded(w)
    check_linear(to_np(ops.mxfp4_linear(codes, scales, wc[0], wsc[0], N, torch.float32)).astype(np.float64), xq, wq, False)
    wide = torch.full((T, N + 3), 7.0, dtype=torch.bfloat16, device="cuda")  # rows that no vector store can reach
    ops.mxfp4_linear(codes, scales, wc[0], wsc[0], N, y=wide[:, :N])
    check_linear(to_np(wide[:, :N].float()).astype(np.float64), xq, wq, True)
    assert bool((wide[:, N:] == 7.0).all())


@pytest.mark.parametrize("T", [1, 20, 300])
def test_linear_extremes(ops, T):
    """NaN blocks reach exactly their row or column; zero rows give zeros; huge and tiny scales meet."""
    K, N = 320, 80
    x, xb, w, wb = linear_case(T, T, K, N)
    x32, w32 = x.astype(np.float32), w.astype(np.float32)
    x32[T // 2, 40] = np.nan
    if T > 1:
        x32[0] = 0
        x32[T - 1] *= np.float32(2.0 ** 60)
    w32[7, 300] = np.inf
    w32[11] = 0
    w32[12] *= np.float32(2.0 ** -90)
    (x, xb), (w, wb) = bf16(x32), bf16(w32)
    wc, wsc, _ = ops.mxfp4_quantize_weights(dev_bf16(wb)[None])
    codes, scales = ops.mxfp4_quantize(dev_bf16(xb))
    got = to_np(ops.mxfp4_linear(codes, scales, wc[0], wsc[0], N, torch.float32)).astype(np.float64)
    check_linear(got, mx.rounded(x), mx.rounded(w), False)
    assert np.isnan(got[T // 2]).all() and np.isnan(got[:, 7]).all()
    assert not np.isnan(np.delete(np.delete(got, T // 2, 0), 7, 1)).any()


def test_linear_no_tokens_and_other_stream(ops):
    x, xb, w, wb = linear_case(5, 40, 288, 64)
    wc, wsc, _ = ops.mxfp4_quantize_weights(dev_bf16(wb)[None])
    c, s = ops.mxfp4_quantize(torch.empty((0, 288), dtype=torch.bfloat16, device="cuda"))
    assert tuple(ops.mxfp4_linear(c, s, wc[0], wsc[0], 64).shape) == (0, 64)
    xd = dev_bf16(xb)
    c, s = ops.mxfp4_quantize(xd)
    want = ops.mxfp4_linear(c, s, wc[0], wsc[0], 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c2, s2, y2 = torch.zeros_like(c), torch.zeros_like(s), torch.zeros_like(want)
    side.wait_stream(torch.cuda.current_stream())
    ops.mxfp4_quantize(xd, codes=c2, scales=s2, stream=side)
    ops.mxfp4_linear(c2, s2, wc[0], wsc[0], 64, y=y2, stream=side)
    side.synchronize()
    assert torch.equal(y2, want)


def routing(rng, T, E, k, kind):
    """topk_ids [T, k] and weights; kind: even, one (every token's first pick is expert 1), few (the last experts idle)."""
    ids = np.stack([rng.permutation(E if kind != "few" else max(k, E // 2))[:k] for _ in range(T)])
    if kind == "one":
        for row in ids:
            if 1 in row:
                row[row == 1] = row[0]
            row[0] = 1
    w = rng.uniform(0.05, 1.5, (T, k)).astype(np.float32)
    flat = ids.reshape(-1)
    counts = np.bincount(flat, minlength=E)
    return ids, w, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), np.argsort(flat, kind="stable").astype(np.int32)


def run_experts(ops, x_bits, w13_bits, w2_bits, ids, w, offsets, order, E, k, H, I):
    T = x_bits.shape[0]
    w13 = ops.mxfp4_quantize_weights(dev_bf16(w13_bits).view(E, 2 * I, H))[:2]
    w2 = ops.mxfp4_quantize_weights(dev_bf16(w2_bits).view(E, H, I))
    codes, scales = ops.mxfp4_quantize(dev_bf16(x_bits))
    # outputs and workspace start as garbage: nothing may depend on what they held
    po = torch.full((T * k, H), float("nan"), dtype=torch.float16, device="cuda")
    ps = torch.full((T * k,), float("nan"), dtype=torch.float32, device="cuda")
    ws = torch.full((max(ops.mxfp4_ffn_workspace_bytes(T, k, E, H, I), 1),), 0xFF, dtype=torch.uint8, device="cuda")
    ops.mxfp4_grouped_ffn(codes, scales, *w13, *w2, H, I, k, torch.from_numpy(offsets).cuda(),
                          torch.from_numpy(order).cuda(), torch.from_numpy(w).cuda(), po, ps, workspace=ws)
    return po, ps


EXPERTS = [(1, 4, 2, 64, 32, "even"), (1, 8, 8, 256, 128, "even"), (3, 16, 4, 288, 96, "few"), (16, 80, 8, 512, 256, "even"),
           (33, 8, 2, 256, 128, "one"), (64, 8, 2, 256, 128, "even"), (70, 4, 1, 96, 544, "one"),
           (150, 6, 3, 320, 160, "few"), (300, 4, 2, 544, 288, "one"), (513, 5, 2, 256, 96, "even"),
           # every tile shape of both stages
           (40, 48, 4, 1056, 1504, "few"), (512, 16, 4, 2752, 1408, "one"), (1024, 2, 2, 4096, 4096, "even")]


@pytest.mark.parametrize("T,E,k,H,I,kind", EXPERTS)
def test_experts(ops, T, E, k, H, I, kind):
    say(f"experts T={T} E={E} k={k} H={H} I={I} {kind}")
    rng = np.random.default_rng(T * H + I)
    x, xb = bf16(draw(rng, T, H))
    w13, b13 = bf16(rng.standard_normal((E, 2 * I, H)) * H ** -0.5)
    w2, b2 = bf16(rng.standard_normal((E, H, I)) * I ** -0.5)
    ids, w, offsets, order = routing(rng, T, E, k, kind)
    po, ps = run_experts(ops, xb, b13, b2, ids, w, offsets, order, E, k, H, I)
    got, scale = pair_rows(po, ps), to_np(ps).astype(np.float64)
    xq = mx.rounded(x)
    worst = off = norm = 0.0
    for e in range(E):
        p = order[offsets[e]: offsets[e + 1]]
        if p.size == 0:
            continue
        w13q, w2q, w2byte = mx.rounded(w13[e]), mx.rounded(w2[e]), mx.quantize(w2[e])[1].max()
        xe = xq[p // k]
        z, mag = xe @ w13q.T, np.abs(xe) @ np.abs(w13q).T
        g, u = z[:, :I], z[:, I:]
        eg, eu = (H + 8) * U * mag[:, :I], (H + 8) * U * mag[:, I:]
        s = mx.silu(g)
        h = s * u
        hq, reach = mx.grid_reach(h, 1.1 * np.abs(u) * eg + np.abs(s) * eu + (8 + np.abs(g)) * 2 * U * np.abs(h))
        wp = w.reshape(-1)[p].astype(np.float64)[:, None]
        ref = wp * (hq @ w2q.T)
        top = (np.abs(hq) + reach) @ np.abs(w2q).T
        bound = wp * (reach @ np.abs(w2q).T + (I + 8) * U * top)
        E_ = mx.pair_exponent(wp[:, 0], mx.quantize(h)[1].max(1), np.full(p.size, w2byte), I)
        assert (np.abs(np.log2(scale[p]) - E_) <= 1).all() and (np.log2(scale[p]) == np.rint(np.log2(scale[p]))).all()
        bound = bound + 2.0 ** -11 * (np.abs(ref) + bound) + 2.0 ** (E_[:, None] + 1 - 25)
        worst = max(worst, float(np.max(np.abs(got[p] - ref) / bound)))
        off, norm = off + float(((got[p] - ref) ** 2).sum()), norm + float((ref ** 2).sum())
    print(f"  error / bound {worst:.3f}, rel-L2 {(off / norm) ** 0.5:.2e}", flush=True)
    assert worst <= 1.0 and (off / norm) ** 0.5 <= 4e-3


@pytest.mark.parametrize("T", [2, 200])
def test_experts_extremes(ops, T):
    """A token with a NaN gives NaN pair rows and touches no other; a zero token gives zero rows, also under a large
    routing weight; the combine reads the rows."""
    E, k, H, I = 4, 2, 288, 96
    rng = np.random.default_rng(T)
    x32 = draw(rng, T, H).astype(np.float32)
    x32[0, 3] = np.nan
    x32[1] = 0
    x, xb = bf16(x32)
    _, b13 = bf16(rng.standard_normal((E, 2 * I, H)) * H ** -0.5)
    _, b2 = bf16(rng.standard_normal((E, H, I)) * I ** -0.5)
    ids, w, offsets, order = routing(rng, T, E, k, "even")
    w[1] = 1e6
    po, ps = run_experts(ops, xb, b13, b2, ids, w, offsets, order, E, k, H, I)
    got = pair_rows(po, ps)
    assert np.isnan(got[:k]).all() and (got[k:2 * k] == 0).all() and np.isfinite(got[k:]).all()
    y = to_np(ops.moe_combine(po, ps, T, k, torch.float32)).astype(np.float64)
    assert np.allclose(y[1:], got.reshape(T, k, H).sum(1)[1:], rtol=1e-5, atol=1e-5)
    again = run_experts(ops, xb, b13, b2, ids, w, offsets, order, E, k, H, I)
    assert torch.equal(again[0].view(torch.int16), po.view(torch.int16)) and torch.equal(again[1], ps)


def test_experts_no_tokens(ops):
    E, k, H, I = 4, 2, 64, 32
    z = np.zeros((E * 2 * I, H), np.float32)
    po, ps = run_experts(ops, np.zeros((0, H), np.uint16), bf16(z)[1], bf16(np.zeros((E * H, I)))[1], None,
                         np.zeros((0, k), np.float32), np.zeros(E + 1, np.int32), np.zeros(0, np.int32), E, k, H, I)
    assert po.numel() == 0 and ps.numel() == 0


def test_binding_refusals(ops):
    """What the binding refuses of tensors on the device, before anything is enqueued."""
    x = torch.zeros((4, 288), dtype=torch.bfloat16, device="cuda")
    c, s = ops.mxfp4_quantize(x)
    wc, ws, top = ops.mxfp4_quantize_weights(torch.zeros((2, 40, 288), dtype=torch.bfloat16, device="cuda"))

    def raises(kind, match, f):
        with pytest.raises(kind, match=match):
            f()

    raises(TypeError, "codes must be torch.uint8, got torch.float32", lambda: ops.mxfp4_quantize(x, codes=c.float()))
    raises(ValueError, r"codes must have shape \(4, 256\), got \(4, 128\)", lambda: ops.mxfp4_quantize(x, codes=c[:, :128]))
    raises(ValueError, "unit column stride", lambda: ops.mxfp4_quantize(x.t()))
    raises(ops.MoEError, "MOE_ERR_SHAPE.*multiple of 32", lambda: ops.mxfp4_quantize(x[:, :40]))
    raises(ops.MoEError, "MOE_ERR_ALIGN", lambda: ops.mxfp4_quantize(x[:, 1:33]))
    raises(TypeError, "output type", lambda: ops.mxfp4_dequantize(c, s, 288, torch.float16))
    raises(ValueError, r"out must have shape \(4, 288\)", lambda: ops.mxfp4_dequantize(c, s, 288, out=x[:2]))
    raises(ValueError, "w_codes must have shape", lambda: ops.mxfp4_linear(c, s, wc[0], ws[0], 72))
    raises(ValueError, "x_codes must have shape", lambda: ops.mxfp4_linear(c[:, :128], s, wc[0], ws[0], 40))
    raises(ValueError, "codes must be contiguous", lambda: ops.mxfp4_quantize(x, codes=c.t().contiguous().t()))
    off, srt = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    tw = torch.zeros((4, 1), device="cuda")
    bad = torch.zeros((4, 2), device="cuda")
    w2 = ops.mxfp4_quantize_weights(torch.zeros((2, 288, 32), dtype=torch.bfloat16, device="cuda"))
    w13 = ops.mxfp4_quantize_weights(torch.zeros((2, 64, 288), dtype=torch.bfloat16, device="cuda"))[:2]
    raises(ValueError, "topk_w must have shape", lambda: ops.mxfp4_grouped_ffn(c, s, *w13, *w2, 288, 32, 1, off, srt, bad))
    raises(ops.MoEError, "MOE_ERR_WORKSPACE",
           lambda: ops.mxfp4_grouped_ffn(c, s, *w13, *w2, 288, 32, 1, off, srt, tw,
                                         workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")))
    raises(ValueError, "residual must have shape", lambda: ops.moe_norm_out(x, x[:2]))
    raises(ValueError, r"gate must be \[T, 1\]", lambda: ops.moe_norm_out(x, x, gate=x[:2]))
    raises(ValueError, "need w_next", lambda: ops.moe_norm_out(x, x, quantize=True))
    raises(ops.MoEError, "MOE_ERR_NULL.*neither n nor codes", lambda: ops.moe_norm_in(x, x[0], n=False))
    raises(ops.MoEError, "MOE_ERR_SHAPE.*row stride", lambda: ops.moe_norm_in(x[:1].expand(4, 288), x[0]))
