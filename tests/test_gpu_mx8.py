"""GPU parity of the MXFP8 operators against oracle/mx8.py (float64).

Bitwise: codes, scale bytes, read-back values, the norms and their MXFP8 forms.

Products are checked element by element, u = 2^-24 (FP32):
* an FP32 sum of K exact products, in any order: (K + 8) u * sum |x||w|;
* where the result is not FP32, the matrix instruction may drop what lies 16 binades below the largest product of a
  block (and the largest is known to within a factor of two): 32 products, 2^-15 of the largest each, so 2^-10 of every
  block's largest |x| times its largest |w|;
* the epilogue: bias and residual one FP32 rounding each; the activations' slopes are under 1.13, and their own errors,
  from the hardware's exponential and reciprocal on a rounded argument, are (8 + 4 |z| + 4 |z|^3) 2 u |act(z)| (the cube for
  the tanh form's argument) or, by erf, 4 u |z|;
* h = silu(g) u known to delta (as for MXFP4) may move by mx8.grid_reach(h, delta);
* a pair row is FP16 under a power of two: 2^-11 of the value, or half a subnormal step, 2^(E - 25).  In the 2-norm:
  g and u are off by some d = 1e-5 of their size (the dropped products), h by sqrt(2) d; an element of h then rounds to
  the other side with probability 0.8 sqrt(2) d / s for E4M3's spacing s (2^-3 to 2^-4 of the value), by s, so q(h) and f
  are off by sqrt(0.8 sqrt(2) d s) = 1e-3, beside 2.1e-4 for FP16; twice that is allowed;
BF16 results add half an ulp, 2^-8 of the value; in the 2-norm that is at most 2^-8 / sqrt(3) = 2.3e-3."""

import math

import numpy as np
import pytest
import torch

from gpu_cases import dev_bf16, pair_rows, say, to_np
from oracle import mx, mx8
from oracle import norm as onorm
from test_gpu_mx import bf16, draw, routing, special

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def f64(t):
    return to_np(t.float()).astype(np.float64)


def block_max(x):
    return np.abs(x).reshape(x.shape[0], -1, 32).max(-1)


def sum_bound(x, w, rough):
    """Bound of the error of x @ w.T, elementwise."""
    b = (x.shape[1] + 8) * U * (np.abs(x) @ np.abs(w).T)
    return b + 2.0 ** -10 * (block_max(x) @ block_max(w).T) if rough else b


# ---------------------------------------------------------------------------------------------


def special8(x):
    """As special, with borders of E4M3."""
    x = special(x)
    blocks = x.reshape(x.shape[0], -1, 32)
    pick = [np.array([448.0] + [2.0 ** -9 * (k + 0.5) for k in range(31)]),
            np.array([300.0] + [(1 + (2 * k + 1) / 16) * 2.0 ** (k % 9 - 6) for k in range(31)]),
            np.array([511.0, 464.0, 480.0, 463.9, -449.0] + [-0.0] * 27), np.full(32, 2.0 ** -118), np.full(32, -2.0 ** -135)]
    for i, v in enumerate(pick):
        blocks[(i + 1) % x.shape[0], (i * 5 + 1) % blocks.shape[1]] = v
    return x


@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (1, 6144, 0), (3, 64, 8), (17, 288, 24), (64, 256, 0),
                                           (129, 2080, 32), (5, 8224, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_bitwise(ops, rows, cols, pad, dtype):
    say(f"quantize {rows}x{cols}+{pad} {dtype}")
    rng = np.random.default_rng(rows * cols)
    x = draw(rng, rows, cols + pad).astype(np.float32)
    x[:, :cols] = special8(np.ascontiguousarray(x[:, :cols]))
    if dtype == torch.bfloat16:
        v, bits = bf16(x)
        t = dev_bf16(bits)[:, :cols]
    else:
        v, t = x.astype(np.float64), torch.from_numpy(x).cuda()[:, :cols]
    codes, scales = ops.mxfp8_quantize(t)
    oc, ob = mx8.quantize(v[:, :cols])
    pc, ps = mx8.row_form(oc, ob)
    assert np.array_equal(to_np(scales), ps)
    assert np.array_equal(to_np(codes), pc)
    back = mx8.dequantize(oc, ob)
    got = ops.mxfp8_dequantize(codes, scales, cols, torch.float32)
    assert np.array_equal(f64(got), back, equal_nan=True)
    low = ops.mxfp8_dequantize(codes, scales, cols)
    assert low.dtype == torch.bfloat16 and torch.equal(low.view(torch.int16)[~got.isnan()],
                                                       got.to(torch.bfloat16).view(torch.int16)[~got.isnan()])
    assert bool(low.isnan().eq(got.isnan()).all())
    wide = torch.full((rows, cols + 16), 7.0, dtype=torch.float32, device="cuda")
    ops.mxfp8_dequantize(codes, scales, cols, out=wide[:, :cols])
    assert np.array_equal(f64(wide[:, :cols]), back, equal_nan=True) and bool((wide[:, cols:] == 7.0).all())


def test_every_bf16_value(ops):
    """Every BF16 bit pattern as a block's second element, under a first of 2^0 .. 2^3 times it or of a fixed size."""
    bits = np.arange(65536, dtype=np.uint16).reshape(-1, 1)
    x = np.zeros((65536, 32), np.uint16)
    x[:, 1] = bits[:, 0]
    x[:, 0] = 0x4380 + (bits[:, 0] & 0x7F)  # 256 .. 511
    from workloads import gen

    v = gen.bf16_bits_to_f32(x).astype(np.float64)
    codes, scales = ops.mxfp8_quantize(dev_bf16(x))
    oc, ob = mx8.quantize(v)
    assert np.array_equal(to_np(codes)[:, :32], oc) and np.array_equal(to_np(scales)[:, :1], ob)


def test_quantize_no_rows(ops):
    c, s = ops.mxfp8_quantize(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert tuple(c.shape) == (0, 256) and tuple(s.shape) == (0, 8)
    assert tuple(ops.mxfp8_dequantize(c, s, 64).shape) == (0, 64)


@pytest.mark.parametrize("T,H,pad", [(1, 32, 0), (3, 288, 8), (5, 992, 3), (2, 2048, 0), (3, 4128, 0), (4, 6144, 0),
                                     (2, 16384, 8), (2050, 1056, 0), (2049, 1984, 0)])
def test_norms(ops, T, H, pad):
    """n and r' are the float64 results, rounded to FP32 and to BF16; the MXFP8 form is mxfp8_quantize of n, bit for bit, with and
    without n.

    Sums are FP64 over FP32 sums of four squares: one rounding of the innermost product (of FP32 y; a BF16 value's square
    is exact) and three of the sums, 4 u of a row's mean square at most, so 1 / rms is good to 2 u and a product with it
    to 2^-23, beside u for the FP32 value and half a BF16 step.  The roundings of a row's groups are independent, and their mean is 100 times
    smaller: less than one result in 10^5 may lie that close to a border."""
    say(f"norms {T}x{H}+{pad}")
    rng = np.random.default_rng(H)
    (xv, xb), (yv, yb) = (bf16(rng.standard_normal((T, H + pad)) * np.exp(rng.standard_normal((T, 1)))) for _ in range(2))
    xv, yv, x, y = xv[:, :H], yv[:, :H], dev_bf16(xb)[:, :H], dev_bf16(yb)[:, :H]
    wv, wb = bf16(1 + 0.3 * rng.standard_normal(H))
    w = dev_bf16(wb)
    y32 = (yv * (1 + 1e-4 * rng.standard_normal((T, H)))).astype(np.float32)

    def check_codes(n, codes, scales):
        qc, qs = ops.mxfp8_quantize(n)
        assert torch.equal(codes, qc) and torch.equal(scales, qs)

    def close(got, ref, z):
        g = f64(got)
        half = np.ldexp(1.0, np.maximum(np.frexp(np.maximum(np.abs(g), np.abs(ref)))[1], -125) - 9)
        assert (np.abs(g - ref) <= half + U * np.abs(ref) + 2.0 ** -23 * np.abs(z)).all()
        differ = int((g != bf16(ref)[0]).sum())
        print(f"  {differ} of {ref.size} not correctly rounded", flush=True)
        assert differ <= 1 + ref.size // 100000

    n, codes, scales = ops.moe_norm_in_mxfp8(x, w, 1e-6)
    ref = onorm.norm(xv, wv, np.float32(1e-6))
    close(n, ref, ref)
    check_codes(n, codes, scales)
    skipped = ops.moe_norm_in_mxfp8(x, w, 1e-6, n=False)
    assert skipped[0] is None and torch.equal(skipped[1], codes) and torch.equal(skipped[2], scales)
    for yt, ym in ((y, yv), (torch.from_numpy(y32).cuda(), y32.astype(np.float64))):
        for gate, gm in ((None, None), (w[None], wv[None]), (x[:, :1], xv[:, :1]), (x, xv)):
            r, n, codes, scales = ops.moe_norm_out_mxfp8(yt, x, w, w, gate=gate, residual_scale=0.5)
            ref = onorm.residual(ym, xv, wv, gm, 0.5, np.float32(1e-6))
            close(r, ref, ref - xv)
            ref = onorm.norm(f64(r), wv, np.float32(1e-6))  # of the residual that is kept
            close(n, ref, ref)
            check_codes(n, codes, scales)
    r, n, codes, scales = ops.moe_norm_out_mxfp8(y, x, None, w, n=False, codes=torch.full_like(codes, 99),
                                                 scales=torch.full_like(scales, 99))
    rm = bf16(xv + yv)[0]
    assert n is None and np.array_equal(f64(r), rm)  # a sum of two BF16 values
    check_codes(ops.moe_norm_in_mxfp8(r, w)[0], codes, scales)
    inplace = x.clone()
    ops.moe_norm_out_mxfp8(y, inplace, None, w, out=inplace)
    assert torch.equal(inplace, r)


def test_norms_extremes(ops):
    """NaN and infinities stay in their rows; zero rows give zeros; huge and tiny rows do not overflow the sums."""
    H = 288
    x = torch.randn(6, H, device="cuda").to(torch.bfloat16)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    x[0, 7], x[1, 9], x[2], x[3], x[4] = float("nan"), float("inf"), 0.0, 1e30, 1e-30
    n, codes, scales = ops.moe_norm_in_mxfp8(x, w, 1e-6)
    v = ops.mxfp8_dequantize(codes, scales, H)
    assert bool(n[0].isnan().all()) and bool(v[0].isnan().all()) and bool(n[1, 9].isnan())
    assert bool((n[2] == 0).all()) and bool((v[2] == 0).all()) and bool((n[3] == 1).all()) and bool((v[3] == 1).all())
    assert not bool(n[2:].isnan().any()) and torch.equal(n[5], ops.moe_norm_in_mxfp8(x[5:], w, 1e-6)[0][0])


# ---------------------------------------------------------------------------------------------


def act64(name, z):
    if name == "relu":
        return np.maximum(z, 0.0), np.zeros_like(z)
    if name == "silu":
        a = mx.silu(z)
        return a, (8 + 4 * np.abs(z)) * 2 * U * np.abs(a)
    if name == "gelu":
        a = 0.5 * z * (1.0 + np.vectorize(math.erf)(z / math.sqrt(2.0)))
        return a, 4 * U * np.abs(z)
    if name == "gelu_tanh":
        u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
        a = z / (1.0 + np.exp(np.minimum(-2.0 * u, 700.0)))
        return a, (8 + 4 * np.abs(z) + 4 * np.abs(z) ** 3) * 2 * U * np.abs(a)
    return z, np.zeros_like(z)


def check_linear(got, xq, wq, bf16_out, bias=None, act=None, residual=None):
    z, bound = xq @ wq.T, sum_bound(xq, wq, bf16_out)
    if bias is not None:
        z = z + bias
        bound = bound + U * np.abs(z)
    ref, own = act64(act, z)
    bound = (1.13 if act else 1.0) * bound + own
    if residual is not None:
        ref = ref + residual
        bound = bound + U * np.abs(ref)
    bound = bound + (2.0 ** -8 * (np.abs(ref) + bound) if bf16_out else U * np.abs(ref)) + 1e-37
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan)
    d = np.where(nan, 0, got - np.where(nan, 0, ref))
    worst = np.max(np.abs(d) / np.where(nan, 1, bound))
    off = float(np.sqrt((d ** 2).sum() / max((np.where(nan, 0, ref) ** 2).sum(), 1e-300)))
    print(f"  error / bound {worst:.3f}, rel-L2 {off:.2e}", flush=True)
    assert worst <= 1.0
    if bf16_out and ref.size > 1000:
        assert off <= 2.4e-3


def linear_case(seed, T, K, N):
    rng = np.random.default_rng(seed)
    x, xb = bf16(draw(rng, T, K))
    w, wb = bf16(draw(rng, N, K) * 0.05)
    return rng, x, xb, w, wb


LINEAR = [(1, 32, 1), (1, 256, 33), (1, 2080, 1000), (2, 64, 31), (3, 6144, 96), (15, 288, 64), (16, 1024, 257),
          (17, 320, 40), (31, 96, 130), (32, 512, 32), (33, 544, 300), (64, 768, 512), (65, 1312, 70), (77, 2080, 1000),
          (128, 256, 256), (129, 800, 260), (255, 288, 511), (256, 1024, 256), (257, 544, 513), (384, 4096, 320),
          (515, 352, 1030), (1031, 288, 289),
          # every tile shape, with ragged last tiles and short and long reductions
          (20, 288, 16420), (400, 288, 4203), (390, 1568, 4200), (900, 320, 6203), (897, 1344, 6200), (1800, 288, 6507),
          (1797, 1888, 6504), (1797, 4128, 6504), (1200, 2080, 600), (1100, 96, 700)]


@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear(ops, T, K, N):
    say(f"linear T={T} K={K} N={N}")
    rng, x, xb, w, wb = linear_case(T * K + N, T, K, N)
    wc, wsc, _ = ops.mxfp4_quantize_weights(dev_bf16(wb)[None])
    codes, scales = ops.mxfp8_quantize(dev_bf16(xb))
    xq, wq = mx8.rounded(x), mx.rounded(w)
    b, bb = bf16(rng.standard_normal(N))
    r, rb = bf16(rng.standard_normal((T, N + 5)))
    bias, res = dev_bf16(bb), dev_bf16(rb)[:, :N]
    check_linear(f64(ops.mxfp8_linear(codes, scales, wc[0], wsc[0], N, torch.float32)), xq, wq, False)
    wide = torch.full((T, N + 3), 7.0, dtype=torch.bfloat16, device="cuda")  # rows that no vector store can reach
    ops.mxfp8_linear(codes, scales, wc[0], wsc[0], N, bias=bias, residual=res, y=wide[:, :N])
    check_linear(f64(wide[:, :N]), xq, wq, True, b, None, r[:, :N])
    assert bool((wide[:, N:] == 7.0).all())
    big = T * K * N > 1e9
    for act in ("silu",) if big else ("relu", "silu", "gelu", "gelu_tanh"):
        check_linear(f64(ops.mxfp8_linear(codes, scales, wc[0], wsc[0], N, torch.float32, bias=bias, activation=act,
                                          residual=res)), xq, wq, False, b, act, r[:, :N])
    check_linear(f64(ops.mxfp8_linear(codes, scales, wc[0], wsc[0], N, activation="gelu_tanh")), xq, wq, True, None,
                 "gelu_tanh")


@pytest.mark.parametrize("T,K,N", [(1, 288, 80), (5, 256, 33), (70, 544, 130), (300, 288, 517), (800, 1056, 6160)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_in_place(ops, T, K, N, dtype):
    """y is the residual: the same result as into another tensor, in every shape of tile."""
    rng, x, xb, w, wb = linear_case(T + N, T, K, N)
    wc, wsc, _ = ops.mxfp4_quantize_weights(dev_bf16(wb)[None])
    codes, scales = ops.mxfp8_quantize(dev_bf16(xb))
    r = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).cuda().to(dtype)
    want = ops.mxfp8_linear(codes, scales, wc[0], wsc[0], N, dtype, residual=r)
    assert ops.mxfp8_linear(codes, scales, wc[0], wsc[0], N, residual=r, y=r) is not None
    assert torch.equal(r, want)
    other = torch.bfloat16 if dtype == torch.float32 else torch.float32  # a residual of the other type
    r2 = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).cuda().to(other)
    got = ops.mxfp8_linear(codes, scales, wc[0], wsc[0], N, dtype, residual=r2)
    check_linear(f64(got), mx8.rounded(x), mx.rounded(w), dtype == torch.bfloat16, None, None, f64(r2))


@pytest.mark.parametrize("T", [1, 20, 300])
def test_linear_extremes(ops, T):
    """NaN blocks reach exactly their row or column; zero rows give zeros; huge and tiny scales meet."""
    K, N = 320, 80
    _, x, xb, w, wb = linear_case(T, T, K, N)
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
    codes, scales = ops.mxfp8_quantize(dev_bf16(xb))
    got = f64(ops.mxfp8_linear(codes, scales, wc[0], wsc[0], N, torch.float32))
    check_linear(got, mx8.rounded(x), mx.rounded(w), False)
    assert np.isnan(got[T // 2]).all() and np.isnan(got[:, 7]).all()
    assert not np.isnan(np.delete(np.delete(got, T // 2, 0), 7, 1)).any()
    relu = f64(ops.mxfp8_linear(codes, scales, wc[0], wsc[0], N, torch.float32, activation="relu"))
    assert np.array_equal(np.isnan(relu), np.isnan(got)) and (relu[~np.isnan(relu)] >= 0).all()


@pytest.mark.parametrize("T,K,N", [(1, 6144, 64), (40, 6144, 64), (300, 6144, 300)])
def test_linear_outliers_in_fp32(ops, T, K, N):
    """Channels of 300 times the rest's size: FP32 results stay FP32 sums (dropping the small products would leave 7e-5)."""
    rng, x, xb, w, wb = linear_case(T, T, K, N)
    x32 = x.astype(np.float32)
    x32[:, 5::64] *= np.float32(300.0)
    x, xb = bf16(x32)
    wc, wsc, _ = ops.mxfp4_quantize_weights(dev_bf16(wb)[None])
    codes, scales = ops.mxfp8_quantize(dev_bf16(xb))
    xq, wq = mx8.rounded(x), mx.rounded(w)
    got, ref = f64(ops.mxfp8_linear(codes, scales, wc[0], wsc[0], N, torch.float32)), xq @ wq.T
    check_linear(got, xq, wq, False)
    off = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    print(f"  rel-L2 {off:.2e}")
    assert off <= 1e-6


def test_linear_no_tokens_and_other_stream(ops):
    _, x, xb, w, wb = linear_case(5, 40, 288, 64)
    wc, wsc, _ = ops.mxfp4_quantize_weights(dev_bf16(wb)[None])
    c, s = ops.mxfp8_quantize(torch.empty((0, 288), dtype=torch.bfloat16, device="cuda"))
    assert tuple(ops.mxfp8_linear(c, s, wc[0], wsc[0], 64).shape) == (0, 64)
    xd = dev_bf16(xb)
    c, s = ops.mxfp8_quantize(xd)
    want = ops.mxfp8_linear(c, s, wc[0], wsc[0], 64, residual=xd[:, :64])
    c2, s2, y2 = torch.zeros_like(c), torch.zeros_like(s), torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ops.mxfp8_quantize(xd, codes=c2, scales=s2, stream=side)
    ops.mxfp8_linear(c2, s2, wc[0], wsc[0], 64, residual=xd[:, :64], y=y2, stream=side)
    side.synchronize()
    assert torch.equal(y2, want)


# ---------------------------------------------------------------------------------------------


def run_experts(ops, x_bits, w13_bits, w2_bits, w, offsets, order, E, k, H, I):
    T = x_bits.shape[0]
    w13 = ops.mxfp4_quantize_weights(dev_bf16(w13_bits).view(E, 2 * I, H))[:2]
    w2 = ops.mxfp4_quantize_weights(dev_bf16(w2_bits).view(E, H, I))
    codes, scales = ops.mxfp8_quantize(dev_bf16(x_bits))
    # outputs and workspace start as garbage: nothing may depend on what they held
    po = torch.full((T * k, H), float("nan"), dtype=torch.float16, device="cuda")
    ps = torch.full((T * k,), float("nan"), dtype=torch.float32, device="cuda")
    ws = torch.full((max(ops.mxfp8_ffn_workspace_bytes(T, k, E, H, I), 1),), 0xFF, dtype=torch.uint8, device="cuda")
    ops.mxfp8_grouped_ffn(codes, scales, *w13, *w2, H, I, k, torch.from_numpy(offsets).cuda(),
                          torch.from_numpy(order).cuda(), torch.from_numpy(w).cuda(), po, ps, workspace=ws)
    return po, ps


def expert64(xe, w13q, w2q, I, rough):
    """One expert's f for rows xe, a bound of its error, and h (before its rounding)."""
    z, b = xe @ w13q.T, sum_bound(xe, w13q, rough)
    g, u, eg, eu = z[:, :I], z[:, I:], b[:, :I], b[:, I:]
    s = mx.silu(g)
    h = s * u
    hq, reach = mx8.grid_reach(h, 1.1 * np.abs(u) * eg + np.abs(s) * eu + (8 + np.abs(g)) * 2 * U * np.abs(h))
    f = hq @ w2q.T
    return f, reach @ np.abs(w2q).T + sum_bound(np.abs(hq) + reach, w2q, rough), h


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
    po, ps = run_experts(ops, xb, b13, b2, w, offsets, order, E, k, H, I)
    got, scale = pair_rows(po, ps), to_np(ps).astype(np.float64)
    xq = mx8.rounded(x)
    worst = off = norm = 0.0
    for e in range(E):
        p = order[offsets[e]: offsets[e + 1]]
        if p.size == 0:
            continue
        w2q, w2byte = mx.rounded(w2[e]), mx.quantize(w2[e])[1].max()
        f, bound, h = expert64(xq[p // k], mx.rounded(w13[e]), w2q, I, True)
        wp = w.reshape(-1)[p].astype(np.float64)[:, None]
        ref, bound = wp * f, wp * bound
        E_ = mx8.pair_exponent(wp[:, 0], mx8.quantize(h)[1].max(1), np.full(p.size, w2byte), I)
        assert (np.abs(np.log2(scale[p]) - E_) <= 1).all() and (np.log2(scale[p]) == np.rint(np.log2(scale[p]))).all()
        bound = bound + 2.0 ** -11 * (np.abs(ref) + bound) + 2.0 ** (E_[:, None] + 1 - 25)
        worst = max(worst, float(np.max(np.abs(got[p] - ref) / bound)))
        off, norm = off + float(((got[p] - ref) ** 2).sum()), norm + float((ref ** 2).sum())
    print(f"  error / bound {worst:.3f}, rel-L2 {(off / norm) ** 0.5:.2e}", flush=True)
    assert worst <= 1.0 and (off / norm) ** 0.5 <= 2e-3


@pytest.mark.parametrize("T", [2, 200])
def test_experts_extremes(ops, T):
    """A token with a NaN gives NaN pair rows and touches no other; a zero token gives zero rows, also under a large
    routing weight; the combine reads the rows; a second call gives the same bits."""
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
    po, ps = run_experts(ops, xb, b13, b2, w, offsets, order, E, k, H, I)
    got = pair_rows(po, ps)
    assert np.isnan(got[:k]).all() and (got[k:2 * k] == 0).all() and np.isfinite(got[k:]).all()
    y = f64(ops.moe_combine(po, ps, T, k, torch.float32))
    assert np.allclose(y[1:], got.reshape(T, k, H).sum(1)[1:], rtol=1e-5, atol=1e-5)
    again = run_experts(ops, xb, b13, b2, w, offsets, order, E, k, H, I)
    assert torch.equal(again[0].view(torch.int16), po.view(torch.int16)) and torch.equal(again[1], ps)


def test_experts_no_tokens(ops):
    E, k, H, I = 4, 2, 64, 32
    z = np.zeros((E * 2 * I, H), np.float32)
    po, ps = run_experts(ops, np.zeros((0, H), np.uint16), bf16(z)[1], bf16(np.zeros((E * H, I)))[1],
                         np.zeros((0, k), np.float32), np.zeros(E + 1, np.int32), np.zeros(0, np.int32), E, k, H, I)
    assert po.numel() == 0 and ps.numel() == 0


# ---------------------------------------------------------------------------------------------


def test_binding_refusals(ops):
    """What the binding refuses of tensors on the device, before anything is enqueued."""
    x = torch.zeros((4, 288), dtype=torch.bfloat16, device="cuda")
    c, s = ops.mxfp8_quantize(x)
    wc, ws, _ = ops.mxfp4_quantize_weights(torch.zeros((2, 40, 288), dtype=torch.bfloat16, device="cuda"))

    def raises(kind, match, f):
        with pytest.raises(kind, match=match):
            f()

    raises(ValueError, r"codes must have shape \(4, 512\), got \(4, 256\)", lambda: ops.mxfp8_quantize(x, codes=c[:, :256]))
    raises(ops.MoEError, "MOE_ERR_SHAPE.*multiple of 32", lambda: ops.mxfp8_quantize(x[:, :40]))
    raises(TypeError, "output type", lambda: ops.mxfp8_dequantize(c, s, 288, torch.float16))
    lin = lambda **kw: ops.mxfp8_linear(c, s, wc[0], ws[0], 40, **kw)  # noqa: E731
    raises(ValueError, "activation must be one of", lambda: lin(activation="tanh"))
    raises(ValueError, r"bias must have shape \(40,\)", lambda: lin(bias=x[0]))
    raises(TypeError, "bias must be torch.bfloat16", lambda: lin(bias=torch.zeros(40, device="cuda")))
    raises(ValueError, r"residual must have shape \(4, 40\)", lambda: lin(residual=x))
    raises(TypeError, "residual must be a tensor of torch.bfloat16 or torch.float32",
           lambda: lin(residual=torch.zeros((4, 40), dtype=torch.float16, device="cuda")))
    raises(ValueError, "x_codes must have shape", lambda: ops.mxfp8_linear(*ops.mxfp4_quantize(x), wc[0], ws[0], 40))
    f = torch.zeros((4, 40), device="cuda")
    raises(ops.MoEError, "MOE_ERR_SHAPE.*type and stride",
           lambda: lin(residual=f, y=f.view(torch.bfloat16).view(-1)[:160].view(4, 40)))
    raises(TypeError, "w_next must be", lambda: ops.moe_norm_out_mxfp8(x, x, None, None))
    raises(ValueError, "w_router_bf16 must have shape",
           lambda: ops.mxfp8_moe_layer(x, x[:, :32], s, 1, 1.0, wc, ws, wc, ws))
