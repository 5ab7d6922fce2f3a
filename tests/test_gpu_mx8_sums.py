"""The MXFP8 products' sums are FP32 sums in every kernel, whatever type their results have.

Small products beside large ones that cancel: a block's two largest products are 1536 and -1536, the others multiples of
2^-10, some 20 binades below.  Every partial sum, in any order, is a multiple of 2^-10 and under 2^14, which FP32 holds
exactly, so the only rounding left is that of the result."""

import numpy as np
import pytest
import torch

from gpu_cases import dev_bf16, pair_rows, say, to_np
from oracle import mx, mx8
from test_gpu_mx import bf16, draw, routing
from test_gpu_mx8 import EXPERTS as ALL_EXPERTS
from test_gpu_mx8 import LINEAR, expert64, f64, linear_case, run_experts, sum_bound

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -9  # E4M3's least step


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def cancelling_rows(rng, T, K):
    """x [T, K]: multiples of 2^-9, up to 14; one block of a row starts with 256, 256, the others with zeros."""
    x = TINY * rng.integers(-14, 15, (T, K // 32, 32))
    x[:, :, 2] = 14 * TINY  # 448 steps of the block
    x[:, :, :2] = 0
    x[np.arange(T), (np.arange(T) * 7 + 3) % (K // 32), :2] = 256
    return x.reshape(T, K)


def cancelling_weights(rng, N, K):
    """w [N, K]: E2M1 values; every block starts with 6, -6."""
    w = rng.choice([-4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4], (N, K // 32, 32))
    w[:, :, 0], w[:, :, 1] = 6, -6
    return w.reshape(N, K)


@pytest.mark.parametrize("T,K,N", [c for c in LINEAR if c[1] >= 64] + [(1, 288, 50000), (16, 288, 70000), (64, 544, 65600)])
def test_linear_small_products(ops, T, K, N):
    say(f"small products, linear T={T} K={K} N={N}")
    rng = np.random.default_rng(T + K + N)
    (x, xb), (w, wb) = bf16(cancelling_rows(rng, T, K)), bf16(cancelling_weights(rng, N, K))
    assert np.array_equal(mx8.rounded(x), x) and np.array_equal(mx.rounded(w), w)
    wc, ws, _ = ops.mxfp4_quantize_weights(dev_bf16(wb)[None])
    codes, scales = ops.mxfp8_quantize(dev_bf16(xb))
    ref = x @ w.T
    for dtype in (torch.float32, torch.bfloat16):
        got = f64(ops.mxfp8_linear(codes, scales, wc[0], ws[0], N, dtype))
        assert np.array_equal(got, ref if dtype == torch.float32 else bf16(ref)[0]), dtype


EXPERTS = [(1, 4, 2, 96, 64), (16, 8, 2, 288, 96), (33, 80, 8, 512, 256), (200, 4, 2, 544, 288), (512, 8, 4, 1056, 704),
           (1024, 2, 2, 1056, 1056)]


@pytest.mark.parametrize("T,E,k,H,I", EXPERTS)
def test_experts_small_products(ops, T, E, k, H, I):
    """gate is 32 (and silu(32) is), up 8 in two features of every block and multiples of 2^-14 in the others, by products
    that cancel: h is 256, 256 and multiples of 2^-9, and the down product cancels again.  What is left is the pair
    row's rounding, 2^-11 of it or half a subnormal step, 2^(E - 25)."""
    say(f"small products, experts T={T} E={E} k={k} H={H} I={I}")
    rng = np.random.default_rng(T + H + I)
    x = np.zeros((T, H))
    x[:, :32] = cancelling_rows(rng, T, 32)
    x[:, 32], x[:, 33] = 32, 8
    w13 = np.zeros((E, 2 * I, H))
    w13[:, :I, 32] = 1
    i = np.arange(I)
    big = i % 32 < 2
    w13[:, I + i[big], 33] = 1
    small = i[~big]
    w13[:, I + small, 0], w13[:, I + small, 1] = 6 * 2.0 ** -5, -6 * 2.0 ** -5
    w13[:, I + small, 2 + small % 30] = 2.0 ** -5
    w2 = np.stack([cancelling_weights(rng, H, I) for _ in range(E)])
    (x, xb), (w13, b13), (w2, b2) = bf16(x), bf16(w13), bf16(w2)
    assert np.array_equal(mx8.rounded(x), x)
    ids, w, offsets, order = routing(rng, T, E, k, "even")
    w[:] = 1
    got = pair_rows(*run_experts(ops, xb, b13, b2, w, offsets, order, E, k, H, I))
    for e in range(E):
        p = order[offsets[e]: offsets[e + 1]]
        if p.size == 0:
            continue
        z = x[p // k] @ w13[e].T
        assert (z[:, :I] == 32).all()
        h = 32 * z[:, I:]
        hq, byte = mx8.quantize(h)
        assert np.array_equal(mx8.dequantize(hq, byte), h)
        ref = h @ w2[e].T
        assert np.abs(ref).max() < 2 ** 14
        E_ = mx8.pair_exponent(np.ones(p.size), byte.max(1), np.full(p.size, mx.quantize(w2[e])[1].max()), I)
        assert (np.abs(got[p] - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** (E_[:, None] - 25)).all()


@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear_bf16_bound(ops, T, K, N):
    """BF16 results are FP32 sums, within (K + 8) u of the sum of magnitudes, rounded once: half a BF16 step, 2^-8 of it."""
    say(f"bf16 bound, linear T={T} K={K} N={N}")
    rng, x, xb, w, wb = linear_case(T * K + N + 1, T, K, N)
    wc, ws, _ = ops.mxfp4_quantize_weights(dev_bf16(wb)[None])
    xq, wq = mx8.rounded(x), mx.rounded(w)
    ref, bound = xq @ wq.T, sum_bound(xq, wq, False)
    got = f64(ops.mxfp8_linear(*ops.mxfp8_quantize(dev_bf16(xb)), wc[0], ws[0], N))
    assert (np.abs(got - ref) <= bound + 2.0 ** -8 * (np.abs(ref) + bound) + 1e-37).all()


@pytest.mark.parametrize("T,E,k,H,I,kind", ALL_EXPERTS)
def test_experts_bound(ops, T, E, k, H, I, kind):
    """Pair rows within the bound of FP32 sums, with what the codes of h can move by them, and FP16's rounding."""
    say(f"bound, experts T={T} E={E} k={k} H={H} I={I} {kind}")
    rng = np.random.default_rng(T * H + I + 1)
    x, xb = bf16(draw(rng, T, H))
    w13, b13 = bf16(rng.standard_normal((E, 2 * I, H)) * H ** -0.5)
    w2, b2 = bf16(rng.standard_normal((E, H, I)) * I ** -0.5)
    ids, w, offsets, order = routing(rng, T, E, k, kind)
    got, xq = pair_rows(*run_experts(ops, xb, b13, b2, w, offsets, order, E, k, H, I)), mx8.rounded(x)
    for e in range(E):
        p = order[offsets[e]: offsets[e + 1]]
        if p.size == 0:
            continue
        f, bound, h = expert64(xq[p // k], mx.rounded(w13[e]), mx.rounded(w2[e]), I, False)
        wp = w.reshape(-1)[p].astype(np.float64)[:, None]
        E_ = mx8.pair_exponent(wp[:, 0], mx8.quantize(h)[1].max(1), np.full(p.size, mx.quantize(w2[e])[1].max()), I)
        ref, bound = wp * f, wp * bound
        bound = bound + 2.0 ** -11 * (np.abs(ref) + bound) + 2.0 ** (E_[:, None] + 1 - 25)
        assert (np.abs(got[p] - ref) <= bound).all()


@pytest.mark.parametrize("T,E,k,H,I", [(40, 8, 2, 1024, 512), (300, 16, 4, 2048, 768), (1024, 4, 2, 1024, 1024)])
@pytest.mark.parametrize("outliers", [1.0, 300.0])
def test_experts_in_the_2_norm(ops, T, E, k, H, I, outliers):
    """Against the definition, also with channels of 300 times the rest's size: g and u are off by d = 2e-7 of their size
    in the 2-norm (an FP32 sum of K products has some sqrt(K) of its roundings of 2^-24 / sqrt 3, under 1.6e-6 / 8 at K =
    2048), so h by sqrt(2) d, and q(h) by sqrt(0.8 sqrt(2) d s) for E4M3's spacing s of at most 2^-3: 1.7e-4.  FP16 adds
    2^-11 / sqrt 3 = 2.8e-4.  Together 3.3e-4; twice that is allowed.  (Sums that drop small products are at 1e-3.)"""
    say(f"experts in the 2-norm T={T} E={E} k={k} H={H} I={I} {outliers}")
    rng = np.random.default_rng(T * H + I)
    x32 = draw(rng, T, H).astype(np.float32)
    x32[:, 5::64] *= np.float32(outliers)
    x, xb = bf16(x32)
    w13, b13 = bf16(rng.standard_normal((E, 2 * I, H)) * H ** -0.5 / outliers ** 0.5)
    w2, b2 = bf16(rng.standard_normal((E, H, I)) * I ** -0.5)
    ids, w, offsets, order = routing(rng, T, E, k, "even")
    got = pair_rows(*run_experts(ops, xb, b13, b2, w, offsets, order, E, k, H, I))
    xq, off, norm = mx8.rounded(x), 0.0, 0.0
    for e in range(E):
        p = order[offsets[e]: offsets[e + 1]]
        if p.size == 0:
            continue
        z = xq[p // k] @ mx.rounded(w13[e]).T
        f = mx8.rounded(mx.silu(z[:, :I]) * z[:, I:]) @ mx.rounded(w2[e]).T
        ref = w.reshape(-1)[p].astype(np.float64)[:, None] * f
        off, norm = off + float(((got[p] - ref) ** 2).sum()), norm + float((ref ** 2).sum())
    print(f"  rel-L2 {(off / norm) ** 0.5:.2e}", flush=True)
    assert (off / norm) ** 0.5 <= 6.6e-4


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 512, 256), (16, 24, 4, 1024, 512), (32, 24, 4, 1024, 512)])
def test_experts_and_layer_agree(ops, T, E, k, H, I):
    """A layer call and the operators it stands for multiply alike: they differ by the pair rows' FP16 and few codes of h
    (the bound of the test before)."""
    from test_gpu_mx8_layer import Case

    c = Case(T, E, k, H, I, seed=9)
    d = c.device(ops)
    y, ids, _ = c.call(ops, d, out_dtype=torch.float32)
    r = ops.moe_route(d["x"], d["wr"], d["bias"], k, c.rsf)
    assert torch.equal(r.topk_ids, ids)
    po, ps = ops.mxfp8_grouped_ffn(*ops.mxfp8_quantize(d["x"]), *d["w13"], *d["w2"], H, I, k, r.expert_offsets,
                                   r.sorted_pair_ids, r.topk_w)
    want = f64(ops.moe_combine(po, ps, T, k, torch.float32))
    off = np.linalg.norm(f64(y) - want) / np.linalg.norm(want)
    print(f"  rel-L2 {off:.2e}", flush=True)
    assert off <= 6.6e-4
