"""The MXFP8 products in their large tiles: 256 x 256 and 256 x 128 of the dense product, 256 x 64 of both expert stages, with ragged
ends and short and long reductions.

The references of the dense products are formed on the device in 64 bits from weights that MXFP4 holds exactly (every block has a
6 under its power of two) and from the values that x's codes stand for.  Bounds as in tests/test_gpu_mx8.py, for FP32 sums."""

import pytest
import torch

from gpu_cases import say
from test_gpu_mx8_sums import test_experts_bound as check_experts_bound
from test_gpu_mx8_sums import test_experts_small_products as check_experts_small_products

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def weights(g, N, K):
    """[N, K] in float64: E2M1 values under a power of two a block, the first of each block 6."""
    grid = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    w = grid[torch.randint(0, 15, (N, K // 32, 32), generator=g, device="cuda")]
    w[..., 0] = 6
    return (w * torch.exp2(torch.randint(-6, 0, (N, K // 32, 1), generator=g, device="cuda").double())).view(N, K)


@pytest.mark.parametrize("T,K,N", [(250, 1056, 65500), (500, 1312, 32699), (1001, 992, 16380), (4090, 1568, 4093),
                                   (120, 1056, 65500), (4000, 1120, 2020), (8100, 800, 1021),
                                   (255, 4128, 65533), (1023, 3872, 16381)])
def test_linear_in_large_tiles(ops, T, K, N):
    say(f"large tiles T={T} K={K} N={N}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T + K + N)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = weights(g, N, K)
    x = (randn(T, K) * torch.exp(randn(K))).to(torch.bfloat16)
    wc, ws, _ = ops.mxfp4_quantize_weights(w.to(torch.bfloat16)[None])
    codes, scales = ops.mxfp8_quantize(x)
    xq = ops.mxfp8_dequantize(codes, scales, K, torch.float32).double()
    ref = xq @ w.t()
    bound = (K + 8) * U * (xq.abs() @ w.t().abs())
    del w

    def check(got, ref, bound):
        last = 2.0 ** -8 if got.dtype == torch.bfloat16 else U
        d = (got.double() - ref).abs() - bound - last * (ref.abs() + bound)
        print(f"  {got.dtype} rel-L2 {((got.double() - ref).norm() / ref.norm()).item():.2e}", flush=True)
        assert bool((d <= 0).all())

    check(ops.mxfp8_linear(codes, scales, wc[0], ws[0], N, torch.float32), ref, bound)
    low = torch.full((T, N + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.mxfp8_linear(codes, scales, wc[0], ws[0], N, y=low[:, :N])
    check(low[:, :N], ref, bound)
    assert bool((low[:, N:] == 7.0).all())
    again = ops.mxfp8_linear(codes, scales, wc[0], ws[0], N)
    assert torch.equal(again, low[:, :N])
    del low, again
    bias, r = randn(N).to(torch.bfloat16), randn(T, N + 5)
    z = ref + bias.double()
    act = z * torch.sigmoid(z)
    bound = 1.13 * (bound + U * z.abs()) + (8 + 4 * z.abs()) * 2 * U * act.abs()
    del ref, z
    for dtype in (torch.float32, torch.bfloat16):
        res = r.to(dtype)
        want = act + res[:, :N].double()
        y = ops.mxfp8_linear(codes, scales, wc[0], ws[0], N, dtype, bias=bias, activation="silu", residual=res[:, :N])
        check(y, want, bound + U * want.abs())
        inner = res[:, :N]
        ops.mxfp8_linear(codes, scales, wc[0], ws[0], N, bias=bias, activation="silu", residual=inner, y=inner)
        assert torch.equal(inner, y) and torch.equal(res[:, N:], r.to(dtype)[:, N:])


EXPERTS = [(40, 40, 4, 2848, 96, "even"), (300, 40, 4, 2848, 2208, "few"), (2100, 8, 2, 2080, 64, "even"),
           (1500, 5, 3, 1056, 1120, "few"), (700, 6, 6, 2336, 1184, "one")]


@pytest.mark.parametrize("T,E,k,H,I,kind", EXPERTS)
def test_experts_in_large_tiles(ops, T, E, k, H, I, kind):
    check_experts_bound(ops, T, E, k, H, I, kind)


@pytest.mark.parametrize("T,E,k,H,I", [(40, 40, 4, 2848, 96), (2100, 8, 2, 2080, 64), (1500, 5, 3, 1056, 1120)])
def test_experts_small_products_in_large_tiles(ops, T, E, k, H, I):
    check_experts_small_products(ops, T, E, k, H, I)
