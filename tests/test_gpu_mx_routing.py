"""GPU parity of the MXFP4 experts under routings that moe_route does not write.

The checks and their bounds are test_gpu_mx.test_experts', with the routing replaced by one made here."""

import numpy as np
import pytest
import torch

import test_gpu_mx as mxt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def routed(ids, rng):
    """ids [T, k] -> what test_gpu_mx.routing returns"""
    T, k = ids.shape
    w = rng.uniform(0.05, 1.5, (T, k)).astype(np.float32)
    flat = ids.reshape(-1)
    counts = np.bincount(flat, minlength=int(flat.max()) + 1)
    return ids, w, counts, np.argsort(flat, kind="stable").astype(np.int32)


def with_ids(monkeypatch, make):
    """test_experts routes by make(rng, T, E, k) -> ids from here on."""

    def routing(rng, T, E, k, kind):
        ids, w, counts, order = routed(make(rng, T, E, k), rng)
        counts = np.concatenate([counts, np.zeros(E - counts.size, counts.dtype)])
        return ids, w, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), order

    monkeypatch.setattr(mxt, "routing", routing)


# T tokens no more than a tile of 64 (128) tokens holds, their pairs several times as many
@pytest.mark.parametrize("T,E,k,H,I", [(64, 3, 2, 288, 96), (33, 4, 4, 96, 64), (5, 8, 8, 256, 128),
                                       (120, 16, 16, 2848, 1440)])
def test_repeated_experts(ops, monkeypatch, T, E, k, H, I):
    """A token that names an expert more than once: an expert then has more pairs than there are tokens."""

    def make(rng, T, E, k):
        ids = rng.integers(0, E, (T, k))
        ids[: (2 * T + 2) // 3] = E - 1  # two thirds of the tokens name the last expert k times
        return ids

    with_ids(monkeypatch, make)
    mxt.test_experts(ops, T, E, k, H, I, "repeated")


# streaming; 128 x 64 tiles; 256 x 128 tiles
@pytest.mark.parametrize("T,E,k,H,I", [(2, 4, 2, 288, 96), (200, 4, 2, 288, 96), (2048, 256, 8, 96, 64)])
def test_nan_weights_leave_the_other_features(ops, T, E, k, H, I):
    """NaN blocks in an expert's down weights make NaN of their own features; every other one is, bit for bit, what it
    is with zeros in their place."""
    rng = np.random.default_rng(T)
    _, xb = mxt.bf16(mxt.draw(rng, T, H))
    _, b13 = mxt.bf16(rng.standard_normal((E, 2 * I, H)) * H ** -0.5)
    w2 = (rng.standard_normal((E, H, I)) * I ** -0.5).astype(np.float32)
    bad = np.zeros((E, H), bool)
    clean = w2.copy()
    for e, row, block, value in ((0, 5, 1, np.nan), (0, H - 1, 0, -np.inf), (2, 33, I // 32 - 1, np.inf)):
        w2[e, row, 32 * block + 7] = value
        clean[e, row, 32 * block: 32 * block + 32] = 0
        bad[e, row] = True
    w2[3] = np.nan  # an expert with nothing else
    clean[3] = 0
    bad[3] = True
    ids, w, offsets, order = mxt.routing(rng, T, E, k, "even")
    w[0] = 3e4  # a row whose scale matters
    args = (ids, w, offsets, order, E, k, H, I)
    po, ps = mxt.run_experts(ops, xb, b13, mxt.bf16(w2)[1], *args)
    want, want_scale = mxt.run_experts(ops, xb, b13, mxt.bf16(clean)[1], *args)
    assert torch.equal(ps, want_scale)
    mask = torch.from_numpy(bad[ids.reshape(-1)]).cuda()  # [T*k, H]: the pair's expert has NaN in this feature
    assert bool(torch.isnan(po[mask]).all())
    assert torch.equal(po[~mask].view(torch.int16), want[~mask].view(torch.int16))
    assert bool((want[~mask] != 0).any())


# 65 to 256 experts, whose tiles are found over all the lanes of a wave (four experts a lane): 128 x 64 and 256 x 128
# tiles; pairs everywhere, only in the last half, only at every seventh expert
@pytest.mark.parametrize("T,E,k,H,I", [(200, 70, 8, 320, 160), (300, 128, 8, 96, 64), (600, 256, 8, 96, 64),
                                       (2048, 256, 8, 96, 64), (999, 130, 5, 64, 288), (700, 255, 6, 64, 32)])
@pytest.mark.parametrize("where", ["all", "late", "sparse"])
def test_many_experts(ops, monkeypatch, T, E, k, H, I, where):
    def make(rng, T, E, k):
        pool = {"all": np.arange(E), "late": np.arange(E // 2, E), "sparse": np.arange(E - 1, 0, -7)}[where]
        return np.stack([rng.permutation(pool)[:k] for _ in range(T)])

    with_ids(monkeypatch, make)
    mxt.test_experts(ops, T, E, k, H, I, where)


# rows on 16 bytes, written eight BF16 at a time: every tile shape (128 x 64, 128 x 128, 256 x 128, 256 x 256), ragged
# last tiles in both directions, and rows of which the last piece goes by elements
@pytest.mark.parametrize("T,K,N", [(1, 288, 64), (40, 288, 8200), (400, 288, 4208), (390, 1568, 4200), (900, 320, 6216),
                                   (897, 1344, 6200), (1800, 288, 6512), (1797, 1888, 6504), (1797, 4128, 6504)])
@pytest.mark.parametrize("extra", [0, 5])
def test_linear_bf16_vector_stores(ops, T, K, N, extra):
    mxt.say(f"linear BF16 T={T} K={K} N={N}+{extra}")
    x, xb, w, wb = mxt.linear_case(T + K + N, T, K, N + extra)
    wc, wsc, _ = ops.mxfp4_quantize_weights(mxt.dev_bf16(wb)[None])
    codes, scales = ops.mxfp4_quantize(mxt.dev_bf16(xb))
    n = N + extra
    y = torch.full((T, -(-n // 8) * 8), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.mxfp4_linear(codes, scales, wc[0], wsc[0], n, y=y[:, :n])
    mxt.check_linear(mxt.to_np(y[:, :n].float()).astype(np.float64), mxt.mx.rounded(x), mxt.mx.rounded(w), True)
    assert bool((y[:, n:] == 7.0).all())
    assert torch.equal(ops.mxfp4_linear(codes, scales, wc[0], wsc[0], n), y[:, :n])
