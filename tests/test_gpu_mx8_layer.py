"""The whole layer for a few tokens against the float64 routing and experts, and against the operators it stands for.

Bounds: those of tests/test_gpu_mx8.py for FP32 sums (the layer multiplies activations in two operands throughout); the
sum over a token's experts is k more FP32 products and sums; routing weights are one FP32 rounding of an FP64 value (and
of a hardware-accurate sigmoid), 2^-23."""

import numpy as np
import pytest
import torch

from gpu_cases import dev_bf16, say, to_np
from oracle import mx, mx8
from oracle import routing as oroute
from test_gpu_mx import bf16, draw
from test_gpu_mx8 import expert64, f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


class Case:
    def __init__(self, T, E, k, H, I, seed=0, x32=None, skew=0.3):
        rng = np.random.default_rng(T * H + I + E + seed)
        self.T, self.E, self.k, self.H, self.I, self.rsf = T, E, k, H, I, 2.5
        self.x, self.xb = bf16(draw(rng, T, H) if x32 is None else x32)
        self.wr, self.wrb = bf16(rng.standard_normal((E, H)) * H ** -0.5)
        self.bias = (skew * rng.standard_normal(E)).astype(np.float32)
        self.w13, self.b13 = bf16(rng.standard_normal((E, 2 * I, H)) * H ** -0.5)
        self.w2, self.b2 = bf16(rng.standard_normal((E, H, I)) * I ** -0.5)

    def device(self, ops):
        q13 = ops.mxfp4_quantize_weights(dev_bf16(self.b13))
        q2 = ops.mxfp4_quantize_weights(dev_bf16(self.b2))
        return dict(x=dev_bf16(self.xb), wr=dev_bf16(self.wrb), bias=torch.from_numpy(self.bias).cuda(), w13=q13[:2], w2=q2)

    def call(self, ops, d, **kw):
        return ops.mxfp8_moe_layer(d["x"], d["wr"], d["bias"], self.k, self.rsf, *d["w13"], *d["w2"][:2], **kw)

    def garbage(self, ops):
        n = ops.mxfp8_moe_layer_workspace_bytes(self.T, self.H, self.E, self.k, self.I)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


CASES = [(1, 1, 1, 32, 32), (1, 8, 2, 256, 128), (1, 80, 8, 512, 288), (2, 5, 5, 288, 96), (3, 256, 7, 64, 32),
         (4, 16, 3, 320, 160), (5, 7, 1, 1056, 544), (8, 80, 8, 768, 256), (9, 128, 8, 256, 64), (16, 8, 2, 256, 128),
         (17, 80, 8, 544, 288), (31, 12, 6, 96, 1504), (32, 40, 8, 2080, 320), (32, 256, 256, 64, 32)]


@pytest.mark.parametrize("T,E,k,H,I", CASES)
def test_layer(ops, T, E, k, H, I):
    say(f"layer T={T} E={E} k={k} H={H} I={I}")
    c = Case(T, E, k, H, I)
    d = c.device(ops)
    y, ids, w = c.call(ops, d, out_dtype=torch.float32, workspace=c.garbage(ops))
    ref_ids, _, w64, gap = oroute.route(c.xb, c.wrb, c.bias, k, c.rsf)
    assert gap.min() > 1e-12  # the draws hold no near tie
    ids, w = to_np(ids), to_np(w).astype(np.float64)
    assert np.array_equal(ids, ref_ids)
    assert (np.abs(w - w64) <= 2.0 ** -23 * w64).all()
    xq = mx8.rounded(c.x)
    ref, bound, mag = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if t.size == 0:
            continue
        f, b, _ = expert64(xq[t], mx.rounded(c.w13[e]), mx.rounded(c.w2[e]), I, False)
        wt = w[t, j][:, None]
        ref[t] += wt * f
        bound[t] += wt * b
        mag[t] += np.abs(wt * f) + wt * b
    bound += (k + 10 + I // 256 * k) * U * mag + 1e-37
    got = f64(y)
    worst, off = float(np.max(np.abs(got - ref) / bound)), float(np.linalg.norm(got - ref) / np.linalg.norm(ref))
    print(f"  error / bound {worst:.3f}, rel-L2 {off:.2e}", flush=True)
    assert worst <= 1.0 and off <= 1e-3
    # BF16 results are the FP32 ones, rounded; into given tensors, and the same bits again
    yb = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
    ib, wb = torch.zeros_like(c.call(ops, d)[1]), torch.zeros((T, k), device="cuda")
    out = c.call(ops, d, y=yb, topk_ids=ib, topk_w=wb)
    assert out[0].data_ptr() == yb.data_ptr() and torch.equal(yb, y.to(torch.bfloat16))
    assert np.array_equal(to_np(ib), ids) and np.array_equal(to_np(wb).astype(np.float64), w)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 128), (16, 80, 8, 512, 256), (32, 10, 3, 288, 96)])
def test_layer_is_its_operators(ops, T, E, k, H, I):
    """Routing equals moe_route's; y is the combine of mxfp8_grouped_ffn's pair rows to within their FP16."""
    c = Case(T, E, k, H, I, seed=5)
    d = c.device(ops)
    y, ids, w = c.call(ops, d, out_dtype=torch.float32)
    r = ops.moe_route(d["x"], d["wr"], d["bias"], k, c.rsf)
    assert torch.equal(r.topk_ids, ids) and bool(((r.topk_w - w).abs() <= 2.0 ** -23 * w).all())
    po, ps = ops.mxfp8_grouped_ffn(*ops.mxfp8_quantize(d["x"]), *d["w13"], *d["w2"], H, I, k, r.expert_offsets,
                                   r.sorted_pair_ids, r.topk_w)
    want = f64(ops.moe_combine(po, ps, T, k, torch.float32))
    # q(h) of the tiled product is off by 1e-3 at most twice over (tests/test_gpu_mx8.py), that of the layer by far less
    assert np.linalg.norm(f64(y) - want) <= 2e-3 * np.linalg.norm(want)


def test_layer_strided_and_unaligned_rows(ops):
    c = Case(6, 12, 4, 288, 96)
    d = c.device(ops)
    want = c.call(ops, d)
    for pad in (1, 5, 8):
        wide = torch.full((6, 288 + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, pad:] = d["x"]
        got = c.call(ops, dict(d, x=wide[:, pad:]))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_layer_ties_and_nan_scores(ops):
    """Equal scores go to the lower expert; NaN ranks last; every slot is written."""
    c = Case(3, 9, 5, 64, 32)
    c.wrb[:] = c.wrb[2]  # every expert ties
    c.bias[:] = 0.25
    c.bias[7] = np.nan
    c.bias[1] = 0.5
    d = c.device(ops)
    _, ids, w = c.call(ops, d, workspace=c.garbage(ops))
    assert to_np(ids).tolist() == [[1, 0, 2, 3, 4]] * 3
    assert np.allclose(to_np(w), 0.5)
    x32 = c.x.astype(np.float32)
    x32[1, 3] = np.nan  # all its scores are NaN: experts by index, and its row is NaN
    d = dict(d, x=dev_bf16(bf16(x32)[1]))
    y, ids, _ = c.call(ops, d)
    assert to_np(ids).tolist() == [[1, 0, 2, 3, 4], [0, 1, 2, 3, 4], [1, 0, 2, 3, 4]]
    assert bool(y[1].isnan().all()) and not bool(y[[0, 2]].isnan().any())


def test_layer_nan_weights_stay_with_their_tokens(ops):
    """An expert with a NaN block spoils the tokens that chose it, and no other; zero tokens give zeros."""
    c = Case(20, 6, 2, 288, 96)
    x32 = c.x.astype(np.float32)
    x32[4] = 0
    c.x, c.xb = bf16(x32)
    want = oroute.route(c.xb, c.wrb, c.bias, c.k, c.rsf)[0]
    chosen = [int((want == e).any(1).sum()) for e in range(c.E)]
    e = next(e for e in range(c.E) if 0 < chosen[e] < c.T)  # some tokens choose it, and some do not
    bad = c.w13.astype(np.float32)
    bad[e, 5, 7] = np.inf
    c.b13 = bf16(bad)[1]
    y, ids, _ = c.call(ops, c.device(ops))
    hit = (ids == e).any(1)
    assert bool(hit.any()) and not bool(hit.all())
    assert bool(y[hit].isnan().any(1).all()) and not bool(y[~hit].isnan().any())
    assert bool((y[4] == 0).all()) or bool(hit[4])


def test_layer_no_tokens_and_refusals(ops):
    c = Case(4, 6, 2, 64, 32)
    d = c.device(ops)
    empty = c.call(ops, dict(d, x=d["x"][:0]))
    assert [tuple(t.shape) for t in empty] == [(0, 64), (0, 2), (0, 2)]

    def raises(kind, match, f):
        with pytest.raises(kind, match=match):
            f()

    raises(ops.MoEError, "MOE_ERR_SHAPE.*T <= 32", lambda: c.call(ops, dict(d, x=d["x"].repeat(9, 1))))
    raises(ops.MoEError, "MOE_ERR_WORKSPACE", lambda: c.call(ops, d, workspace=c.garbage(ops)[:256]))
    raises(ValueError, "1 <= k <= E", lambda: ops.mxfp8_moe_layer(d["x"], d["wr"], d["bias"], 7, 1.0, *d["w13"], *d["w2"][:2]))
    raises(ops.MoEError, "MOE_ERR_SHAPE.*scaling", lambda: ops.mxfp8_moe_layer(d["x"], d["wr"], d["bias"], 2, 0.0, *d["w13"],
                                                                               *d["w2"][:2]))
    raises(ValueError, "w2_codes must have shape", lambda: ops.mxfp8_moe_layer(d["x"], d["wr"], d["bias"], 2, 1.0, *d["w13"],
                                                                               d["w2"][0][:5], d["w2"][1]))
    raises(ValueError, r"y must have shape \(4, 64\)", lambda: c.call(ops, d, y=torch.empty((4, 32), device="cuda")))


def test_layer_on_streams_and_in_graphs(ops):
    """Two calls at once on two streams; two captured calls that share a workspace, replayed in turn with eager work between."""
    a, b = Case(1, 16, 4, 512, 256), Case(7, 16, 4, 512, 256)
    da, db = a.device(ops), b.device(ops)
    want_a, want_b = a.call(ops, da), b.call(ops, db)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got_a, got_b = a.call(ops, da, stream=s1), b.call(ops, db, stream=s2)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got_a + got_b, want_a + want_b))
    ws = torch.empty(max(c.garbage(ops).numel() for c in (a, b)), dtype=torch.uint8, device="cuda")
    graphs = []
    for c, d in ((a, da), (b, db)):
        out = c.call(ops, d, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(ops, d, workspace=ws, y=out[0], topk_ids=out[1], topk_w=out[2])
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), want in zip(graphs, (want_a, want_b)):
            for t in out:
                t.fill_(0)
            ws.fill_(0xFF)
            g.replay()
            assert all(torch.equal(u, v) for u, v in zip(out, want))
            assert all(torch.equal(u, v) for u, v in zip(a.call(ops, da), want_a))


def test_layer_many_ties(ops):
    """Ties and near ties among many experts, which a kernel of its own ranks: by the whole score, then the lower index."""
    c = Case(24, 200, 6, 64, 32)
    c.wrb[:] = c.wrb[2]
    c.bias[:] = 0.25
    c.bias[9] = np.nan
    c.bias[150] = np.nextafter(np.float32(0.25), np.float32(1))  # the next FP32 value: an upper half of its FP64 key differs
    c.bias[77] = 0.5
    c.bias[30] = 0.125
    _, ids, w = c.call(ops, c.device(ops), workspace=c.garbage(ops))
    assert to_np(ids).tolist() == [[77, 150, 0, 1, 2, 3]] * c.T
    assert np.allclose(to_np(w), c.rsf / c.k)
    x32 = c.x.astype(np.float32)
    x32[:] = 0  # scores of 1/2 and a bias that only a key's lower half shows
    c.bias[:] = 0
    c.bias[[180, 4]] = 2.0 ** -40
    c.bias[11] = 2.0 ** -39
    d = dict(c.device(ops), x=dev_bf16(bf16(x32)[1]))
    assert to_np(c.call(ops, d)[1]).tolist() == [[11, 4, 180, 0, 1, 2]] * c.T


def test_layer_of_shared_products_repeats(ops):
    """Workgroups that share a feature group's products join them in one order: calls and replays are alike bit for bit."""
    c = Case(16, 80, 8, 512, 512)
    d = c.device(ops)
    ws = c.garbage(ops)
    want = c.call(ops, d, workspace=ws)
    out = tuple(torch.empty_like(t) for t in want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(ops, d, workspace=ws, y=out[0], topk_ids=out[1], topk_w=out[2])
    for i in range(20):
        for t in out:
            t.fill_(0)
        if i % 2:
            ws.fill_(0xFF)
        g.replay()
        assert all(torch.equal(u, v) for u, v in zip(out, want))
        assert all(torch.equal(u, v) for u, v in zip(c.call(ops, d), want))
