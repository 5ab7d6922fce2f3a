"""MXFP4Block with MXFP8 activations: its operators run together as a decoder layer would use them, for few tokens (the
layer in few launches) and many, with and without the norm after attention."""

import numpy as np
import pytest
import torch

from gpu_cases import rel_l2, to_np
from oracle import mx, mx8
from oracle import norm as onorm
from test_gpu_mx_block import inputs, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import mx_block, ops

    return ops, mx_block


@pytest.mark.parametrize("T", [1, 17, 200])
@pytest.mark.parametrize("post", [True, False])
def test_block_steps(mods, T, post):
    """Each step against the oracle applied to that step's actual input."""
    ops, mx_block = mods
    E, k, H, I, K = 8, 2, 320, 96, 288
    bias = torch.randn(H, device="cuda").to(torch.bfloat16)
    blk = mx_block.random_block(E, k, H, I, K, seed=T, act_bits=8, b_o=bias, **({} if post else {"w_post_attn": None}))
    attn, res = inputs(T, K, H, T)
    out = blk(attn, res)
    b = blk._bufs[(T, K)]

    def matrix(packed, e, n, kk):
        c, s = ops.mxfp4_unpack_weights(packed[0][e:e + 1].contiguous(), packed[1][e:e + 1].contiguous(), n, kk)
        c = to_np(c)[0]
        return mx.dequantize(np.stack([c & 15, c >> 4], -1).reshape(n, kk), to_np(s)[0])

    half = lambda got, ref: np.max(np.abs(got - ref) / (np.abs(ref) + 1e-3)) <= 2.0 ** -8 * 1.01  # noqa: E731  of BF16
    o = mx8.rounded(values(attn)) @ matrix((blk.w_o[0][None], blk.w_o[1][None]), 0, H, K).T + values(bias)
    if post:
        assert rel_l2(values(b["o"]), o) < 2.4e-3
        assert half(values(b["r1"]), onorm.residual(values(b["o"]), values(res), values(blk.norms[0]), None, 1.0, blk.eps))
    else:
        assert rel_l2(values(b["r1"]), o + values(res)) < 2.4e-3
    assert half(values(b["n1"]), onorm.norm(values(b["r1"]), values(blk.norms[1]), blk.eps))
    pc, ps = mx8.row_form(*mx8.quantize(values(b["n1"])))
    assert np.array_equal(to_np(b["x"]["codes"]), pc) and np.array_equal(to_np(b["x"]["scales"]), ps)
    ids, w = to_np(out.route.topk_ids), to_np(out.route.topk_w).astype(np.float64)
    r = ops.moe_route(b["n1"], blk.w_router, blk.bias, k, blk.rsf)
    assert np.array_equal(ids, to_np(r.topk_ids))
    xq, y = mx8.rounded(values(b["n1"])), np.zeros((T, H))
    for e in range(E):
        t, j = np.where(ids == e)
        if t.size:
            z = xq[t] @ matrix(blk.w13, e, 2 * I, H).T
            f = mx8.rounded(mx.silu(z[:, :I]) * z[:, I:]) @ matrix(blk.w2, e, H, I).T
            np.add.at(y, t, f * w[t, j][:, None])
    assert rel_l2(values(out.y), y) < 2e-3  # FP16 pair rows, and the odd h that rounds the other way (see test_gpu_mx8.py)
    r2 = onorm.residual(values(out.y), values(b["r1"]), values(blk.norms[2]), values(blk.gate), blk.residual_scale, blk.eps)
    assert half(values(out.residual), r2)
    c, s = ops.mxfp8_quantize(out.n)
    assert torch.equal(out.codes, c) and torch.equal(out.scales, s)


def test_block_reuses_its_buffers_and_enters(mods):
    ops, mx_block = mods
    blk = mx_block.random_block(seed=3, act_bits=8)
    attn, res = inputs(40, 512, 512, 1)
    want = [t.clone() for t in (lambda o: (o.residual, o.n, o.y))(blk(attn, res))]
    blk(*inputs(3, 512, 512, 2))
    again = blk(attn, res)
    assert all(torch.equal(a, b) for a, b in zip((again.residual, again.n, again.y), want))
    n, c, s = blk.enter(res, blk.norms[1])
    assert torch.equal(n, ops.moe_norm_in_mxfp8(res, blk.norms[1])[0]) and torch.equal(c, ops.mxfp8_quantize(n)[0])
    assert tuple(blk(attn[:0], res[:0]).n.shape) == (0, 512)


@pytest.mark.parametrize("T", [1, 32, 300])
def test_block_in_a_graph(mods, T):
    ops, mx_block = mods
    blk = mx_block.random_block(seed=5, act_bits=8)
    attn, res = inputs(T, 512, 512, 9)
    want = [t.clone() for t in (lambda o: (o.residual, o.n, o.codes, o.y))(blk(attn, res))]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = blk(attn, res)
    for i in range(4):
        for t in (out.residual, out.n, out.codes, out.y):
            t.zero_()
        other = blk(*inputs(7 + 30 * i, 512, 512, i))  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((out.residual, out.n, out.codes, out.y), want):
            assert torch.equal(got, ref), f"replay {i}"
        assert bool(torch.isfinite(other.y).all())


def test_block_refusals(mods):
    _, mx_block = mods
    with pytest.raises(ValueError, match="act_bits"):
        mx_block.random_block(act_bits=6)
    with pytest.raises(ValueError, match="b_o needs"):
        mx_block.random_block(b_o=torch.zeros(512, dtype=torch.bfloat16, device="cuda"))
