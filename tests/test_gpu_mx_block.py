"""MXFP4Block: the operators run together as a decoder layer would use them.

Each step is checked against the oracle applied to that step's actual input (a rounding that falls the other way
early on would otherwise hide everything after it), the whole block against the same calls made one by one, and a
captured graph, replayed with other work in between, against the eager pass."""

import numpy as np
import pytest
import torch

from gpu_cases import dev_bf16, rel_l2, to_np
from oracle import mx
from oracle import norm as onorm
from workloads import gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import mx_block, ops

    return ops, mx_block


def values(t):
    return to_np(t.float()).astype(np.float64)


def inputs(T, K, H, seed):
    rng = np.random.default_rng(seed)
    bits = lambda a: dev_bf16(gen.f32_to_bf16_bits(a.astype(np.float32)))  # noqa: E731
    return bits(rng.standard_normal((T, K))), bits(rng.standard_normal((T, H)))


@pytest.mark.parametrize("T", [1, 17, 200])
def test_block_steps(mods, T):
    ops, mx_block = mods
    E, k, H, I, K = 8, 2, 320, 96, 288
    blk = mx_block.random_block(E, k, H, I, K, seed=T)
    attn, res = inputs(T, K, H, T)
    out = blk(attn, res)
    b = blk._bufs[(T, K)]
    # projection: the packed weights read back through the library's exact inverse
    c, s = ops.mxfp4_unpack_weights(blk.w_o[0][None], blk.w_o[1][None], H, K)
    codes = to_np(c)[0]
    w_o = mx.dequantize(np.stack([codes & 15, codes >> 4], -1).reshape(H, K), to_np(s)[0])
    assert rel_l2(values(b["o"]), mx.rounded(values(attn)) @ w_o.T) < 1e-5
    # residual and the norm before the experts: half an ulp of BF16 (2^-8), FP32 noise
    r1 = onorm.residual(values(b["o"]), values(res), values(blk.norms[0]), None, 1.0, blk.eps)
    assert np.max(np.abs(values(b["r1"]) - r1) / (np.abs(r1) + 1e-3)) <= 2.0 ** -8 * 1.01
    n1 = onorm.norm(values(b["r1"]), values(blk.norms[1]), blk.eps)
    assert np.max(np.abs(values(b["n1"]) - n1) / (np.abs(n1) + 1e-3)) <= 2.0 ** -8 * 1.01
    pc, ps = mx.row_form(*mx.quantize(values(b["n1"])))
    assert np.array_equal(to_np(b["x"]["codes"]), pc) and np.array_equal(to_np(b["x"]["scales"]), ps)
    # after the experts
    r2 = onorm.residual(values(out.y), values(b["r1"]), values(blk.norms[2]), values(blk.gate), blk.residual_scale, blk.eps)
    assert np.max(np.abs(values(out.residual) - r2) / (np.abs(r2) + 1e-3)) <= 2.0 ** -8 * 1.01
    c, s = ops.mxfp4_quantize(out.n)
    assert torch.equal(out.codes, c) and torch.equal(out.scales, s)
    # the experts: an independent sum over pairs, from the route the block took
    ids, w = to_np(out.route.topk_ids), to_np(out.route.topk_w).astype(np.float64)
    xq = mx.rounded(values(b["n1"]))
    y = np.zeros((T, H))

    def matrix(packed, e, n, kk):
        c, s = ops.mxfp4_unpack_weights(packed[0][e:e + 1].contiguous(), packed[1][e:e + 1].contiguous(), n, kk)
        c = to_np(c)[0]
        return mx.dequantize(np.stack([c & 15, c >> 4], -1).reshape(n, kk), to_np(s)[0])

    for e in range(E):
        t, j = np.where(ids == e)
        if t.size:
            z = xq[t] @ matrix(blk.w13, e, 2 * I, H).T
            f = mx.rounded(mx.silu(z[:, :I]) * z[:, I:]) @ matrix(blk.w2, e, H, I).T
            np.add.at(y, t, f * w[t, j][:, None])
    assert rel_l2(values(out.y), y) < 4e-3  # FP16 pair rows, and the odd h that rounds the other way


def test_block_is_its_calls_and_reuses_its_buffers(mods):
    ops, mx_block = mods
    blk = mx_block.random_block(seed=3)
    for T in (40, 3, 40):
        attn, res = inputs(T, 512, 512, T)
        out = blk(attn, res)
        c, s = ops.mxfp4_quantize(attn)
        o = ops.mxfp4_linear(c, s, *blk.w_o, 512, torch.float32)
        r1, n1, c, s = ops.moe_norm_out(o, res, blk.norms[0], blk.norms[1], quantize=True)
        r = ops.moe_route(n1, blk.w_router, blk.bias, blk.k, blk.rsf)
        y = ops.moe_combine(*ops.mxfp4_grouped_ffn(c, s, *blk.w13, *blk.w2, 512, 256, blk.k, r.expert_offsets,
                                                   r.sorted_pair_ids, r.topk_w), T, blk.k, torch.float32)
        r2, n2 = ops.moe_norm_out(y, r1, blk.norms[2], blk.norms[3], gate=blk.gate, residual_scale=0.5)
        assert torch.equal(out.residual, r2) and torch.equal(out.n, n2) and torch.equal(out.y, y)
    n, c, s = blk.enter(res, blk.norms[1])
    assert torch.equal(n, ops.moe_norm_in(res, blk.norms[1])) and torch.equal(c, ops.mxfp4_quantize(n)[0])


@pytest.mark.parametrize("T", [1, 300])
def test_block_in_a_graph(mods, T):
    ops, mx_block = mods
    blk = mx_block.random_block(seed=5)
    attn, res = inputs(T, 512, 512, 9)
    want = [t.clone() for t in (lambda o: (o.residual, o.n, o.codes, o.y))(blk(attn, res))]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = blk(attn, res)
    for i in range(4):
        for t in (out.residual, out.n, out.codes, out.y):
            t.zero_()
        other = blk(*inputs(7 + i, 512, 512, i))  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((out.residual, out.n, out.codes, out.y), want):
            assert torch.equal(got, ref), f"replay {i}"
        assert bool(torch.isfinite(other.y).all())


def test_block_refuses_odd_intermediate(mods):
    _, mx_block = mods
    with pytest.raises(ValueError, match="multiple of 32"):
        mx_block.random_block(I=48)
