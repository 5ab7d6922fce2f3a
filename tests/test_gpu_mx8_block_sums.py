"""MXFP4Block with MXFP8 activations keeps its sums in FP32 between its operators."""

import pytest
import torch

from test_gpu_mx_block import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 17, 200])
def test_block_norms_the_projection_in_fp32(T):
    """With a norm after attention the projection is rounded once, when the residual is added: the block's residual and
    normed input are those of the operators with an FP32 projection, bit for bit."""
    from nvfp4_w4a4_mixture_amd import mx_block, ops

    E, k, H, I, K = 8, 2, 320, 96, 288
    bias = torch.randn(H, device="cuda").to(torch.bfloat16)
    blk = mx_block.random_block(E, k, H, I, K, seed=T + 1, act_bits=8, b_o=bias)
    attn, res = inputs(T, K, H, T)
    blk(attn, res)
    b = blk._bufs[(T, K)]
    o = ops.mxfp8_linear(*ops.mxfp8_quantize(attn), *blk.w_o, H, torch.float32, bias=bias)
    r1, n, codes, scales = ops.moe_norm_out_mxfp8(o, res, blk.norms[0], blk.norms[1], eps=blk.eps)
    assert torch.equal(b["r1"], r1) and torch.equal(b["n1"], n)
    assert torch.equal(b["x"]["codes"], codes) and torch.equal(b["x"]["scales"], scales)
    low = ops.moe_norm_out_mxfp8(o.to(torch.bfloat16), res, blk.norms[0], blk.norms[1], eps=blk.eps)[0]
    assert not torch.equal(low, r1)  # what a BF16 projection would give differs
