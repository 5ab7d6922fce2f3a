"""What a call with stream= allocates belongs to that stream.

The caching allocator hands a freed block on in the order of the stream it was allocated for.  A missing output or
workspace of a call on another stream must come from that stream's pool: a workspace is dropped when the call returns,
with its kernels still queued.  The allocator's own record of allocations shows it, whatever the timing."""

import pytest
import torch

pytestmark = pytest.mark.gpu

E, K, H, I, T = 4, 2, 256, 128, 24


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from nvfp4_w4a4_mixture_amd import ops as _ops

    return _ops


def allocations(call):
    """Runs call() and returns (its result, the streams that its allocations were made for)."""
    torch.cuda.synchronize()
    torch.cuda.memory._record_memory_history(enabled="all", context=None)
    try:
        out = call()
        trace = torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)
    return out, [t["stream"] for t in trace if t["action"] == "alloc"]


def flat(out):
    if isinstance(out, (tuple, list)):
        return [t for o in out for t in flat(o)]
    return [] if out is None else [out]


def bf16(*shape, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def check(call, count):
    """call(stream): the same results on a side stream as on the current one, `count` allocations, all of them the
    side stream's; the current stream is the one it was."""
    want = flat(call(None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    before = torch.cuda.current_stream()
    out, streams = allocations(lambda: call(side))
    assert torch.cuda.current_stream() == before
    assert len(streams) == count and all(s == side.cuda_stream for s in streams), (streams, side.cuda_stream)
    side.synchronize()
    for a, b in zip(flat(out), want, strict=True):
        assert torch.equal(a, b)
    # the default stream given by name is the current one here
    _, streams = allocations(lambda: call(torch.cuda.default_stream()))
    torch.cuda.synchronize()
    assert len(streams) == count and not any(streams)


def mx_inputs(ops):
    x = bf16(T, H)
    c, s = ops.mxfp4_quantize(x)
    w13 = ops.mxfp4_quantize_weights(bf16(E, 2 * I, H, seed=1))[:2]
    w2 = ops.mxfp4_quantize_weights(bf16(E, H, I, seed=2))
    r = ops.moe_route(x, bf16(E, H, seed=3), torch.zeros(E, device="cuda"), K, 2.5)
    return x, c, s, w13, w2, r


def test_mx_products(ops):
    x, c, s, w13, w2, r = mx_inputs(ops)
    check(lambda st: ops.mxfp4_quantize(x, stream=st), 2)
    check(lambda st: ops.mxfp4_dequantize(c, s, H, stream=st), 1)
    check(lambda st: ops.mxfp4_linear(c, s, w13[0][0], w13[1][0], 2 * I, stream=st), 1)
    check(lambda st: ops.mxfp4_grouped_ffn(c, s, *w13, *w2, H, I, K, r.expert_offsets, r.sorted_pair_ids, r.topk_w,
                                           stream=st), 3)  # pair rows, their scales, the workspace
    po, ps = ops.mxfp4_grouped_ffn(c, s, *w13, *w2, H, I, K, r.expert_offsets, r.sorted_pair_ids, r.topk_w)
    check(lambda st: ops.moe_combine(po, ps, T, K, stream=st), 1)


def test_norms(ops):
    x, w = bf16(T, H), bf16(H, seed=1)
    check(lambda st: ops.moe_norm_in(x, w, quantize=True, stream=st), 3)
    check(lambda st: ops.moe_norm_out(x, x, w, w, quantize=True, stream=st), 4)


def test_a_refusal_leaves_the_current_stream(ops):
    x, side = bf16(T, H), torch.cuda.Stream()
    before = torch.cuda.current_stream()
    with pytest.raises(ops.MoEError, match="multiple of 32"):
        ops.mxfp4_quantize(x[:, :40], stream=side)
    with pytest.raises(ValueError, match="codes must have shape"):
        ops.mxfp4_quantize(x, codes=torch.empty((T, 1), dtype=torch.uint8, device="cuda"), stream=side)
    assert torch.cuda.current_stream() == before


def test_weight_packing(ops):
    w = bf16(E, 96, H)
    check(lambda st: ops.mxfp4_quantize_weights(w, stream=st), 3)
    codes, scales, _ = ops.mxfp4_quantize_weights(w)
    check(lambda st: ops.mxfp4_unpack_weights(codes, scales, 96, H, stream=st), 2)
    c, s = ops.mxfp4_unpack_weights(codes, scales, 96, H)
    check(lambda st: ops.mxfp4_pack_weights(c, s, stream=st), 3)


def test_nvfp4_layer(ops):
    x, wr, bias = bf16(T, H), bf16(E, H, seed=3), torch.zeros(E, device="cuda")
    gs = torch.full((1,), 40.0, device="cuda")
    check(lambda st: ops.moe_route(x, wr, bias, K, 2.5, stream=st), 6)
    check(lambda st: ops.moe_route_quantize(x, wr, bias, K, 2.5, gs, stream=st), 8)
    check(lambda st: ops.nvfp4_quantize_act(x, gs, stream=st), 2)
    w = bf16(2 * E, I, H, seed=1)
    check(lambda st: ops.nvfp4_quantize_weights(w, stream=st), 3)
    c13, s13, g13 = ops.nvfp4_quantize_weights(w)
    w13 = (c13.view(E, 2 * I, H // 2), s13.view(E, 2 * I // 16, H // 128, 16, 8), g13.view(E, 2))
    w2 = ops.nvfp4_quantize_weights(bf16(E, H, I, seed=2))
    h_gs = torch.full((E,), 40.0, device="cuda")
    r, xc, xs = ops.moe_route_quantize(x, wr, bias, K, 2.5, gs)
    pairs = (r.expert_offsets, r.sorted_pair_ids, r.topk_w)
    check(lambda st: ops.moe_nvfp4_grouped_ffn(xc, xs, gs, *w13, *w2, h_gs, K, *pairs, pair_sqnorm=True, stream=st), 4)
    check(lambda st: ops.moe_nvfp4_gate_up_swiglu(xc, xs, gs, *w13, h_gs, K, *pairs[:2], stream=st), 3)
    hc, hs = ops.moe_nvfp4_gate_up_swiglu(xc, xs, gs, *w13, h_gs, K, *pairs[:2])
    check(lambda st: ops.moe_nvfp4_down_scatter(hc, hs, h_gs, T, *w2, K, *pairs, pair_sqnorm=True, stream=st), 4)
    po, ps, sq = ops.moe_nvfp4_down_scatter(hc, hs, h_gs, T, *w2, K, *pairs, pair_sqnorm=True)
    check(lambda st: ops.moe_combine_reap(po, ps, T, K, sq, r.topk_w, *pairs[:2], E, stream=st), 2)
    check(lambda st: ops.reap_saliency(sq, r.topk_w, *pairs[:2], T, K, E, stream=st), 1)
    sal = ops.reap_saliency(sq, r.topk_w, *pairs[:2], T, K, E)
    check(lambda st: ops.reap_prune_select(sal, 2, stream=st), 1)
    keep = ops.reap_prune_select(sal, 2)
    check(lambda st: ops.moe_gather_experts(wr, keep, stream=st), 1)
    ws13, ws2 = bf16(2 * I, H, seed=4), bf16(H, I, seed=5)
    check(lambda st: ops.moe_shared_expert(x, ws13, ws2, stream=st), 2)
    check(lambda st: ops.moe_shared_gate_up(x, ws13, stream=st), 2)
    h = ops.moe_shared_gate_up(x, ws13)
    check(lambda st: ops.moe_shared_down(h, ws2, stream=st), 2)
    shared = ops.moe_shared_down(h, ws2)
    check(lambda st: ops.moe_combine_block(po, ps, shared, T, K, stream=st), 1)
    check(lambda st: ops.hadamard_rotate_bf16(x, None, 128, stream=st), 1)
    check(lambda st: ops.moe_nvfp4_unpack_weights(*w13[:2], 0, stream=st), 2)
