"""The part of a decoder layer that follows attention, in MXFP4, as one object.

    c, s       = mxfp4_quantize(attention output)
    o          = mxfp4_linear(c, s, W_o)                                 (FP32)
    r1, n, c, s = moe_norm_out(o, residual, w_post_attn, w_pre_moe)       (residual, norm before the experts, quantized)
    route      = moe_route(n)                                            (BF16 router)
    pair rows  = mxfp4_grouped_ffn(c, s, route)
    y          = moe_combine(pair rows)                                  (FP32)
    r2, n, c, s = moe_norm_out(y, r1, w_post_moe, w_next, gate, scale)    (residual, the next layer's first norm, quantized)

``enter`` is the norm before a first layer.  The buffers of the token counts
used last are kept and reused (``buffers.Buffers``), so a forward pass of one of
them enqueues only kernels on the current stream, and a pass can be captured in
a HIP graph.

``python -m nvfp4_w4a4_mixture_amd.mx_block`` runs one block with random
weights and prints its shapes and time.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import ops
from .buffers import Buffers


@dataclass
class BlockOut:
    residual: torch.Tensor  # BF16 [T, H]: r2
    n: torch.Tensor  # BF16 [T, H]: the next layer's normed input
    codes: torch.Tensor  # n in MXFP4 (padded rows)
    scales: torch.Tensor
    route: ops.RouteOut
    y: torch.Tensor  # FP32 [T, H]: the experts' weighted sum


class MXFP4Block:
    def __init__(self, w_o, w_router_bf16, bias, k: int, rsf: float, w13, w2, w_pre_moe, w_next,
                 w_post_attn: Optional[torch.Tensor] = None, w_post_moe: Optional[torch.Tensor] = None,
                 gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0, eps: float = 1e-6):
        """w_o: packed (codes, scales) of the output projection [H, K]; w13, w2: packed (codes, scales, max_scale) of
        the experts [E, 2I, H] (gate rows, then up rows) and [E, H, I]; norm weights BF16 [H], a post norm may be
        None; gate: None or BF16 [1, H]."""
        self.w_o = w_o[:2]
        self.w_router, self.bias, self.k, self.rsf = w_router_bf16, bias, int(k), float(rsf)
        self.w13, self.w2 = w13[:2], w2
        self.E, self.H = w_router_bf16.shape
        self.I = w13[0].shape[1] * 16  # 2I / 32 row groups
        self.norms = (w_post_attn, w_pre_moe, w_post_moe, w_next)
        self.gate, self.residual_scale, self.eps = gate, float(residual_scale), float(eps)
        self.device = w_router_bf16.device
        self._bufs = Buffers(self.device)

    @classmethod
    def from_bf16(cls, w_o, w_router_bf16, bias, k, rsf, w13, w2, w_pre_moe, w_next, **kw) -> "MXFP4Block":
        """Quantizes BF16 weights w_o [H, K], w13 [E, 2I, H], w2 [E, H, I] with the library."""
        if w13.shape[1] % 64:
            raise ValueError("the expert intermediate size must be a multiple of 32")
        co, so, _ = ops.mxfp4_quantize_weights(w_o[None])
        return cls((co[0], so[0]), w_router_bf16, bias, k, rsf, ops.mxfp4_quantize_weights(w13),
                   ops.mxfp4_quantize_weights(w2), w_pre_moe, w_next, **kw)

    def _buffers(self, T: int, K: int) -> dict:
        d, E, H, I, k = self.device, self.E, self.H, self.I, self.k
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=d)  # noqa: E731
        rows = lambda c: dict(codes=new((T, -(-c // 256) * 128), torch.uint8),  # noqa: E731
                              scales=new((T, -(-c // 256) * 8), torch.uint8))
        return dict(a=rows(K), o=new((T, H), torch.float32), r1=new((T, H), torch.bfloat16),
                    n1=new((T, H), torch.bfloat16), x=rows(H),
                    route=ops.RouteOut(new((T, k), torch.int32), new((T, k), torch.float32), new((E,), torch.int32),
                                       new((E + 1,), torch.int32), new((T * k,), torch.int32)),
                    route_ws=new((max(ops.moe_route_workspace_bytes(T, H, E, k), 1),), torch.uint8),
                    ffn_ws=new((max(ops.mxfp4_ffn_workspace_bytes(T, k, E, H, I), 1),), torch.uint8),
                    pair_out=new((T * k, H), torch.float16), pair_scale=new((T * k,), torch.float32),
                    y=new((T, H), torch.float32), r2=new((T, H), torch.bfloat16), n2=new((T, H), torch.bfloat16),
                    out=rows(H))

    def enter(self, x: torch.Tensor, w: torch.Tensor):
        """The norm before a first layer: (n, codes, scales) of x [T, H]."""
        return ops.moe_norm_in(x, w, self.eps, quantize=True)

    def forward(self, attn: torch.Tensor, residual: torch.Tensor) -> BlockOut:
        """attn [T, K] BF16 (attention's output, before its projection), residual [T, H] BF16.

        The returned tensors are the block's buffers for this T: the next call of the same T overwrites them."""
        T, K = attn.shape
        b = self._bufs.take((T, K), lambda: self._buffers(T, K))
        w_post_attn, w_pre, w_post_moe, w_next = self.norms
        ops.mxfp4_quantize(attn, **b["a"])
        ops.mxfp4_linear(b["a"]["codes"], b["a"]["scales"], *self.w_o, self.H, y=b["o"])
        ops.moe_norm_out(b["o"], residual, w_post_attn, w_pre, eps=self.eps, out=b["r1"], n=b["n1"], **b["x"])
        r = ops.moe_route(b["n1"], self.w_router, self.bias, self.k, self.rsf, out=b["route"], workspace=b["route_ws"])
        ops.mxfp4_grouped_ffn(b["x"]["codes"], b["x"]["scales"], *self.w13, *self.w2, self.H, self.I, self.k,
                              r.expert_offsets, r.sorted_pair_ids, r.topk_w, b["pair_out"], b["pair_scale"],
                              workspace=b["ffn_ws"])
        ops.moe_combine(b["pair_out"], b["pair_scale"], T, self.k, torch.float32, y=b["y"])
        ops.moe_norm_out(b["y"], b["r1"], w_post_moe, w_next, gate=self.gate, residual_scale=self.residual_scale,
                         eps=self.eps, out=b["r2"], n=b["n2"], **b["out"])
        return BlockOut(b["r2"], b["n2"], b["out"]["codes"], b["out"]["scales"], r, b["y"])

    __call__ = forward


def random_block(E: int = 8, k: int = 2, H: int = 512, I: int = 256, K: int = 512, seed: int = 0,
                 device="cuda") -> MXFP4Block:
    """A block of random weights (normal, scaled to keep activations near unit size)."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device=device) * scale).to(torch.bfloat16)  # noqa: E731
    w = lambda: (1 + 0.1 * torch.randn(H, generator=g, device=device)).to(torch.bfloat16)  # noqa: E731
    return MXFP4Block.from_bf16(r(H, K, scale=K ** -0.5), r(E, H, scale=H ** -0.5), torch.zeros(E, device=device), k, 2.5,
                                r(E, 2 * I, H, scale=H ** -0.5), r(E, H, I, scale=I ** -0.5), w(), w(), w_post_attn=w(),
                                w_post_moe=w(), gate=r(1, H), residual_scale=0.5)


if __name__ == "__main__":
    blk = random_block(E=16, k=4, H=2048, I=1024, K=2048)
    for T in (1, 16, 512, 4096):
        x = torch.randn(T, 2048, device="cuda").to(torch.bfloat16)
        out = blk(x, x)
        torch.cuda.synchronize()
        a, z = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(20):
            out = blk(x, x)
        z.record()
        torch.cuda.synchronize()
        print(f"T={T}: n {tuple(out.n.shape)}, |n| rms {out.n.float().square().mean().sqrt().item():.3f}, "
              f"{a.elapsed_time(z) / 20 * 1e3:.1f} us a block", flush=True)
