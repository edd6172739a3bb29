"""A mixture-of-experts feed-forward block from this package's operators.

    python examples/moe_block.py            # on an MI355X

Between two attention layers of a decoder, in three forms:

  * ``prefill``: many tokens, FP8.  The attention output is normed, gated and
    added to the residual stream, the stream normed again and quantized 1x128
    in one pass; the quantized rows go to their experts' order, through both
    projections with the activation in one call, whose result is quantized and
    whose projections are kept in 8 bits, and the second product, and come back
    weighted.
  * ``decode``: a few tokens, 4-bit weights.  The same with bf16 rows and
    matrix-vector products, which read only the experts that are used.
  * ``backward``: the gradient of ``prefill`` with respect to the attention
    output, the residual stream, the gate, the norms' weights and the routing
    weights (the experts' weights are held fixed, as in fine-tuning around
    them; their input gradients are FP8 products with the same weights, the
    activation's gradient comes quantized from the kept projections).  Nothing
    in it waits for the GPU.

Each is compared with the same block in fp32 torch on the unquantized weights.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_fine_grained_token_amd as F  # noqa: E402

EPS = 1e-6


class MoeBlock:
    """Weights of one block: E experts of width `inner`, SiLU-gated."""

    def __init__(self, width, inner, experts, top_k, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, sigma=1.0, mean=0.0, dtype=torch.bfloat16):
            return (torch.randn(shape, generator=g, device="cuda") * sigma + mean).to(dtype)

        self.width, self.inner, self.experts, self.top_k = width, inner, experts, top_k
        self.w_post = normal(width, sigma=0.1, mean=1.0, dtype=torch.float32)
        self.w_pre = normal(width, sigma=0.1, mean=1.0, dtype=torch.float32)
        self.gate = normal(width, sigma=0.1, mean=0.8, dtype=torch.float32)
        self.residual_scale, self.branch_scale = 1.0, 0.7
        self.router = normal(experts, width, sigma=0.5 / width ** 0.5)
        self.up = normal(experts, 2 * inner, width, sigma=width ** -0.5)
        self.down = normal(experts, width, inner, sigma=inner ** -0.5)
        self.up_fp8, self.up_scales = self._fp8(self.up)
        self.down_fp8, self.down_scales = self._fp8(self.down)
        self.up_w4 = F.fp8_w4_quant_1x128(self.up)
        self.down_w4 = F.fp8_w4_quant_1x32(self.down)

    @staticmethod
    def _fp8(w):
        experts, n, k = w.shape
        q, s = F.fp8_quant_weight_128x128(w.reshape(experts * n, k))
        return q.reshape(w.shape), s.reshape(experts, n // 128, k // 128)

    def route(self, n):
        """Weights and experts of each token (the router itself is small)."""
        best, ids = torch.topk(n.float() @ self.router.float().t(), self.top_k, dim=1)
        return torch.softmax(best, dim=1).contiguous(), ids.contiguous()

    @staticmethod
    def activate(h):
        half = h.shape[1] // 2
        return (torch.nn.functional.silu(h[:, :half].float()) * h[:, half:].float()).to(h.dtype)

    def _norms(self):
        return {"residual_scale": self.residual_scale, "branch_scale": self.branch_scale}

    def prefill(self, y, r):
        """(new residual stream, block output, what the gradient needs)."""
        n = torch.empty_like(y)
        r_out, q, scales, rstd_post, rstd_pre = F.fp8_norm_residual_quant_1x128(
            y, r, self.w_post, self.gate, self.w_pre, eps=EPS, n=n, **self._norms())
        weights, ids = self.route(n)
        offsets, slot_row, _ = F.fp8_moe_sort(ids, self.experts)
        xs, xs_scales = F.fp8_moe_dispatch(q, slot_row, scales=scales)
        a, a_scales, h, h_scales = F.fp8_block_grouped_gemm_gated_quant_1x128(
            xs, xs_scales, self.up_fp8, self.up_scales, offsets, checkpoint=True)
        ys = F.fp8_block_grouped_gemm(a, a_scales, self.down_fp8, self.down_scales, offsets)
        out = F.fp8_moe_combine(ys, slot_row, weights)
        return r_out, out, (y, r_out, rstd_post, rstd_pre, weights, offsets, slot_row, h,
                            h_scales, ys)

    def decode(self, y, r):
        """The same for a few tokens, on the 4-bit weights."""
        r_out, n, _, _ = F.fp8_norm_residual(y, r, self.w_post, self.gate, self.w_pre, eps=EPS,
                                             **self._norms())
        weights, ids = self.route(n)
        offsets, slot_row, _, xs = F.fp8_moe_sort_dispatch(n, ids, self.experts)
        h = F.fp8_w4_grouped_matvec(xs, *self.up_w4, offsets)
        ys = F.fp8_w4_grouped_matvec(self.activate(h), *self.down_w4, offsets)
        return r_out, F.fp8_moe_combine(ys, slot_row, weights)

    def backward(self, dr_out, dout, saved):
        """Gradients of (y, r, w_post, gate, w_pre, routing weights) from those
        of the new residual stream and of the block output."""
        (y, r_out, rstd_post, rstd_pre, weights, offsets, slot_row, h, h_scales,
         ys) = saved
        dys, dweights = F.fp8_moe_combine_grad(dout, ys, slot_row, weights)
        da = F.fp8_block_grouped_gemm_dgrad(*F.fp8_quant_act_1x128(dys), self.down_fp8,
                                            self.down_scales, offsets)
        dh = F.fp8_gated_grad_quant_1x128(da, h, h_scales)
        dxs = F.fp8_block_grouped_gemm_dgrad(*dh, self.up_fp8, self.up_scales, offsets)
        dn = F.fp8_moe_dispatch_grad(dxs, slot_row)
        dy, dr, dw_post, dgate, dw_pre = F.fp8_norm_residual_grad(
            dn, dr_out, y, r_out, rstd_post, rstd_pre, self.w_post, self.gate, self.w_pre,
            **self._norms())
        return dy, dr, dw_post, dgate, dw_pre, dweights

    def plain(self, y, r, routing, weights=None):
        """The block in fp32 torch on the unquantized weights, for given
        experts; differentiable."""
        def norm(v, w):
            return v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * w
        r_out = self.residual_scale * r + self.branch_scale * self.gate * norm(y, self.w_post)
        n = norm(r_out, self.w_pre)
        weights = routing[0] if weights is None else weights
        out = torch.zeros_like(n)
        for e in range(self.experts):
            t, j = torch.nonzero(routing[1] == e, as_tuple=True)
            if t.numel():
                h = n[t] @ self.up[e].float().t()
                a = torch.nn.functional.silu(h[:, :self.inner]) * h[:, self.inner:]
                out = out.index_add(0, t, weights[t, j, None] * (a @ self.down[e].float().t()))
        return r_out, out


def off(a, b):
    """Relative distance of a from b."""
    return float((a.float() - b.float()).norm() / b.float().norm())


def main(width=1024, inner=512, experts=8, top_k=2, tokens=300, decoded=3):
    block = MoeBlock(width, inner, experts, top_k)
    g = torch.Generator(device="cuda").manual_seed(1)

    def rows(n):
        return torch.randn((n, width), generator=g, device="cuda").to(torch.bfloat16)

    report = {}
    y, r = rows(tokens), rows(tokens)
    r_out, out, saved = block.prefill(y, r)
    routing = block.route(F.fp8_norm_residual(y, r, block.w_post, block.gate, block.w_pre,
                                              eps=EPS, **block._norms())[1])
    want_r, want = block.plain(y.float(), r.float(), routing)
    report["prefill stream"], report["prefill output"] = off(r_out, want_r), off(out, want)

    yd, rd = rows(decoded), rows(decoded)
    r_d, out_d = block.decode(yd, rd)
    n_d = F.fp8_norm_residual(yd, rd, block.w_post, block.gate, block.w_pre, eps=EPS,
                              **block._norms())[1]
    want_r, want = block.plain(yd.float(), rd.float(), block.route(n_d))
    report["decode stream"], report["decode output (4 bits)"] = off(r_d, want_r), off(out_d, want)

    dr_out, dout = rows(tokens), rows(tokens)
    got = block.backward(dr_out, dout, saved)
    leaves = [t.float().detach().requires_grad_() for t in (y, r, routing[0])]
    params = [p.requires_grad_() for p in (block.w_post, block.gate, block.w_pre)]
    a, b = block.plain(leaves[0], leaves[1], routing, leaves[2])
    want = torch.autograd.grad([a, b], leaves[:2] + params + leaves[2:],
                               [dr_out.float(), dout.float()])
    for p in params:
        p.requires_grad_(False)
    for name, x, w in zip(("dy", "dr", "dw_post", "dgate", "dw_pre", "dweights"), got, want):
        report["gradient " + name] = off(x, w)
    return report


if __name__ == "__main__":
    for what, far in main().items():
        print(f"{what:24s} relative distance from fp32: {far:.4f}")
