"""The mixture-of-experts half of a transformer block in FP8, forward and backward.

    python examples/fp8_moe_block.py [--tokens 4096] [--experts 32] [--topk 4] [--width 2048] [--hidden 1024]

What comes from the block's first half is added to the residual stream and
normed.  The norm writes the FP8 operand of the products that follow: a shared
expert takes it as it is, the routed ones a token's row once for each choice of
the router.  An expert is W2 (silu(Wg x) * Wu x), with Wg and Wu in one stack
W1; the activation goes into the second product as an FP8 operand as well.
The router scores with sigmoids; a bias balances the choice and groups limit
it.  Master weights stay in bf16, projected onto the MXFP4 grid each step; the
gradient passes straight through.
"""

import argparse
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]

import block_scaled_precision_x32_gb300 as mxq  # noqa: E402
from fp8_moe_layer import Combine, Straight, relative  # noqa: E402


class Norm(torch.autograd.Function):
    """(y, h, E4M3 bytes of y, their scales) of x + residual."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        r = mxq.mxq_rmsnorm(x, weight, residual, normed=True, stats=True)
        ctx.save_for_backward(r.h, weight, r.rstd)
        ctx.mark_non_differentiable(r.data, r.scales)
        return r.y, r.h, r.data, r.scales

    @staticmethod
    def backward(ctx, g, g_h, *_):
        h, weight, rstd = ctx.saved_tensors
        d_h, d_weight = mxq.mxq_rmsnorm_grad(g.contiguous(), h, weight, rstd, g_h=g_h.contiguous())
        return d_h, d_h, d_weight.to(weight.dtype)


class Route(torch.autograd.Function):
    """(weights, experts) of the router's logits."""

    @staticmethod
    def forward(ctx, logits, bias, topk, groups, topk_groups):
        ids, weights = mxq.mxq_moe_route(logits, topk, bias=bias, score="sigmoid", groups=groups, topk_groups=topk_groups, group_top=2)
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    def backward(ctx, g, _):
        logits, ids = ctx.saved_tensors
        return mxq.mxq_moe_route_grad(g.contiguous(), logits, ids, score="sigmoid"), None, None, None, None


def projected(w):
    """A weight [N, K], or a stack [E, N, K] with N a multiple of 128, as 128x128 blockwise FP8."""
    q, tile = mxq.mxq_fp8_block128_direct(w.detach().reshape(-1, w.shape[-1]))
    return q.view(w.shape), tile.view(w.shape[:-2] + (w.shape[-2] // 128, -1))


def product(q, c, w, order, dtype):
    if order is None:
        return mxq.mxq_fp8_matmul(q, c, *w, out_dtype=dtype)
    return mxq.mxq_fp8_grouped_matmul(q, c, *w, order.offsets, out_dtype=dtype)


def product_grads(g, columns, w, order, dtype, w_dtype):
    """(gradient of the operand, gradient of the weight) of a product; columns: the operand with 128x1 scales."""
    rows, cols = mxq.mxq_fp8_quant_1x128(g), mxq.mxq_fp8_quant_128x1(g)
    if order is None:
        return mxq.mxq_fp8_matmul_dgrad(*rows, *w, out_dtype=dtype), mxq.mxq_fp8_matmul_wgrad(*cols, *columns, out_dtype=w_dtype)
    return (mxq.mxq_fp8_grouped_matmul_dgrad(*rows, *w, order.offsets, out_dtype=dtype),
            mxq.mxq_fp8_grouped_matmul_wgrad(*cols, *columns, order.offsets, out_dtype=w_dtype))


class First(torch.autograd.Function):
    """W1 y for the quantized rows of y, all of them or those of the router's order."""

    @staticmethod
    def forward(ctx, y, data, scales, w, order):
        wq = projected(w)
        ctx.save_for_backward(y, *wq)
        ctx.order, ctx.w_dtype = order, w.dtype
        if order is not None:
            data, scales = mxq.mxq_fp8_dispatch(data, scales, order.source, order.slots.shape[1])
        return product(data, scales, wq, order, y.dtype)

    @staticmethod
    def backward(ctx, g):
        y, *wq = ctx.saved_tensors
        order = ctx.order
        columns = mxq.mxq_fp8_quant_128x1(y) if order is None else mxq.mxq_fp8_quant_128x1(y, order.source, order.slots.shape[1])
        d, d_w = product_grads(g.contiguous(), columns, wq, order, y.dtype, ctx.w_dtype)
        return d if order is None else mxq.mxq_moe_dispatch_grad(d, order.slots), None, None, d_w, None


class Second(torch.autograd.Function):
    """W2 (silu(gate) * up) for the rows x = [gate | up]."""

    @staticmethod
    def forward(ctx, x, w, order):
        wq = projected(w)
        ctx.save_for_backward(x, *wq)
        ctx.order, ctx.w_dtype = order, w.dtype
        return product(*mxq.mxq_fp8_silu_mul_1x128(x), wq, order, x.dtype)

    @staticmethod
    def backward(ctx, g):
        x, *wq = ctx.saved_tensors
        d, d_w = product_grads(g.contiguous(), mxq.mxq_fp8_silu_mul_128x1(x), wq, ctx.order, x.dtype, ctx.w_dtype)
        return mxq.mxq_silu_mul_grad(d, x), d_w, None


class MoEBlock(torch.nn.Module):
    def __init__(self, width, hidden, experts, topk, groups=1, topk_groups=1, device="cuda", dtype=torch.bfloat16):
        super().__init__()
        self.topk, self.groups, self.topk_groups = topk, groups, topk_groups
        new = lambda *s, fan: torch.nn.Parameter(torch.randn(*s, device=device, dtype=dtype) * fan**-0.5)  # noqa: E731
        self.norm = torch.nn.Parameter(1 + 0.1 * torch.randn(width, device=device, dtype=dtype))
        self.router = new(experts, width, fan=width)
        self.w1, self.w2 = new(experts, 2 * hidden, width, fan=width), new(experts, width, hidden, fan=hidden)
        self.s1, self.s2 = new(2 * hidden, width, fan=width), new(width, hidden, fan=hidden)
        self.register_buffer("bias", 0.05 * torch.randn(experts, device=device))  # of the balancing, not of the gradient

    def forward(self, x, residual):
        """(the experts' sum, the new residual stream, the router's choices)"""
        y, h, data, scales = Norm.apply(x, residual, self.norm)
        weights, ids = Route.apply(y.float() @ self.router.float().t(), self.bias, self.topk, self.groups, self.topk_groups)
        order = mxq.mxq_moe_sort(ids, self.router.shape[0], align=128)  # whole 128x1 blocks for the weight gradients
        routed = Second.apply(First.apply(y, data, scales, self.w1, order), self.w2, order)
        shared = Second.apply(First.apply(y, data, scales, self.s1, None), self.s2, None)
        return shared + Combine.apply(routed, weights, order), h, ids

    def serve(self, x, residual, weights):
        """The forward pass for serving: the weights laid out once, the residual stream updated in place."""
        w1, w2, s1, s2, router = weights
        r = mxq.mxq_rmsnorm(x, self.norm, residual, normed=True, h=residual)
        ids, p = mxq.mxq_moe_route(r.y.float() @ router, self.topk, bias=self.bias, score="sigmoid", groups=self.groups,
                                   topk_groups=self.topk_groups, group_top=2)
        order = mxq.mxq_moe_sort(ids, self.router.shape[0])
        rows = product(*mxq.mxq_fp8_dispatch(r.data, r.scales, order.source, self.topk), w1, order, x.dtype)
        routed = product(*mxq.mxq_fp8_silu_mul_1x128(rows), w2, order, x.dtype)
        shared = product(*mxq.mxq_fp8_silu_mul_1x128(product(r.data, r.scales, s1, None, x.dtype)), s2, None, x.dtype)
        return shared + mxq.mxq_moe_combine(routed, order.slots, p)

    def laid_out(self):
        return tuple(projected(w) for w in (self.w1, self.w2, self.s1, self.s2)) + (self.router.detach().float().t().contiguous(),)

    def reference(self, x, residual, ids):
        """The same in fp32 on the projected weights, for given choices of experts."""
        h = (x + residual).float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * self.norm.float()
        w1, w2, s1, s2 = (Straight.apply(w) for w in (self.w1, self.w2, self.s1, self.s2))

        def expert(v, a, b):
            gate, up = (v @ a.t()).chunk(2, 1)
            return (torch.nn.functional.silu(gate) * up) @ b.t()

        p = torch.sigmoid(y @ self.router.float().t()).gather(1, ids.long())
        p = p / p.sum(1, keepdim=True)
        out = expert(y, s1, s2)
        for e in range(self.router.shape[0]):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            out = out.index_add(0, t, expert(y[t], w1[e], w2[e]) * p[t, j, None])
        return out, h


def compare(block, x, residual):
    """Relative differences from the fp32 block: outputs, serving outputs, gradients."""
    leaves = {"x": x, "residual": residual} | dict(block.named_parameters())
    g, g_h = torch.randn_like(x), torch.randn_like(x)
    out, h, ids = block(x, residual)
    d_got = torch.autograd.grad([out, h], list(leaves.values()), [g, g_h])
    want, want_h = block.reference(x, residual, ids)
    d_want = torch.autograd.grad([want, want_h], list(leaves.values()), [g.float(), g_h.float()])
    with torch.no_grad():
        stream = residual.detach().clone()
        served = block.serve(x.detach(), stream, block.laid_out())
    return {"output": relative(out, want), "stream": relative(h, want_h), "served": relative(served, want), "served stream": relative(stream, want_h)} | {
        "d " + n: relative(a, b) for n, a, b in zip(leaves, d_got, d_want)}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("experts", 32), ("topk", 4), ("width", 2048), ("hidden", 1024)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    torch.manual_seed(0)
    block = MoEBlock(a.width, a.hidden, a.experts, a.topk)
    x, residual = (torch.randn(a.tokens, a.width, device="cuda", dtype=torch.bfloat16, requires_grad=True) for _ in range(2))
    print("relative difference from fp32:", {k: round(v, 4) for k, v in compare(block, x, residual).items()})

    def timed(f, n=20):
        for _ in range(3):
            f()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(n):
            f()
        end.record()
        torch.cuda.synchronize()
        return start.elapsed_time(end) / n

    g = torch.randn_like(x)
    print("training step (forward and backward): %.3f ms" % timed(lambda: torch.autograd.backward(block(x, residual)[:2], [g, g])))
    with torch.no_grad():
        weights = block.laid_out()
        for n in (a.tokens, 32):
            few, stream = x[:n].detach(), residual[:n].detach().clone()
            print("serving, %d tokens: %.3f ms" % (n, timed(lambda: block.serve(few, stream, weights))))


if __name__ == "__main__":
    main()
