"""A mixture-of-experts layer that computes in FP8, forward and backward.

    python examples/fp8_moe_layer.py [--tokens 4096] [--experts 32] [--topk 2] [--width 2048] [--hidden 4096]

The master weights stay in bf16.  Each step projects them onto the MXFP4 grid
and lays them out as 128x128 blockwise FP8 (the direct conversion), sorts the
router's choices, takes the tokens to the experts' order, and runs both
layers' products, and those of their gradients, on FP8 operands.  The
gradient passes straight through to the master weights.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_precision_x32_gb300 as mxq  # noqa: E402


class Dispatch(torch.autograd.Function):
    """Token rows in the experts' order."""

    @staticmethod
    def forward(ctx, x, order):
        ctx.order = order
        return mxq.mxq_moe_dispatch(x, order.source, order.slots.shape[1])

    @staticmethod
    def backward(ctx, g):
        return mxq.mxq_moe_dispatch_grad(g.contiguous(), ctx.order.slots), None


class Combine(torch.autograd.Function):
    """The experts' rows summed back to their tokens with the router's weights."""

    @staticmethod
    def forward(ctx, y, weights, order):
        ctx.save_for_backward(y, weights)
        ctx.order = order
        return mxq.mxq_moe_combine(y, order.slots, weights)

    @staticmethod
    def backward(ctx, g):
        y, weights = ctx.saved_tensors
        d_rows, d_weights = mxq.mxq_moe_combine_grad(g.contiguous(), y, ctx.order.source, ctx.order.slots, weights)
        return d_rows, d_weights, None


class ExpertLinear(torch.autograd.Function):
    """y[r] = W[e(r)] x[r] for a stack W [E, N, K] of weights, N a multiple of
    128, so that no 128x128 tile lies across two experts."""

    @staticmethod
    def forward(ctx, x, w, order):
        E, N, K = w.shape
        wq, tile = mxq.mxq_fp8_block128_direct(w.view(E * N, K))
        wq, tile = wq.view(E, N, K), tile.view(E, N // 128, -1)
        ctx.save_for_backward(x, wq, tile, order.offsets)
        ctx.w_dtype = w.dtype
        return mxq.mxq_fp8_grouped_matmul(*mxq.mxq_fp8_quant_1x128(x), wq, tile, order.offsets, out_dtype=x.dtype)

    @staticmethod
    def backward(ctx, g):
        x, wq, tile, offsets = ctx.saved_tensors
        g = g.contiguous()
        d_x = mxq.mxq_fp8_grouped_matmul_dgrad(*mxq.mxq_fp8_quant_1x128(g), wq, tile, offsets, out_dtype=x.dtype)
        d_w = mxq.mxq_fp8_grouped_matmul_wgrad(*mxq.mxq_fp8_quant_128x1(g), *mxq.mxq_fp8_quant_128x1(x), offsets,
                                               out_dtype=ctx.w_dtype)
        return d_x, d_w, None


class MoELayer(torch.nn.Module):
    """topk of `experts` two-layer networks per token: W2 silu(W1 x)."""

    def __init__(self, width, hidden, experts, topk, device="cuda", dtype=torch.bfloat16):
        super().__init__()
        self.topk = topk
        new = lambda *s, fan: torch.nn.Parameter(torch.randn(*s, device=device, dtype=dtype) * fan**-0.5)  # noqa: E731
        self.router = new(experts, width, fan=width)
        self.w1 = new(experts, hidden, width, fan=width)
        self.w2 = new(experts, width, hidden, fan=hidden)

    def route(self, x):
        """(experts [tokens, topk] int32, weights [tokens, topk] fp32)"""
        weights, ids = torch.softmax(x.float() @ self.router.float().t(), 1).topk(self.topk, dim=1)
        return ids.int(), weights / weights.sum(1, keepdim=True)

    def forward(self, x):
        ids, weights = self.route(x)
        order = mxq.mxq_moe_sort(ids, self.router.shape[0], align=128)  # whole 128x1 blocks for the weight gradient
        h = ExpertLinear.apply(Dispatch.apply(x, order), self.w1, order)
        y = ExpertLinear.apply(torch.nn.functional.silu(h), self.w2, order)
        return Combine.apply(y, weights, order)

    def serve(self, x, stacks):
        """The forward pass for serving: the weights laid out once
        (`stacks`), tokens gathered and quantized in one pass."""
        ids, weights = self.route(x)
        order = mxq.mxq_moe_sort(ids, self.router.shape[0])
        (q1, t1), (q2, t2) = stacks
        h = mxq.mxq_fp8_grouped_matmul(*mxq.mxq_fp8_quant_1x128(x, order.source, self.topk), q1, t1, order.offsets)
        y = mxq.mxq_fp8_grouped_matmul(*mxq.mxq_fp8_quant_1x128(torch.nn.functional.silu(h)), q2, t2, order.offsets)
        return mxq.mxq_moe_combine(y, order.slots, weights)

    def stacks(self):
        out = []
        for w in (self.w1, self.w2):
            E, N, K = w.shape
            q, t = mxq.mxq_fp8_block128_direct(w.detach().view(E * N, K))
            out.append((q.view(E, N, K), t.view(E, N // 128, -1)))
        return out

    def reference(self, x):
        """The same layer in fp32 on the projected weights, expert by expert."""
        ids, weights = self.route(x)
        x = x.float()
        y = torch.zeros_like(x)
        w1, w2 = (Straight.apply(w) for w in (self.w1, self.w2))
        for e in range(self.router.shape[0]):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            out = torch.nn.functional.silu(x[t] @ w1[e].t()) @ w2[e].t()
            y = y.index_add(0, t, out * weights[t, j, None])
        return y


class Straight(torch.autograd.Function):
    """The MXFP4 projection in fp32, its gradient passed straight through."""

    @staticmethod
    def forward(ctx, w):
        return mxq.mxq_fake_quant_mxfp4(w).float()

    @staticmethod
    def backward(ctx, g):
        return g


def relative(a, b):
    return float((a.detach().float() - b.detach().float()).norm() / b.detach().float().norm())


def compare(layer, x):
    """Relative differences from the fp32 layer: output, serving output,
    gradients of the input, of both stacks and of the router."""
    leaves = [x, layer.w1, layer.w2, layer.router]
    g = torch.randn_like(x)
    got = layer(x)
    d_got = torch.autograd.grad(got, leaves, g)
    want = layer.reference(x)
    d_want = torch.autograd.grad(want, leaves, g.float())
    with torch.no_grad():
        served = layer.serve(x, layer.stacks())
    return {"output": relative(got, want), "served": relative(served, want)} | {
        n: relative(a, b) for n, a, b in zip(("input", "w1", "w2", "router"), d_got, d_want)}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("experts", 32), ("topk", 2), ("width", 2048), ("hidden", 4096)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    torch.manual_seed(0)
    layer = MoELayer(a.width, a.hidden, a.experts, a.topk)
    x = torch.randn(a.tokens, a.width, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    print("relative difference from fp32:", {k: round(v, 4) for k, v in compare(layer, x).items()})

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
    stacks = layer.stacks()
    print("training step (forward and backward): %.3f ms" % timed(lambda: torch.autograd.backward(layer(x), g)))
    with torch.no_grad():
        print("serving, %d tokens: %.3f ms" % (a.tokens, timed(lambda: layer.serve(x, stacks))))
        few = x[:32].detach()
        print("serving, %d tokens: %.3f ms" % (len(few), timed(lambda: layer.serve(few, stacks))))


if __name__ == "__main__":
    main()
