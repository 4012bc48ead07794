"""A routed layer around experts of one's own: an INT8 layer as it serves,
and a training step whose experts are plain matrices.

    python examples/experts_around.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from block_quantized_expert_amd import binding as B  # noqa: E402


def int8_weights(w):
    """Rows of w [n_experts][rows][cols] rounded to int8, a scale per row."""
    e, r, c = w.shape
    q, scale = B.moe_quantize_int8(w.reshape(e * r, c))
    return B.Int8Weight(q.reshape(e, r, c), scale.reshape(e, r))


def int8_layer(x, logits, gate, up, down, top_k, base=None, routed_scale=1.5):
    """y [n][hidden]: route, group, the experts' FFN in int8, combine.  base
    (the residual or the shared expert's output) is added."""
    _, w, grouping = B.moe_route_group(logits, top_k, routed_scale)
    q, s = B.moe_quantize_int8(x)
    h = B.moe_swiglu_int8(gate, up, q, s, grouping, top_k=top_k)
    q, s = B.moe_quantize_int8(h)
    rows = B.moe_product_int8(down, q, s, grouping)
    return B.moe_combine(rows, w, grouping, base=base)


class RouteWeights(torch.autograd.Function):
    """Weights of the top_k experts and the grouping; the gradient goes to the
    logits of the experts chosen."""

    @staticmethod
    def forward(ctx, logits, top_k, routed_scale):
        ids, w, grouping = B.moe_route_group(logits, top_k, routed_scale)
        ctx.save_for_backward(logits, ids)
        ctx.routed_scale = routed_scale
        ctx.mark_non_differentiable(*grouping)
        return (w,) + grouping

    @staticmethod
    def backward(ctx, dw, *_):
        logits, ids = ctx.saved_tensors
        return B.moe_route_backward(logits, ids, dw.contiguous(), ctx.routed_scale), None, None


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, top_k, *grouping):
        ctx.save_for_backward(*grouping)
        ctx.top_k = top_k
        return B.moe_dispatch(x, grouping, top_k)

    @staticmethod
    def backward(ctx, drows):
        dx = B.moe_dispatch_backward(drows.contiguous(), ctx.saved_tensors, ctx.top_k)
        return (dx, None) + (None,) * 4


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, w, *grouping):
        ctx.save_for_backward(rows, w, *grouping)
        return B.moe_combine(rows, w, grouping)

    @staticmethod
    def backward(ctx, dy):
        rows, w, *grouping = ctx.saved_tensors
        drows, dw = B.moe_combine_backward(dy.contiguous(), rows, w, tuple(grouping))
        return (drows, dw) + (None,) * 4


def train_layer(x, router, gate, up, down, top_k, routed_scale=1.5):
    """The same layer with experts in torch: differentiable in x, the router
    and the experts [n_experts][rows][cols]."""
    w, *grouping = RouteWeights.apply(x @ router.t(), top_k, routed_scale)
    rows = Dispatch.apply(x, top_k, *grouping)
    off = grouping[1].tolist()
    out = []
    for e in range(gate.shape[0]):
        r = rows[off[e]:off[e + 1]]
        out.append((torch.nn.functional.silu(r @ gate[e].t()) * (r @ up[e].t())) @ down[e].t())
    out.append(rows[off[-1]:])  # rows that no slot has
    return Combine.apply(torch.cat(out), w, *grouping)


def main():
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    n, hidden, inter, experts, top_k = 512, 1024, 512, 32, 4
    x = normal(n, hidden).bfloat16()
    wg, wu = normal(experts, inter, hidden, scale=hidden ** -0.5), normal(experts, inter, hidden,
                                                                         scale=hidden ** -0.5)
    wd = normal(experts, hidden, inter, scale=inter ** -0.5)
    router = normal(experts, hidden, scale=hidden ** -0.5)
    y = int8_layer(x, x.float() @ router.t(), int8_weights(wg), int8_weights(wu),
                   int8_weights(wd), top_k, base=x)
    print("int8 layer: y", tuple(y.shape), y.dtype, "rms %.3f" % y.float().square().mean().sqrt())

    params = [p.requires_grad_() for p in (router, wg, wu, wd)]
    opt = torch.optim.Adam(params, lr=1e-3)
    xf, target = x.float(), normal(n, hidden)
    for step in range(20):
        loss = (train_layer(xf, *params, top_k) - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        if step % 5 == 0 or step == 19:
            print("training step %2d: loss %.4f" % (step, loss.item()))


if __name__ == "__main__":
    main()
