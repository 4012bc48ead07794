"""A residual stream through norms and MXFP4 layers as it serves, and a training
step through the norm with its residual.

    python examples/norm_mxfp4.py
"""

import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from block_quantized_expert_amd import binding as B  # noqa: E402


def mxfp4_weights(w):
    """Rows of w [rows][cols] or [n_experts][rows][cols] rounded to MXFP4."""
    c = w.shape[-1]
    codes, scales = B.moe_quantize_mxfp4(w.reshape(-1, c))
    return B.Mxfp4Weight(codes.view(*w.shape[:-1], c // 2),
                         B.mxfp4_scale_rows(scales, c).view(*w.shape[:-1], c // 32))


def dense_layer(x, residual, norm, gate, up, down):
    """(y, total): the dense FFN of the normed total = x + residual; norm and
    rounding are one call."""
    codes, scales, total = B.moe_rmsnorm_mxfp4(x, norm, residual=residual)
    h = B.moe_swiglu_mxfp4(gate, up, codes, scales)
    return B.moe_product_mxfp4(down, *B.moe_quantize_mxfp4(h)), total


def routed_layer(x, residual, norm, router, gate, up, down, top_k, routed_scale=1.5):
    """The stream behind a routed FFN: total + the experts' weighted sum.  The
    router reads the normed rows, so norm and rounding are two calls."""
    y, total = B.moe_rmsnorm(x, norm, residual=residual)
    _, w, grouping = B.moe_route_group(y.float() @ router.t(), top_k, routed_scale)
    h = B.moe_swiglu_mxfp4(gate, up, *B.moe_quantize_mxfp4(y), grouping, top_k=top_k)
    rows = B.moe_product_mxfp4(down, *B.moe_quantize_mxfp4(h), grouping)
    return B.moe_combine(rows, w, grouping, base=total)


class AddNorm(torch.autograd.Function):
    """(y, total) of total = x + residual and its norm; what flows back into
    total by its further use is added in the same pass."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        y, total = B.moe_rmsnorm(x, weight, eps, residual=residual)
        ctx.save_for_backward(total, weight)
        ctx.eps, ctx.types = eps, (x.dtype, residual.dtype)
        return y, total

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dtotal):
        total, weight = ctx.saved_tensors
        want = ctx.needs_input_grad[2]  # not of a frozen weight
        d = B.moe_rmsnorm_backward(dy.contiguous(), total, weight, ctx.eps,
                                   dtotal=dtotal.contiguous(), need_dweight=want)
        d, dw = (d[0], d[1].to(weight.dtype)) if want else (d, None)
        return d.to(ctx.types[0]), d.to(ctx.types[1]), dw, None


def main():
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    n, hidden, inter, experts, top_k = 512, 1024, 512, 32, 4
    x, residual = normal(n, hidden).bfloat16(), normal(n, hidden).bfloat16()
    norm = 1 + 0.1 * normal(hidden)
    gate, up = (mxfp4_weights(normal(inter, hidden, scale=hidden ** -0.5)) for _ in range(2))
    down = mxfp4_weights(normal(hidden, inter, scale=inter ** -0.5))
    y, total = dense_layer(x, residual, norm, gate, up, down)
    print("dense layer: y", tuple(y.shape), y.dtype, "rms %.3f" % y.float().square().mean().sqrt())
    gate, up = (mxfp4_weights(normal(experts, inter, hidden, scale=hidden ** -0.5))
                for _ in range(2))
    down = mxfp4_weights(normal(experts, hidden, inter, scale=inter ** -0.5))
    router = normal(experts, hidden, scale=hidden ** -0.5)
    y = routed_layer(y, total, norm, router, gate, up, down, top_k)
    print("routed layer: stream", tuple(y.shape), y.dtype,
          "rms %.3f" % y.float().square().mean().sqrt())

    params = [p.requires_grad_() for p in (norm, normal(hidden, hidden, scale=hidden ** -0.5))]
    opt = torch.optim.Adam(params, lr=1e-3)
    xf, rf, target = x.float(), residual.float(), normal(n, hidden)
    for step in range(20):
        y, total = AddNorm.apply(xf, rf, params[0], 1e-6)
        loss = (total + y @ params[1] - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        if step % 5 == 0 or step == 19:
            print("training step %2d: loss %.4f" % (step, loss.item()))


if __name__ == "__main__":
    main()
