"""The examples' autograd functions: a second derivative, which the calls do not
have, is refused instead of left out; gradients that nobody wants are not taken."""

import importlib.util
import os

import pytest
import torch

from block_quantized_expert_amd import binding as B

pytestmark = pytest.mark.gpu

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


def _load(name):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location(name, os.path.join(EXAMPLES, name + ".py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


@pytest.mark.parametrize("of", [0, 1])
def test_add_norm_refuses_second_derivatives(of):
    example = _load("norm_mxfp4")
    args = [_normal(1, 4, 64).requires_grad_(), _normal(2, 4, 64).requires_grad_(),
            (1 + 0.2 * _normal(3, 64)).requires_grad_()]
    out = example.AddNorm.apply(*args, 1e-6)[of].square().sum()
    grads = torch.autograd.grad(out, args, create_graph=True)
    plain = torch.autograd.grad(example.AddNorm.apply(*args, 1e-6)[of].square().sum(), args)
    assert all(torch.equal(a, b) for a, b in zip(grads, plain))
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grads[0].square().sum().backward()


@pytest.mark.parametrize("frozen", [False, True])
def test_add_norm_takes_the_weights_gradient_where_it_is_wanted(frozen, monkeypatch):
    example = _load("norm_mxfp4")
    x, r = _normal(1, 5, 96).requires_grad_(), _normal(2, 5, 96).requires_grad_()
    w = (1 + 0.2 * _normal(3, 96)).requires_grad_(not frozen)
    asked = []
    call = B.moe_rmsnorm_backward

    def seen(*args, **kw):
        asked.append(kw.get("need_dweight", True))
        return call(*args, **kw)

    monkeypatch.setattr(B, "moe_rmsnorm_backward", seen)
    y, total = example.AddNorm.apply(x, r, w, 1e-6)
    (y * _normal(4, 5, 96) + total).sum().backward()
    assert asked == [not frozen] and (w.grad is None) == frozen
    s = (x + r).detach()
    dx = call(_normal(4, 5, 96), s, w.detach(), 1e-6, dtotal=torch.ones_like(s),
              need_dweight=False)
    assert torch.equal(x.grad, dx) and torch.equal(r.grad, dx)


def test_experts_around_refuse_second_derivatives():
    example = _load("experts_around")
    n, h, m, e, k = 6, 32, 16, 4, 2
    x = _normal(1, n, h).requires_grad_()
    params = [t.requires_grad_() for t in (_normal(2, e, h), _normal(3, e, m, h),
                                           _normal(4, e, m, h), _normal(5, e, h, m))]
    y = example.train_layer(x, *params, k)
    grads = torch.autograd.grad(y.square().sum(), [x] + params, create_graph=True)
    assert all(bool(torch.isfinite(g).all()) for g in grads)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grads[0].square().sum().backward()


def test_each_function_of_experts_around_refuses_second_derivatives():
    example = _load("experts_around")
    n, h, e, k = 6, 32, 4, 2
    logits, x = _normal(1, n, e).requires_grad_(), _normal(2, n, h).requires_grad_()
    w, *grouping = example.RouteWeights.apply(logits, k, 1.5)
    rows = example.Dispatch.apply(x, k, *grouping)
    y = example.Combine.apply(rows, w, *grouping)
    for out, into in ((w, logits), (rows, x), (y, rows), (y, w)):
        g, = torch.autograd.grad(out.square().sum(), into, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.square().sum().backward()
