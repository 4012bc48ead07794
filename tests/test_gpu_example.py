"""The example's layers: the int8 layer against the same layer in 64 bits, the
training step's gradients against torch's in 64 bits."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "experts_around.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("experts_around", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _layer(x, router, gate, up, down, k):
    """The definition, in x's dtype, on the CPU."""
    logits = x @ router.t()
    l, ids = logits.topk(k, dim=1)
    s = torch.nn.functional.softplus(l).sqrt()
    w = 1.5 * s / s.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(gate.shape[0]):
        t, i = (ids == e).nonzero(as_tuple=True)
        r = x[t]
        o = (torch.nn.functional.silu(r @ gate[e].t()) * (r @ up[e].t())) @ down[e].t()
        y = y.index_add(0, t, w[t, i].unsqueeze(1) * o)
    return y


def _inputs(n, h, m, e):
    g = torch.Generator().manual_seed(n)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    return (normal(n, h), normal(e, h) * h ** -0.5, normal(e, m, h) * h ** -0.5,
            normal(e, m, h) * h ** -0.5, normal(e, h, m) * m ** -0.5)


def test_int8_layer(example):
    # A row of normals has its largest value at 3 to 4.5 sigma: a step of at
    # most 4.5 / 127 sigma, an error of step / sqrt(12) = 1 % of a value, in x
    # and in each weight row; the SwiGLU output is longer-tailed (10 sigma and
    # more: 2.5 %).  Four such errors of 1 % for gate and up, one more for the
    # down matrix and h's: sqrt(5 * 1 + 2.5 ** 2) = 3.4 %.  Twice that.
    x, router, gate, up, down = _inputs(200, 256, 128, 16)
    x = x.bfloat16()
    base = x * 0.5
    y = example.int8_layer(x.cuda(), (x.float() @ router.t()).cuda(),
                           *[example.int8_weights(w.cuda()) for w in (gate, up, down)], 4,
                           base=base.cuda()).cpu().double()
    ref = _layer(*[t.double() for t in (x, router, gate, up, down)], 4)
    err = (y - base.double() - ref).square().mean().sqrt() / ref.square().mean().sqrt()
    assert err <= 0.068, err


def test_training_step_gradients(example):
    # fp32 products of up to 256 terms and their gradients: each some
    # sqrt(256) * 2^-24 of its terms, a few of them one after the other
    args = _inputs(96, 256, 64, 12)
    dy = torch.randn(96, 256, generator=torch.Generator().manual_seed(5))
    ref_args = [t.double().requires_grad_() for t in args]
    ref = _layer(*ref_args, 3)
    want = torch.autograd.grad((ref * dy.double()).sum(), ref_args)
    own_args = [t.cuda().requires_grad_() for t in args]
    y = example.train_layer(*own_args, 3)
    got = torch.autograd.grad((y * dy.cuda()).sum(), own_args)
    for name, a, b in zip(("y", "x", "router", "gate", "up", "down"), (y,) + got, (ref,) + want):
        a, b = a.detach().double().cpu(), b.detach()
        assert (a - b).abs().max() <= 2e-5 * b.abs().max(), name
