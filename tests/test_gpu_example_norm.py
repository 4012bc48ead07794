"""The norm and MXFP4 example: its layers against the same layers in 64 bits,
the norm's gradients against torch's in 64 bits, the whole run."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "norm_mxfp4.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("norm_mxfp4", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _norm(s, w, eps=1e-6):
    return s * torch.rsqrt(s.square().mean(1, keepdim=True) + eps) * w


def _normal(seed, *shape, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale


def _rms_error(got, ref):
    got = got.cpu().double()
    return float((got - ref).square().mean().sqrt() / ref.square().mean().sqrt())


# E2M1 has steps of 1/2 below 2, 1 below 4, 2 below 6 and saturates, in units
# that put a block's largest value between 4 and 8.  A normal block of 32 has
# its largest at some 2.1 sigma, so sigma is about 2.6 units, and the squared
# error 0.56 / 48 + 0.32 / 12 + 0.1 / 3 + 0.02 = 0.09: 12 % of sigma.  Rows and
# weights: 17 % of a gate or an up value, 25 % of h, with h's rounding and the
# down weights' sqrt(25^2 + 13^2 + 12^2) = 31 %.  Half as much again.
LAYER = 0.46


def test_dense_layer(example):
    n, h, m = 200, 512, 256
    x, res = _normal(1, n, h).bfloat16(), _normal(2, n, h).bfloat16()
    norm = 1 + 0.1 * _normal(3, h)
    gate, up, down = _normal(4, m, h, scale=h ** -0.5), _normal(5, m, h, scale=h ** -0.5), _normal(
        6, h, m, scale=m ** -0.5)
    y, total = example.dense_layer(x.cuda(), res.cuda(), norm.cuda(),
                                   *[example.mxfp4_weights(w.cuda()) for w in (gate, up, down)])
    want = (x.float() + res.float()).bfloat16()
    assert torch.equal(total.cpu(), want)
    r = _norm(want.double(), norm.double())
    g, u, d = gate.double(), up.double(), down.double()
    ref = (torch.nn.functional.silu(r @ g.t()) * (r @ u.t())) @ d.t()
    assert _rms_error(y, ref) <= LAYER


def test_routed_layer(example):
    n, h, m, e, k = 200, 256, 128, 16, 4
    x, res = _normal(1, n, h).bfloat16(), _normal(2, n, h).bfloat16()
    norm, router = 1 + 0.1 * _normal(3, h), _normal(7, e, h, scale=h ** -0.5)
    gate, up, down = (_normal(4, e, m, h, scale=h ** -0.5), _normal(5, e, m, h, scale=h ** -0.5),
                      _normal(6, e, h, m, scale=m ** -0.5))
    y = example.routed_layer(x.cuda(), res.cuda(), norm.cuda(), router.cuda(),
                             *[example.mxfp4_weights(w.cuda()) for w in (gate, up, down)], k)
    total = (x.float() + res.float()).bfloat16().double()
    r = _norm(total, norm.double())
    logits = r.bfloat16().float() @ router.t()
    l, ids = logits.double().topk(k, dim=1)
    s = torch.nn.functional.softplus(l).sqrt()
    w = 1.5 * s / s.sum(1, keepdim=True)
    ref = torch.zeros_like(total)
    for i in range(e):
        t, j = (ids == i).nonzero(as_tuple=True)
        a = r[t]
        o = (torch.nn.functional.silu(a @ gate[i].double().t()) * (a @ up[i].double().t()))
        ref = ref.index_add(0, t, w[t, j].unsqueeze(1) * (o @ down[i].double().t()))
    assert _rms_error(y.cpu().double() - total, ref) <= LAYER


@pytest.mark.parametrize("n,h", [(5, 96), (700, 1000)])
def test_add_norm_gradients(example, n, h):
    # each value of y and of the gradients is a few roundings of sums of its
    # own terms; a dweight adds n of them: at most (n + 10) 2^-24 of 1.6
    # sqrt(n) sigma, in practice far below 2^-24 n
    args = _normal(1, n, h), _normal(2, n, h), 1 + 0.2 * _normal(3, h)
    dy, dt = _normal(4, n, h), _normal(5, n, h)
    ref_args = [t.double().requires_grad_() for t in args]
    total = ref_args[0] + ref_args[1]
    y = _norm(total, ref_args[2])
    want = torch.autograd.grad((y * dy.double()).sum() + (total * dt.double()).sum(), ref_args)
    own = [t.cuda().requires_grad_() for t in args]
    got_y, got_t = example.AddNorm.apply(*own, 1e-6)
    got = torch.autograd.grad((got_y * dy.cuda()).sum() + (got_t * dt.cuda()).sum(), own)
    for name, a, b in zip(("y", "total", "x", "residual", "weight"), (got_y, got_t) + got,
                          (y, total) + want):
        a, b = a.detach().double().cpu(), b.detach()
        assert (a - b).abs().max() <= (n + 10) * 2.0 ** -24 * b.abs().max(), name


def test_one_of_the_outputs_may_be_unused(example):
    args = [t.cuda().requires_grad_() for t in (_normal(1, 4, 64), _normal(2, 4, 64),
                                                1 + 0.2 * _normal(3, 64))]
    y, total = example.AddNorm.apply(*args, 1e-6)
    only = torch.autograd.grad(total.sum(), args, retain_graph=True)
    assert torch.equal(only[0], torch.ones_like(only[0])) and not only[2].any()
    assert torch.isfinite(torch.autograd.grad(y.sum(), args)[2]).all()


def test_the_example_runs(example, capsys):
    example.main()
    out = capsys.readouterr().out
    assert "dense layer" in out and "routed layer" in out and "training step 19" in out
