"""The 8-bit training example: its weight gradients against torch's in 64 bits, and its loss."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

gp = pytest.importorskip("gpu_path")


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "q8_training.py")
    spec = importlib.util.spec_from_file_location("q8_training", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,width,hidden", [(300, 256, 384), (128, 100, 260)])
def test_gradients(example, tokens, width, hidden):
    """Against the layer in 64 bits, from the same weights and inputs.  What differs is the storage
    in 8 bits: independent roundings of at most 2^-4 (e4m3) or 2^-3 (e5m2) of a value, on average
    below half of that.  A gradient passes at most three of e4m3 (weight, input, activation) and two
    of e5m2: in the root of the sum of squares below sqrt(3 * 2^-10 + 2 * 2^-8) = 0.11."""
    gp.say(f"q8 example gradients {tokens}x{width}x{hidden}")
    torch.manual_seed(1)
    layer = example.FeedForward(tokens, width, hidden)
    layer.weights_to_8_bits()
    x = example.matrix(tokens, width)
    x.copy_(torch.randn((tokens, width), device="cuda"))
    d = example.matrix(tokens, width)
    d.copy_(torch.randn((tokens, width), device="cuda") * 1e-3)
    row = torch.full((layer.n,), 7.0, device="cuda")
    layer.forward(x)
    layer.backward(d, row)
    w = [t.double().cpu().requires_grad_() for t in (layer.wg, layer.wu, layer.wd)]
    xd = x.double().cpu()
    out = (torch.nn.functional.silu(xd @ w[0].t()) * (xd @ w[1].t())) @ w[2].t()
    assert (layer.out.double().cpu() - out).norm() < 0.11 * out.norm()
    out.backward(d.double().cpu())
    for got, want in zip(layer.views(row), w):
        assert (got.double().cpu() - want.grad).norm() < 0.11 * want.grad.norm()


def test_training_learns(example):
    gp.say("q8 example training")
    losses = example.train(steps=30, log=None)
    assert all(l == l for l in losses)
    assert losses[-1] < 0.5 * losses[0]


def test_readme_examples():
    """Every Python example of README.md, one after the other; the 8-bit layer against its inputs.
    A value is off by at most 2^-4 of itself after storage: y by the sum of |x w| times
    2 * 2^-4 + 2^-8 and its rounding, dw (dy is ones) by the sum of |x| times 2^-4; each doubled for
    values below their format's normal range."""
    import re
    gp.say("readme examples")
    src = open(os.path.join(os.path.dirname(__file__), "..", "README.md")).read()
    env: dict = {}
    for code in re.findall(r"```python\n(.*?)```", src, re.S):
        exec(compile(code, "README.md", "exec"), env)
    torch.cuda.synchronize()
    x, w = env["x"].double().cpu(), env["w"].double().cpu()
    y, dw = env["y"].double().cpu(), env["grads"][0, :w.numel()].view(w.shape).double().cpu()
    mass = x.abs() @ w.abs().t()
    assert bool(((y - x @ w.t()).abs() <= 2 * (2 * 2.0 ** -4 + 2.0 ** -8) * mass).all())
    want = x.sum(0).expand_as(w)
    assert bool(((dw - want).abs() <= 2 * 2.0 ** -4 * x.abs().sum(0)).all())


def test_training_learns_with_fast_products(example):
    gp.say("q8 example training, fast")
    losses = example.train(steps=30, log=None, fast=True)
    assert all(l == l for l in losses)
    assert losses[-1] < 0.5 * losses[0]
