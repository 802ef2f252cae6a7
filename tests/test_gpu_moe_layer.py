"""The mixture-of-experts layer of examples/moe_layer.py: the norm, dispatch,
FP8 linear, combine and update operators together, against the same layer in
64 bits.  E4M3 holds 4 bits, so an operand is 2^-4/sqrt(3) = 3.6 % off at most
and a product of two 5 %; gradients pass two such products: 10 % bounds both in
the 2-norm."""
import importlib.util
import os

import pytest
import torch

import scaled_linear_layers_gb300 as fp8

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_layer",
                                                  os.path.join(ROOT, "examples", "moe_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def near(got, want, tol):
    got, want = got.double(), want.double()
    return (got - want).norm().item() <= tol * want.norm().item()


def plain(layer, x, ids, weights):
    """The layer in 64 bits with autograd."""
    x, w, rw = (t.detach().double().requires_grad_() for t in (x, layer.w, weights))
    gain = layer.gain.double().requires_grad_()
    bias = layer.bias.double().requires_grad_()
    xc = x - x.mean(1, keepdim=True)
    y = xc / (xc.square().mean(1, keepdim=True) + 1e-5).sqrt() * gain + bias
    out = x
    for j in range(ids.shape[1]):
        out = out + rw[:, j:j + 1] * torch.einsum("th,tnh->tn", y, w[ids[:, j]])
    return out, {"dx": x, "dw": w, "dweights": rw, "dgain": gain, "dbias": bias}


@pytest.mark.parametrize("tokens, hidden, experts, topk", [(200, 256, 4, 2), (37, 128, 16, 4)])
def test_training_step(example, tokens, hidden, experts, topk):
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    layer = example.MoeLayer(hidden, experts)
    x, dout = rnd(tokens, hidden).bfloat16(), (1e-2 * rnd(tokens, hidden)).bfloat16()
    ids, weights = example.route_tokens(rnd(tokens, experts), topk)
    want, leaves = plain(layer, x, ids, weights)
    (want * dout.double()).sum().backward()
    before = layer.w.clone()
    out, grads = layer.step(x, ids, weights, dout)
    assert near(out, want, 0.1)
    for name, leaf in leaves.items():
        assert near(grads[name], leaf.grad, 0.1), name
    # the weights moved by lr times a matrix whose singular values are near 1
    moved = (before.double() - layer.w.double())[0] / 0.02
    s = torch.linalg.svdvals(moved.cpu())
    assert 0.3 < s[: hidden // 8].mean() < 1.4


def test_serving_matches_the_training_forward(example):
    g = torch.Generator(device="cuda").manual_seed(4)
    layer = example.MoeLayer(256, 8)
    x = torch.randn(64, 256, generator=g, device="cuda").bfloat16()
    ids, weights = example.route_tokens(torch.randn(64, 8, generator=g, device="cuda"), 2)
    want, _ = layer.forward(x, ids, weights)
    assert near(layer.serve(x[:1], ids[:1], weights[:1]), want[:1], 0.1)
    assert near(layer.serve(x, ids, weights), want, 0.1)
    fp8.fp8_check_device_status()


def test_example_runs(example, capsys):
    example.main(tokens=128, hidden=128, experts=4, steps=2)
    assert "served (4, 128)" in capsys.readouterr().out
