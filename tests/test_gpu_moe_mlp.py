"""The router, the experts' products and the gated activation together, with the
norm and the expert rows, as examples/moe_mlp.py runs them: against the same MLP
in 64 bits.  E4M3 holds 4 bits, so an operand is 2^-4/sqrt(3) = 3.6 % off at most
in the 2-norm and a product of two 5.1 %.  Forward: gate and up 5.1 % each, their
activation 1.2 sqrt(2) 5.1 % (1.2 bounds the slope of silu against its value in
the mean), the second product with its own two operands 10.1 %.  Gradients: dact
5.1 %, the checkpoint's gate and up sqrt(5.1^2 + 3.6^2) = 6.2 % each, and one more
product: sqrt(5.1^2 + 2 6.2^2 + 5.1^2) = 11.4 %.  15 % bounds both."""
import importlib.util
import os

import pytest
import torch

import scaled_linear_layers_gb300 as fp8

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOL = 0.15


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_mlp",
                                                  os.path.join(ROOT, "examples", "moe_mlp.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def near(got, want, tol=TOL):
    got, want = got.double(), want.double()
    return (got - want).norm().item() <= tol * want.norm().item()


def plain(layer, x, ids, on):
    """Output, losses and leaves in 64 bits with autograd, for the experts ids."""
    leaves = {"d" + n: getattr(layer, n).detach().double().requires_grad_()
              for n in ("router", "w1", "w2", "gain", "bias")}
    leaves["dx"] = x = x.detach().double().requires_grad_()
    xc = x - x.mean(1, keepdim=True)
    y = xc / (xc.square().mean(1, keepdim=True) + 1e-5).sqrt() * leaves["dgain"] + leaves["dbias"]
    logits = y @ leaves["drouter"].t()
    p = torch.softmax(logits, 1)
    at = ids.clamp(min=0).long()
    weights = p.gather(1, at)
    weights = weights / weights.sum(1, keepdim=True)
    total = torch.zeros_like(x)
    for j in range(ids.shape[1]):
        h = torch.einsum("th,tnh->tn", y, leaves["dw1"][at[:, j]])
        gate, up = h.chunk(2, 1)
        act = torch.nn.functional.silu(gate) * up
        total = total + weights[:, j:j + 1] * torch.einsum("tw,thw->th", act, leaves["dw2"][at[:, j]])
    n, e, k = on.sum(), p.shape[1], ids.shape[1]
    counts = torch.bincount(at[on].reshape(-1), minlength=e).double()
    balance = e * (counts / (n * k) * (p[on].sum(0) / n)).sum()
    z = torch.logsumexp(logits[on], 1).square().sum() / n
    return x + on[:, None] * total, torch.stack([balance, z]), leaves


@pytest.mark.parametrize("tokens, hidden, width, experts, topk, padding",
                         [(200, 256, 128, 4, 2, 0), (37, 128, 256, 16, 4, 9), (1, 128, 128, 3, 1, 0)])
def test_training_step(example, tokens, hidden, width, experts, topk, padding):
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    layer = example.MoeMlp(hidden, width, experts, topk)
    x, dout = rnd(tokens, hidden).bfloat16(), (1e-2 * rnd(tokens, hidden)).bfloat16()
    mask = torch.arange(tokens, device="cuda") < tokens - padding
    dlosses = torch.tensor([0.3, 0.02], device="cuda")
    out, losses, ctx = layer.forward(x, mask)
    grads = layer.backward(dout, dlosses, ctx)
    fp8.fp8_check_device_status()
    ids = ctx[5].ids
    assert torch.equal(ids[:, 0] >= 0, mask)
    want, want_losses, leaves = plain(layer, x, ids, mask)
    ((want * dout.double()).sum() + (want_losses * dlosses.double()).sum()).backward()
    assert near(out - x, want - x)
    # y is bf16, so logits are 2^-8 |l| off at most
    assert torch.allclose(losses.double(), want_losses, rtol=0.02)
    for name, leaf in leaves.items():
        assert near(grads[name], leaf.grad), name
    assert torch.equal(out[~mask], x[~mask])


def test_serving_from_one_graph(example):
    """A captured forward serves tokens that choose other experts at each replay,
    with the bits of an eager call."""
    layer = example.MoeMlp(256, 384, 16, 4, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    inputs = [torch.randn(5, 256, generator=g, device="cuda").bfloat16() for _ in range(4)]
    eager = [layer.serve(x) for x in inputs]
    held = inputs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        served = layer.serve(held)
    for x, want in zip(inputs, eager):
        held.copy_(x)
        graph.replay()
        assert torch.equal(served, want)
    for x, want in zip(inputs, eager):
        assert near(layer.forward(x)[0] - x, want - x)
        one = torch.cat([layer.serve(x[i:i + 1]) for i in range(5)])
        assert near(one - x, want - x, 1e-2)
    fp8.fp8_check_device_status()


def test_example_runs(example, capsys):
    example.main(tokens=128, hidden=128, width=128, experts=4, steps=2)
    assert "served (4, 128)" in capsys.readouterr().out
