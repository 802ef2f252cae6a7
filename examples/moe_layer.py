"""One mixture-of-experts layer on the package's operators.

The layer is ``x + sum over a token's experts of weight * W_e norm(x)`` with
one FP8 linear an expert, a stand-in for an expert's MLP:

    norm -> sort -> dispatch -> each expert's FP8 linear -> combine

``MoeLayer.step`` is a training step: forward, backward (combine, the linears'
two products, dispatch, norm) and the update of the experts' weights by their
orthogonalised gradients.  ``MoeLayer.serve`` is a forward of a few tokens
whose rows are dispatched as E4M3 bytes under a scale kept from training, so
the linears take them as they are.

Run it:  python examples/moe_layer.py [tokens hidden experts topk steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import scaled_linear_layers_gb300 as fp8  # noqa: E402

EPS = 1e-5
MULTIPLE = 16  # rows of an expert's segment: what the tensorwise FP8 GEMMs take


def _empty(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda")


class Routing:
    """The sorted order of one batch's assignments (ids [tokens, topk])."""

    def __init__(self, ids, experts):
        n = ids.numel()
        self.capacity = fp8.fp8_moe_capacity(n, experts, MULTIPLE)
        self.row_of = _empty(torch.int32, *ids.shape)
        self.source = _empty(torch.int32, self.capacity)
        self.offsets = _empty(torch.int32, experts + 1)
        self.counts = _empty(torch.int32, experts)
        workspace = _empty(torch.uint8, fp8.fp8_moe_sort_workspace_bytes(n, experts))
        fp8.fp8_moe_sort(ids, experts, MULTIPLE, self.row_of, self.source, self.offsets,
                         self.counts, workspace)

    def segments(self):
        """[(expert, first row, past the last row)] of the experts with rows.
        The linears' sizes are host arguments, so this waits for the sort."""
        at = self.offsets.tolist()
        return [(e, lo, hi) for e, (lo, hi) in enumerate(zip(at, at[1:])) if hi > lo]


def _quantized(t):
    """E4M3 bytes of t, of its transpose, and the scale (current scaling)."""
    r, c = t.shape
    q, qt = _empty(torch.uint8, r, c), _empty(torch.uint8, c, r)
    scale, inv, amax = (_empty(torch.float32, 1) for _ in range(3))
    fp8.fp8_quantize_transpose(t, fp8.DYNAMIC, scale, inv, q, qt, amax_out=amax)
    return q, qt, scale


class MoeLayer:
    def __init__(self, hidden, experts, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.experts = hidden, experts
        self.gain = torch.ones(hidden, device="cuda")
        self.bias = torch.zeros(hidden, device="cuda")
        self.w = (torch.randn(experts, hidden, hidden, generator=g, device="cuda")
                  * hidden ** -0.5).to(torch.bfloat16)
        self.scale, self.scale_inv = (torch.ones(1, device="cuda") for _ in range(2))
        self.update_workspace = _empty(
            torch.uint8, fp8.fp8_orthogonalize_workspace_bytes(experts, hidden, hidden))

    def forward(self, x, ids, weights):
        """The layer's output and what backward needs."""
        tokens = x.shape[0]
        y, mean, rstd = torch.empty_like(x), _empty(torch.float32, tokens), _empty(
            torch.float32, tokens)
        amax = _empty(torch.float32, 1)
        fp8.fp8_layer_norm(x, self.gain, self.bias, EPS, y, mean, rstd, amax_out=amax)
        torch.div(amax.clamp(min=1e-12), 448.0, out=self.scale)   # for serve()
        torch.reciprocal(self.scale, out=self.scale_inv)
        route = Routing(ids, self.experts)
        rows = _empty(torch.bfloat16, route.capacity, self.hidden)
        fp8.fp8_moe_dispatch(y, route.row_of, route.source, rows)
        outs, saved = torch.zeros_like(rows), []
        for e, lo, hi in route.segments():
            xq, xqt, xs = _quantized(rows[lo:hi])
            wq, wqt, ws = _quantized(self.w[e])
            fp8.fp8_linear_fprop(xq, xs, wq, ws, hi - lo, self.hidden, self.hidden, fp8.DYNAMIC,
                                 None, outs[lo:hi])
            saved.append((e, lo, hi, xqt, xs, wqt, ws))
        out = torch.empty_like(x)
        fp8.fp8_moe_combine(outs, route.row_of, weights, out)
        return x + out, (x, mean, rstd, route, weights, outs, saved)

    def backward(self, dout, ctx):
        """Gradients by name: dx, dweights (of the routing), dw [experts, ...],
        dgain, dbias."""
        x, mean, rstd, route, weights, outs, saved = ctx
        h = self.hidden
        douts, dweights = torch.empty_like(outs), torch.empty_like(weights)
        fp8.fp8_moe_combine_backward(dout, outs, route.row_of, route.source, weights, douts,
                                     dweights)
        drows, dw = torch.zeros_like(outs), torch.zeros_like(self.w)
        for e, lo, hi, xqt, xs, wqt, ws in saved:
            gq, gqt, gs = _quantized(douts[lo:hi])
            fp8.fp8_linear_dgrad_wgrad(gq, gqt, gs, wqt, ws, xqt, xs, hi - lo, h, h, fp8.DYNAMIC,
                                       drows[lo:hi], dw[e])
        dy, dx = torch.empty_like(x), torch.empty_like(x)
        fp8.fp8_moe_dispatch_backward(drows, route.row_of, dy)
        dgain, dbias = torch.empty_like(self.gain), torch.empty_like(self.bias)
        workspace = _empty(torch.uint8, fp8.fp8_layer_norm_workspace_bytes(*x.shape))
        fp8.fp8_layer_norm_backward(dy, x, self.gain, mean, rstd, dx, dgain, dbias, workspace)
        return {"dx": dx + dout, "dweights": dweights, "dw": dw, "dgain": dgain, "dbias": dbias}

    def step(self, x, ids, weights, dout, lr=0.02):
        """A training step; returns the output and the gradients."""
        out, ctx = self.forward(x, ids, weights)
        grads = self.backward(dout, ctx)
        update = torch.empty_like(grads["dw"])
        fp8.fp8_orthogonalize(grads["dw"], update, self.update_workspace)
        self.w.sub_(update, alpha=lr)
        self.gain.sub_(grads["dgain"], alpha=lr)
        self.bias.sub_(grads["dbias"], alpha=lr)
        fp8.fp8_check_device_status()
        return out, grads

    def serve(self, x, ids, weights):
        """A forward whose dispatch casts the tokens straight to E4M3."""
        y = torch.empty_like(x)
        fp8.fp8_layer_norm(x, self.gain, self.bias, EPS, y)
        route = Routing(ids, self.experts)
        rows = _empty(torch.uint8, route.capacity, self.hidden)
        fp8.fp8_moe_dispatch(y, route.row_of, route.source, rows, scale_inv=self.scale_inv)
        outs = torch.zeros(route.capacity, self.hidden, dtype=torch.bfloat16, device="cuda")
        for e, lo, hi in route.segments():
            wq, _, ws = _quantized(self.w[e])
            fp8.fp8_linear_fprop(rows[lo:hi], self.scale, wq, ws, hi - lo, self.hidden,
                                 self.hidden, fp8.DYNAMIC, None, outs[lo:hi])
        out = torch.empty_like(x)
        fp8.fp8_moe_combine(outs, route.row_of, weights, out)
        return x + out


def route_tokens(logits, topk):
    """ids and weights of each token's topk experts."""
    weights, ids = torch.topk(torch.softmax(logits.float(), 1), topk, dim=1)
    return ids.contiguous(), weights.contiguous()


def main(tokens=2048, hidden=1024, experts=8, topk=2, steps=5):
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = MoeLayer(hidden, experts)
    target = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    ids, weights = route_tokens(torch.randn(tokens, experts, generator=g, device="cuda"), topk)
    for i in range(steps):
        out, ctx = layer.forward(x, ids, weights)
        loss = (out.float() - target.float()).square().mean()
        dout = ((out.float() - target.float()) * (2.0 / tokens)).to(torch.bfloat16)
        layer.step(x, ids, weights, dout)
        print(f"step {i}: loss {loss.item():.4f}")
    one = layer.serve(x[:4], ids[:4], weights[:4])
    print("served", tuple(one.shape))


if __name__ == "__main__":
    main(*map(int, sys.argv[1:]))
