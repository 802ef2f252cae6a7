"""A mixture-of-experts MLP on the package's operators, nothing of it waiting
for the host.

    x + sum over a token's experts of weight * W2_e swiglu(W1_e norm(x))

    norm -> router -> sort -> dispatch -> experts' first linear -> gated
    activation -> experts' second linear -> combine

``MoeMlp.forward`` and ``MoeMlp.backward`` are a training step's two halves:
between the linears only 8 bits an element are kept (the first linear's output
as E4M3 under 1x128 scales), and the balance loss and the loss on the logits'
size have their gradients at the router.  ``MoeMlp.serve`` is a forward of a few
tokens, which a CUDA graph can hold: the experts that the tokens chose are known
on the device alone.

Run it:  python examples/moe_mlp.py [tokens hidden width experts topk steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import scaled_linear_layers_gb300 as fp8  # noqa: E402

EPS = 1e-5
BLOCK = 128  # rows and columns of a scale
BF, F = torch.bfloat16, torch.float32


def _empty(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda")


def quantize_rows(t):
    """E4M3 of t [rows, cols] under 1x128 scales, and of its transpose."""
    r, c = t.shape
    q, qt = _empty(torch.uint8, r, c), _empty(torch.uint8, c, r)
    scale, inv = _empty(F, r, c // BLOCK), _empty(F, r, c // BLOCK)
    scale_t, inv_t = _empty(F, r // BLOCK, c), _empty(F, r // BLOCK, c)
    fp8.fp8_quantize_transpose(t, fp8.BLOCK, scale, inv, q, qt, scale_t, inv_t)
    return q, scale, qt, scale_t


def quantize_weights(w):
    """E4M3 of w [experts, n, k] under 128x128 scales, [k, experts * n] of it too."""
    e, n, k = w.shape
    q, qt = _empty(torch.uint8, e, n, k), _empty(torch.uint8, k, e * n)
    scale, inv = (_empty(F, e, n // BLOCK, k // BLOCK) for _ in range(2))
    fp8.fp8_quantize_transpose(w.view(e * n, k), fp8.BLOCK_2D, scale, inv, q, qt)
    return q, scale, qt


class Routing:
    """The experts of a batch's tokens and the sorted order of their rows."""

    def __init__(self, logits, topk, multiple, mask=None):
        tokens, experts = logits.shape
        self.ids, self.weights = _empty(torch.int32, tokens, topk), _empty(F, tokens, topk)
        self.counts, self.live = _empty(torch.int32, experts), _empty(torch.int32, 1)
        self.losses = _empty(F, 2)
        workspace = _empty(torch.uint8, fp8.fp8_moe_route_workspace_bytes(tokens, experts))
        fp8.fp8_moe_route(logits, self.ids, self.weights, self.counts, self.live, self.losses,
                          workspace, mask=mask)
        n = tokens * topk
        self.capacity = -(-fp8.fp8_moe_capacity(n, experts, multiple) // BLOCK) * BLOCK
        self.row_of = _empty(torch.int32, tokens, topk)
        self.source = _empty(torch.int32, self.capacity)
        self.offsets, counts = _empty(torch.int32, experts + 1), _empty(torch.int32, experts)
        workspace = _empty(torch.uint8, fp8.fp8_moe_sort_workspace_bytes(n, experts))
        fp8.fp8_moe_sort(self.ids, experts, multiple, self.row_of, self.source, self.offsets,
                         counts, workspace)
        self.rows = self.offsets[experts:]  # rows that any expert has, on the device


class MoeMlp:
    def __init__(self, hidden, width, experts, topk, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda scale, *s: (scale * torch.randn(s, generator=g, device="cuda")).to(BF)  # noqa: E731
        self.hidden, self.width, self.experts, self.topk = hidden, width, experts, topk
        self.gain, self.bias = torch.ones(hidden, device="cuda"), torch.zeros(hidden, device="cuda")
        self.router = rnd(hidden ** -0.5, experts, hidden)
        self.w1 = rnd(hidden ** -0.5, experts, 2 * width, hidden)  # gate, up
        self.w2 = rnd(width ** -0.5, experts, hidden, width)
        self.quantize()

    def quantize(self):
        """The experts' E4M3 weights: once for serving, after each update in training."""
        self.q1, self.q2 = quantize_weights(self.w1), quantize_weights(self.w2)

    def forward(self, x, mask=None):
        """Output, losses [2] (balance, logits' size) and what backward needs.
        mask [tokens], 0: padding, which passes unchanged."""
        y, mean, rstd = torch.empty_like(x), _empty(F, x.shape[0]), _empty(F, x.shape[0])
        fp8.fp8_layer_norm(x, self.gain, self.bias, EPS, y, mean, rstd)
        logits = y.float() @ self.router.float().t()
        route = Routing(logits, self.topk, BLOCK, mask)
        cap, w = route.capacity, self.width
        rows = _empty(BF, cap, self.hidden)
        fp8.fp8_moe_dispatch(y, route.row_of, route.source, rows)
        xq, xs, xqt, xst = quantize_rows(rows)
        # rows behind the last segment stay as they are, in every buffer from here
        # on: nothing reads them
        h, out = _empty(BF, cap, 2 * w), _empty(BF, cap, self.hidden)
        fp8.fp8_moe_linear_fprop(xq, xs, *self.q1[:2], route.offsets, h)
        hq, hs = _empty(torch.uint8, cap, 2 * w), _empty(F, cap, 2 * w // BLOCK)
        yq, ys = _empty(torch.uint8, cap, w), _empty(F, cap, w // BLOCK)
        fp8.fp8_swiglu(h, yq=yq, y_scale=ys, hq=hq, h_scale=hs, live=route.rows)
        fp8.fp8_moe_linear_fprop(yq, ys, *self.q2[:2], route.offsets, out)
        total = torch.empty_like(x)
        fp8.fp8_moe_combine(out, route.row_of, route.weights, total)
        return x + total, route.losses, (x, y, mean, rstd, logits, route, xqt, xst, hq, hs, out)

    def backward(self, dout, dlosses, ctx):
        """Gradients by name for the output's and the losses' (fp32 [2])."""
        x, y, mean, rstd, logits, route, xqt, xst, hq, hs, out = ctx
        cap, w = route.capacity, self.width
        dout_rows, dweights = torch.empty_like(out), torch.empty_like(route.weights)
        fp8.fp8_moe_combine_backward(dout, out, route.row_of, route.source, route.weights,
                                     dout_rows, dweights)
        gq, gs, gqt, gst = quantize_rows(dout_rows)
        dact, dh, act = _empty(BF, cap, w), _empty(BF, cap, 2 * w), _empty(BF, cap, w)
        fp8.fp8_moe_linear_dgrad(gq, gs, self.q2[2], self.q2[1], route.offsets, dact)
        fp8.fp8_swiglu_backward(dact, hq, dh, h_scale=hs, y=act, live=route.rows)
        dw1, dw2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
        _, _, aqt, ast = quantize_rows(act)
        fp8.fp8_moe_linear_wgrad(gqt, gst, aqt, ast, route.offsets, dw2)
        gq, gs, gqt, gst = quantize_rows(dh)
        fp8.fp8_moe_linear_wgrad(gqt, gst, xqt, xst, route.offsets, dw1)
        drows = _empty(BF, cap, self.hidden)
        fp8.fp8_moe_linear_dgrad(gq, gs, self.q1[2], self.q1[1], route.offsets, drows)
        dy, dx, dlogits = torch.empty_like(x), torch.empty_like(x), torch.empty_like(logits)
        fp8.fp8_moe_dispatch_backward(drows, route.row_of, dy)
        fp8.fp8_moe_route_backward(logits, route.ids, route.counts, route.live, dlogits, dweights,
                                   dlosses)
        drouter = dlogits.t() @ y.float()
        dy = (dy.float() + dlogits @ self.router.float()).to(BF)
        dgain, dbias = torch.empty_like(self.gain), torch.empty_like(self.bias)
        workspace = _empty(torch.uint8, fp8.fp8_layer_norm_workspace_bytes(*x.shape))
        fp8.fp8_layer_norm_backward(dy, x, self.gain, mean, rstd, dx, dgain, dbias, workspace)
        return {"dx": dx + dout, "dw1": dw1, "dw2": dw2, "drouter": drouter, "dgain": dgain,
                "dbias": dbias}

    def serve(self, x):
        """The output for a few tokens; rows of an expert start anywhere."""
        y = torch.empty_like(x)
        fp8.fp8_layer_norm(x, self.gain, self.bias, EPS, y)
        route = Routing(y.float() @ self.router.float().t(), self.topk, 1)
        cap, w = route.capacity, self.width
        rows = _empty(BF, cap, self.hidden)
        fp8.fp8_moe_dispatch(y, route.row_of, route.source, rows)
        xq = _empty(torch.uint8, cap, self.hidden)
        xs, inv = (_empty(F, cap, self.hidden // BLOCK) for _ in range(2))
        fp8.fp8_quantize(rows, fp8.BLOCK, xs, inv, xq)
        h, out = _empty(BF, cap, 2 * w), _empty(BF, cap, self.hidden)
        fp8.fp8_moe_linear_fprop(xq, xs, *self.q1[:2], route.offsets, h)
        yq, ys = _empty(torch.uint8, cap, w), _empty(F, cap, w // BLOCK)
        fp8.fp8_swiglu(h, yq=yq, y_scale=ys, live=route.rows)
        fp8.fp8_moe_linear_fprop(yq, ys, *self.q2[:2], route.offsets, out)
        total = torch.empty_like(x)
        fp8.fp8_moe_combine(out, route.row_of, route.weights, total)
        return x + total


def main(tokens=2048, hidden=1024, width=2048, experts=8, topk=2, steps=5, lr=0.05):
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = MoeMlp(hidden, width, experts, topk)
    x, target = (torch.randn(tokens, hidden, generator=g, device="cuda").to(BF) for _ in range(2))
    dlosses = torch.tensor([1e-2, 1e-3], device="cuda")
    for i in range(steps):
        out, losses, ctx = layer.forward(x)
        off = out.float() - target.float()
        grads = layer.backward((off * (2.0 / tokens)).to(BF), dlosses, ctx)
        for name in ("router", "w1", "w2", "gain", "bias"):
            getattr(layer, name).sub_(grads["d" + name], alpha=lr)
        layer.quantize()
        fp8.fp8_check_device_status()
        print(f"step {i}: loss {off.square().mean().item():.4f} balance {losses[0].item():.4f}")
    print("served", tuple(layer.serve(x[:4]).shape))


if __name__ == "__main__":
    main(*map(int, sys.argv[1:]))
