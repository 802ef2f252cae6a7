"""The router and the experts' products where weights, outputs and logits pass
2^32 elements or bytes: the last rows and columns are those of a small call or of
the product in 64 bits (tolerance: half a unit of bf16 and k 2^-23 of the terms'
magnitudes for k terms, as every block's partial is exact in fp32's range and
takes three more roundings)."""
import pytest
import torch

import scaled_linear_layers_gb300 as fp8

pytestmark = pytest.mark.gpu
BF, F, D = torch.bfloat16, torch.float32, torch.float64
B = 128


@pytest.fixture(params=["0", "1"])
def few(request, monkeypatch):
    monkeypatch.setenv("FP8LINEAR_MOE_FEW", request.param)
    return request.param


def codes(seed, *shape):
    """E4M3 bytes of both signs, no NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8, device="cuda") & 0xF7


def scales(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(shape, generator=g, device="cuda") + 0.5


def values(q, scale, rows=1):
    """64-bit values of bytes q under tiles of rows x 128."""
    s = scale.to(D).repeat_interleave(rows, 0).repeat_interleave(B, 1)
    return q.contiguous().view(torch.float8_e4m3fn).to(D) * s


def near(got, a, b):
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    tol = 2.0 ** -8 * (1 + 2.0 ** -8) * want.abs() + (1 + 2.0 ** -7) * a.shape[1] * 2.0 ** -23 * mag
    assert ((got.to(D) - want).abs() <= tol).all()


def test_weights_past_32_bits(few):
    E, N, K, cap = 5, 32768, 32768, 7
    offsets = torch.tensor([0, 1, 2, 3, 4, 7], dtype=torch.int32, device="cuda")
    ws = scales(1, E, N // B, K // B)
    xq, xs = codes(2, cap, K), scales(3, cap, K // B)
    x = values(xq, xs)
    w = codes(4, E, N, K)
    y = torch.empty(cap, N, dtype=BF, device="cuda")
    fp8.fp8_moe_linear_fprop(xq, xs, w, ws, offsets, y)
    for e in (0, 4):
        rows = slice(int(offsets[e]), int(offsets[e + 1]))
        for n in (slice(0, 256), slice(N - 256, N)):
            near(y[rows, n], x[rows], values(w[e, n], ws[e, n.start // B:n.stop // B], B))
    wt = w.view(K, E * N)  # other weights, their bytes [K, E N]
    fp8.fp8_moe_linear_dgrad(xq, xs, wt, ws, offsets, y)
    for e in (0, 4):
        rows = slice(int(offsets[e]), int(offsets[e + 1]))
        for k in (slice(0, 256), slice(K - 256, K)):
            wk = values(wt[k, e * N:(e + 1) * N], ws[e, :, k.start // B:k.stop // B].t(), B)
            near(y[rows, k], x[rows], wk)
    fp8.fp8_check_device_status()


def test_rows_past_32_bits(few):
    N, K, cap = 65536, 128, 70016
    offsets = torch.tensor([0, 100, cap], dtype=torch.int32, device="cuda")
    xq, xs, w, ws = codes(5, cap, K), scales(6, cap, 1), codes(7, 2, N, K), scales(8, 2, N // B, 1)
    y = torch.empty(cap, N, dtype=BF, device="cuda")
    fp8.fp8_moe_linear_fprop(xq, xs, w, ws, offsets, y)
    last = slice(cap - 200, cap)
    near(y[last, -512:], values(xq[last], xs[last]), values(w[1, -512:], ws[1, -4:], B))
    near(y[:100, :512], values(xq[:100], xs[:100]), values(w[0, :512], ws[0, :4], B))
    fp8.fp8_check_device_status()


def test_weight_gradients_past_32_bits():
    N = K = 40960
    offsets = torch.tensor([0, 128, 128, 384], dtype=torch.int32, device="cuda")
    gqt, gs, xqt, xs = codes(9, N, 384), scales(10, 3, N), codes(11, K, 384), scales(12, 3, K)
    dw = torch.empty(3, N, K, dtype=BF, device="cuda")
    fp8.fp8_moe_linear_wgrad(gqt, gs, xqt, xs, offsets, dw)
    near(dw[2, -256:, -512:], values(gqt[-256:, 128:], gs[1:, -256:].t()),
         values(xqt[-512:, 128:], xs[1:, -512:].t()))
    assert (dw[1, -256:, -512:] == 0).all()
    fp8.fp8_check_device_status()


def test_logits_past_32_bits():
    tokens, experts, topk = (1 << 22) + 5, 1024, 32
    g = torch.Generator(device="cuda").manual_seed(13)
    logits = torch.empty(tokens, experts, dtype=BF, device="cuda").normal_(generator=g)

    def run(x):
        t = x.shape[0]
        ids = torch.empty(t, topk, dtype=torch.int32, device="cuda")
        weights = torch.empty(t, topk, device="cuda")
        counts = torch.empty(experts, dtype=torch.int32, device="cuda")
        live, losses = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(2, device="cuda")
        ws = torch.empty(fp8.fp8_moe_route_workspace_bytes(t, experts), dtype=torch.uint8, device="cuda")
        fp8.fp8_moe_route(x, ids, weights, counts, live, losses, ws)
        return ids, weights, counts, live, losses

    ids, weights, counts, live, losses = run(logits)
    part = logits[-300:].clone()
    small = run(part)
    assert torch.equal(ids[-300:], small[0]) and torch.equal(weights[-300:], small[1])
    assert live.item() == tokens and counts.sum().item() == tokens * topk
    # both losses are means over many even tokens: 1, and the mean of (log 1024 + 1/2)^2
    assert abs(losses[0].item() - 1) < 1e-2 and abs(losses[1].item() / 7.4315 ** 2 - 1) < 1e-2
    dweights = torch.randn(tokens, topk, generator=g, device="cuda")
    dlosses = torch.tensor([1.0, 0.1], device="cuda") * tokens
    grad, few_grad = torch.empty_like(logits), torch.empty_like(part)
    fp8.fp8_moe_route_backward(logits, ids, counts, live, grad, dweights, dlosses)
    fp8.fp8_moe_route_backward(part, small[0], counts, live, few_grad, dweights[-300:].clone(), dlosses)
    assert torch.equal(grad[-300:], few_grad)
