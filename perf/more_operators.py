"""Cases for the router, the experts' FP8 products and the gated activation.

The three operators that a mixture-of-experts MLP needs beside the sort,
dispatch and combine of its rows:

- the router (``route*``): each token's top-k experts, their weights, the
  experts' counts, the balance loss and the loss on the logits' size; and the
  gradient of the weights and losses at the logits;
- the experts' linears (``moe_*``): the products of E4M3 rows sorted by expert
  with each expert's weight under the block recipe (1x128 tiles of rows,
  128x128 tiles of weights), forward and both gradients;
- the gated activation between an expert's two linears (``swiglu*``): forward,
  with the next linear's E4M3 operand and an 8-bit checkpoint of its input, and
  backward from that checkpoint.

``run`` computes each in its plain form (32-bit elementary operations, rounded
once at the end) or, where ``own`` is true, by the package's entry points.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOP_FLOPS = 2 * 32768 * 4096 * 14336


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # eight tokens of a decode step choose 8 of 64 experts: pure latency
        {"name": "route 8x64 top8", "op": "route", "tokens": 8, "experts": 64, "topk": 8,
         "dtype": "bf16", "renormalize": True, "padding": 0.0, "closed": 0.0},
        # a training batch over many small experts, logits kept in fp32
        {"name": "route f32 16384x256 top8", "op": "route", "tokens": 16384, "experts": 256,
         "topk": 8, "dtype": "f32", "renormalize": True, "padding": 0.0, "closed": 0.0},
        # the gradients of the same batch's weights and losses
        {"name": "route_bwd f32 16384x256 top8", "op": "route_bwd", "tokens": 16384,
         "experts": 256, "topk": 8, "dtype": "f32", "renormalize": True, "padding": 0.0,
         "closed": 0.0},
        # a padded batch, an odd number of experts of which half are closed to
        # a token, weights as the softmax gives them
        {"name": "route_bwd 5003x61 top6", "op": "route_bwd", "tokens": 5003, "experts": 61,
         "topk": 6, "dtype": "bf16", "renormalize": False, "padding": 0.2, "closed": 0.5},
        # eight tokens of a decode step through 64 experts: the weights of the
        # experts that were chosen are all that is read
        {"name": "moe_fprop 8x4096x2048 8of64", "op": "moe_fprop", "tokens": 8, "k": 4096,
         "n": 2048, "experts": 64, "topk": 8, "multiple": 16},
        # a training batch through the gate and up projections of 8 experts of
        # the MLP workload's size
        {"name": "moe_fprop 8192x4096x28672 2of8", "op": "moe_fprop", "tokens": 8192, "k": 4096,
         "n": 28672, "experts": 8, "topk": 2, "multiple": 128},
        # the input gradient of many small experts
        {"name": "moe_dgrad 8192x4096x2048 8of64", "op": "moe_dgrad", "tokens": 8192, "k": 4096,
         "n": 2048, "experts": 64, "topk": 8, "multiple": 128},
        # the weight gradient of one projection of the MLP workload's size
        {"name": "moe_wgrad 16384x4096x14336 2of8", "op": "moe_wgrad", "tokens": 16384,
         "k": 4096, "n": 14336, "experts": 8, "topk": 2, "multiple": 128},
        # one token between the two linears of the MLP workload
        {"name": "swiglu 1x14336", "op": "swiglu", "rows": 1, "cols": 14336, "dtype": "bf16",
         "out": "rows", "save": False},
        # the MLP workload's 16384 tokens: the next linear's E4M3 operand and
        # the 8-bit checkpoint
        {"name": "swiglu fp8 16384x14336", "op": "swiglu", "rows": 16384, "cols": 14336,
         "dtype": "bf16", "out": "e4m3", "save": True},
        # their gradient from the checkpoint, with the activation again
        {"name": "swiglu_bwd 16384x14336", "op": "swiglu_bwd", "rows": 16384, "cols": 14336,
         "dtype": "bf16", "out": "rows", "save": True},
        # fp32 rows of odd width, a ragged number of them
        {"name": "swiglu_bwd f32 3001x1001", "op": "swiglu_bwd", "rows": 3001, "cols": 1001,
         "dtype": "f32", "out": "rows", "save": True},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm: from 128 up, half
    of them multiples of 80 and half odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 128:
        v = v - v % 80 if rng.random() < 0.5 else v | 1
    return max(lo, min(hi, v))


def _blocks(rng, lo, hi):
    """A multiple of 128 of [lo, hi], spread over the logarithm."""
    return BLOCK * round(math.exp(rng.uniform(math.log(lo / BLOCK), math.log(hi / BLOCK))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "moe_fprop", "moe_fprop", "moe_dgrad", "moe_wgrad",
                     "swiglu", "swiglu_bwd"])
    if op.startswith("route"):
        experts = _log(rng, 2, 512)
        topk = rng.randint(1, min(16, experts))
        return {"op": op, "tokens": _log(rng, 1, (16384 * 256) // max(256, experts)),
                "experts": experts, "topk": topk, "dtype": rng.choice(["bf16", "f32"]),
                "renormalize": rng.random() < 0.5, "padding": rng.choice([0.0, 0.2]),
                "closed": rng.choice([0.0, 0.0, 0.5])}
    if op.startswith("moe"):
        # the widest weights that 64-bit products stay quick for
        experts = _log(rng, 2, 127)
        topk = rng.randint(1, min(8, experts))
        k, n = _blocks(rng, 128, 8192), _blocks(rng, 128, 8192)
        while experts * k * n > 2 ** 29:
            k, n = _blocks(rng, 128, 8192), _blocks(rng, 128, 8192)
        most = min(16384, TOP_FLOPS // (8 * k * n * topk), 2 ** 27 // (max(k, n) * topk))
        return {"op": op, "tokens": _log(rng, 1, max(1, most)), "k": k, "n": n,
                "experts": experts, "topk": topk,
                "multiple": 128 if op == "moe_wgrad" else rng.choice([1, 16, 128])}
    cols = _log(rng, 64, 16384)
    return {"op": op, "rows": _log(rng, 1, min(16384, (16384 * 14336) // cols)), "cols": cols,
            "dtype": rng.choice(["bf16", "bf16", "f32"]),
            "out": "rows" if op == "swiglu_bwd" else rng.choice(["rows", "e4m3"]),
            "save": rng.random() < 0.7}


# ------------------------------------------------------------------- work ---

def work(case):
    op = case["op"]
    if op.startswith("route"):
        t, e, k = case["tokens"], case["experts"], case["topk"]
        b = 2 if case["dtype"] == "bf16" else 4
        if op == "route":
            return {"bytes": t * e * b + 8 * t * k + 4 * e + 12, "flops": 4 * t * e}
        return {"bytes": 2 * t * e * b + 8 * t * k + 4 * e + 12, "flops": 10 * t * e}
    if op.startswith("moe"):
        rows, k, n, e = case["tokens"] * case["topk"], case["k"], case["n"], case["experts"]
        # experts that rows chosen evenly reach
        hit = e * (1 - (1 - case["topk"] / e) ** case["tokens"])
        flops = 2 * rows * k * n
        if op == "moe_wgrad":
            return {"bytes": int(rows * (k + n) * (1 + 4 / BLOCK) + 2 * e * k * n),
                    "flops": flops}
        a, d = (k, n) if op == "moe_fprop" else (n, k)
        return {"bytes": int(rows * (a * (1 + 4 / BLOCK) + 2 * d) + hit * k * n), "flops": flops}
    r, c = case["rows"], case["cols"]
    b = 2 if case["dtype"] == "bf16" else 4
    tiles = -(-c // BLOCK)
    saved = r * (2 * c + 8 * tiles)
    if op == "swiglu":
        y = r * (c + 4 * tiles) if case["out"] == "e4m3" else r * c * b
        return {"bytes": 2 * r * c * b + y + (saved if case["save"] else 0), "flops": 8 * r * c}
    h = saved if case["save"] else 2 * r * c * b
    return {"bytes": h + r * c * b + 3 * r * c * b, "flops": 16 * r * c}


# ---------------------------------------------------------------- prepare ---

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _scales(amax):
    """scale and scale_inv of tiles from their largest magnitudes."""
    a = amax.clamp(min=1e-12)
    return a / E4M3_MAX, E4M3_MAX / a


def _e4m3(v):
    """Saturating round to nearest even (the conversion itself does not saturate)."""
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _tiles(x):
    """x [rows, cols] in 32 bits as tiles of 128 columns, zeros behind the last."""
    r, c = x.shape
    n = -(-c // BLOCK)
    return torch.nn.functional.pad(x, (0, n * BLOCK - c)).view(r, n, BLOCK)


def _quantize(x):
    """E4M3 of x [rows, cols] under a scale for each 1x128 tile, and the scales."""
    t = _tiles(x)
    scale, inv = _scales(t.abs().amax(2))
    return _e4m3((t * inv[..., None]).view(x.shape[0], -1)[:, :x.shape[1]]).contiguous(), scale


def _dequantize(q, scale):
    """The 32-bit values that the bytes q [rows, cols] under 1x128 scales stand for."""
    return (_tiles(q.float()) * scale[..., None]).view(q.shape[0], -1)[:, :q.shape[1]]


def _quantize_halves(h):
    """The two halves of h [rows, 2 cols], each with tiles of its own."""
    c = h.shape[1] // 2
    (gq, gs), (uq, us) = _quantize(h[:, :c].float()), _quantize(h[:, c:].float())
    return torch.cat([gq.view(torch.uint8), uq.view(torch.uint8)], 1).view(
        torch.float8_e4m3fn), torch.cat([gs, us], 1)


def _segments(case, g):
    """Rows offsets[e] to offsets[e + 1] - 1 are expert e's, counts[e] of them
    with a token, for tokens that choose their top-k of skewed logits."""
    t, e = case["tokens"], case["experts"]
    logits = _normal(g, t, e) + 0.3 * _normal(g, e)
    ids = torch.topk(logits, case["topk"], dim=1).indices
    counts = torch.bincount(ids.reshape(-1), minlength=e)
    m = case["multiple"]
    padded = (counts + m - 1) // m * m
    return torch.cat([padded.new_zeros(1), padded.cumsum(0)]), counts


def _capacity(case):
    """Rows that every routing of the case's sizes fits, in whole blocks."""
    n = case["tokens"] * case["topk"]
    rows = n + min(n, case["experts"]) * (case["multiple"] - 1)
    return -(-rows // BLOCK) * BLOCK


def _rows(case, g, cols, offsets, counts):
    """Rows of tokens, zero in the padding: normal values, a few channels larger."""
    cap = _capacity(case)
    at = torch.arange(cap, device="cuda")
    expert = torch.searchsorted(offsets[1:], at, right=True).clamp(max=case["experts"] - 1)
    live = (at - offsets[expert] < counts[expert]) & (at < offsets[-1])
    gain = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 10.0, 1.0)
    return _normal(g, cap, cols) * gain * live[:, None]


def _weights(case, g):
    """E4M3 weights [experts, n, k] with 128x128 scales [experts, n/128, k/128]."""
    e, n, k = case["experts"], case["n"], case["k"]
    q = torch.empty(e, n, k, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(e, n // BLOCK, k // BLOCK, device="cuda")
    for i in range(e):
        w = (_normal(g, n, k) * k ** -0.5).view(n // BLOCK, BLOCK, k // BLOCK, BLOCK)
        s[i], inv = _scales(w.abs().amax((1, 3)))
        q[i] = _e4m3((w * inv[:, None, :, None]).view(n, k))
    return q, s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    op, s = case["op"], dict(case)
    if op.startswith("route"):
        t, e = case["tokens"], case["experts"]
        logits = 1.5 * _normal(g, t, e) + 0.5 * _normal(g, e)
        if case["closed"]:
            shut = torch.rand(t, e, generator=g, device="cuda") < case["closed"]
            logits = torch.where(shut, torch.full_like(logits, -math.inf), logits)
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["mask"] = torch.rand(t, generator=g, device="cuda") >= case["padding"]
        if op == "route_bwd":
            got = _plain_route(s)
            s["ids"], s["counts"], s["live"] = got["ids"], got["counts"], got["live"]
            s["dweights"] = _normal(g, t, case["topk"]) / t
            s["dlosses"] = torch.tensor([1e-2, 1e-3], device="cuda")
        return s
    if op.startswith("moe"):
        offsets, counts = _segments(case, g)
        s["offsets"] = offsets.int()
        s["longest"] = int((offsets[1:] - offsets[:-1]).max())
        if op == "moe_wgrad":
            for name, cols in (("g", case["n"]), ("x", case["k"])):
                rows = _rows(case, g, cols, offsets, counts)
                q, scale = _quantize(rows.t().contiguous())
                s[name + "qt"], s[name + "_scale_t"] = q, scale.t().contiguous()
            return s
        wq, s["w_scale"] = _weights(case, g)
        if op == "moe_fprop":
            s["wq"] = wq
            s["xq"], s["x_scale"] = _quantize(_rows(case, g, case["k"], offsets, counts))
        else:  # the transpose of all experts' weights stacked, [k, experts * n]
            wide = wq.view(torch.uint8).view(-1, case["k"])
            s["wqt"] = wide.t().contiguous().view(torch.float8_e4m3fn)
            s["gq"], s["g_scale"] = _quantize(1e-3 * _rows(case, g, case["n"], offsets, counts))
        return s
    r, c, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    # pre-activations: a few channels far larger than the rest
    gain = torch.where(torch.rand(2 * c, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    s["h"] = (_normal(g, r, 2 * c) * gain).to(dt)
    if op == "swiglu_bwd":
        s["dy"] = (1e-3 * _normal(g, r, c)).to(dt)
        if case["save"]:
            s["hq"], s["h_scale"] = _quantize_halves(s.pop("h"))
    return s


# -------------------------------------------------------------------- run ---

def _buffers(s, make):
    """Outputs and workspaces that a user's program allocates once and keeps."""
    if "buffers" not in s:
        s["buffers"] = make()
    return s["buffers"]


def _empty(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _run_own(s):
    import scaled_linear_layers_gb300 as fp8
    op, f32, i32 = s["op"], torch.float32, torch.int32
    if op == "route":
        t, e, k = s["tokens"], s["experts"], s["topk"]
        ids, weights, counts, live, losses, ws = _buffers(s, lambda: (
            _empty(i32, t, k), _empty(f32, t, k), _empty(i32, e), _empty(i32, 1), _empty(f32, 2),
            _empty(torch.uint8, fp8.fp8_moe_route_workspace_bytes(t, e))))
        fp8.fp8_moe_route(s["logits"], ids, weights, counts, live, losses, ws, mask=s["mask"],
                          renormalize=s["renormalize"])
        return {"ids": ids, "weights": weights, "counts": counts, "live": live, "losses": losses}
    if op == "route_bwd":
        dlogits = _buffers(s, lambda: torch.empty_like(s["logits"]))
        fp8.fp8_moe_route_backward(s["logits"], s["ids"], s["counts"], s["live"], dlogits,
                                   dweights=s["dweights"], dlosses=s["dlosses"],
                                   renormalize=s["renormalize"])
        return dlogits
    if op == "moe_fprop":  # rows behind the last segment stay as they were
        y = _buffers(s, lambda: torch.zeros(_capacity(s), s["n"], dtype=torch.bfloat16,
                                            device="cuda"))
        fp8.fp8_moe_linear_fprop(s["xq"], s["x_scale"], s["wq"], s["w_scale"], s["offsets"], y)
        return y
    if op == "moe_dgrad":
        dx = _buffers(s, lambda: torch.zeros(_capacity(s), s["k"], dtype=torch.bfloat16,
                                             device="cuda"))
        fp8.fp8_moe_linear_dgrad(s["gq"], s["g_scale"], s["wqt"], s["w_scale"], s["offsets"], dx)
        return dx
    if op == "moe_wgrad":
        dw = _buffers(s, lambda: _empty(torch.bfloat16, s["experts"], s["n"], s["k"]))
        fp8.fp8_moe_linear_wgrad(s["gqt"], s["g_scale_t"], s["xqt"], s["x_scale_t"], s["offsets"],
                                 dw)
        return dw
    r, c, e4m3 = s["rows"], s["cols"], torch.float8_e4m3fn
    tiles = -(-c // BLOCK)
    if op == "swiglu":
        quant, save = s["out"] == "e4m3", s["save"]
        got = _buffers(s, lambda: {
            "y": None if quant else _empty(s["h"].dtype, r, c),
            "yq": _empty(e4m3, r, c) if quant else None,
            "y_scale": _empty(f32, r, tiles) if quant else None,
            "hq": _empty(e4m3, r, 2 * c) if save else None,
            "h_scale": _empty(f32, r, 2 * tiles) if save else None})
        fp8.fp8_swiglu(s["h"], **got)
        return {k: v for k, v in got.items() if v is not None}
    dh, y = _buffers(s, lambda: (_empty(s["dy"].dtype, r, 2 * c), torch.empty_like(s["dy"])))
    if s["save"]:
        fp8.fp8_swiglu_backward(s["dy"], s["hq"], dh, h_scale=s["h_scale"], y=y)
    else:
        fp8.fp8_swiglu_backward(s["dy"], s["h"], dh, y=y)
    return {"dh": dh, "y": y}


def _plain_route(s):
    x, k, e = s["logits"].float(), s["topk"], s["experts"]
    order = torch.argsort(x, dim=1, descending=True, stable=True)[:, :k]
    kept = (torch.gather(x, 1, order) != -math.inf) & s["mask"][:, None]
    on = kept[:, 0]  # tokens with an expert
    top = torch.where(on[:, None], x, torch.zeros_like(x))
    peak = top.amax(1, keepdim=True)
    ex = torch.exp(top - peak)
    total = ex.sum(1, keepdim=True)
    p = torch.where(on[:, None], ex / total, torch.zeros_like(ex))
    w = torch.where(kept, torch.gather(p, 1, order), torch.zeros((), device=x.device))
    if s["renormalize"]:
        w = torch.where(kept, w / w.sum(1, keepdim=True), torch.zeros_like(w))
    ids = torch.where(kept, order, torch.full_like(order, -1))
    counts = torch.zeros(e + 1, dtype=torch.long, device=x.device)
    counts.scatter_add_(0, torch.where(kept, order, torch.full_like(order, e)).reshape(-1),
                        torch.ones_like(order).reshape(-1))
    live = on.sum()
    n = live.double().clamp(min=1)
    lse = torch.where(on, peak[:, 0] + torch.log(total[:, 0]), torch.zeros_like(peak[:, 0]))
    balance = (counts[:e].double() * p.sum(0, dtype=torch.float64)).sum() * e / (n * n * k)
    z = lse.double().square().sum() / n
    return {"ids": ids.int(), "weights": w, "counts": counts[:e].int(),
            "live": live.int().reshape(1), "losses": torch.stack([balance, z]).float()}


def _padded(s):
    """Row numbers [experts, longest] of the experts' segments, and which exist."""
    at = s["offsets"][:-1, None].long() + torch.arange(s["longest"], device="cuda")
    return at, at < s["offsets"][1:, None]


def _by_expert(s, rows):
    """rows of each expert [experts, longest, cols], zero behind its last."""
    at, there = _padded(s)
    return rows[at.clamp(max=rows.shape[0] - 1)] * there[..., None]


def _back(s, y):
    """The experts' rows in their places, zero behind the last segment."""
    at, there = _padded(s)
    cap = _capacity(s)
    out = torch.zeros(cap + 1, y.shape[2], dtype=torch.bfloat16, device="cuda")
    out[torch.where(there, at, torch.full_like(at, cap))] = y.to(torch.bfloat16)
    return out[:cap]


def _weight_values(q, scale, n, k):
    """[experts, n, k] in 32 bits."""
    e = scale.shape[0]
    w = q.float().view(e, n // BLOCK, BLOCK, k // BLOCK, BLOCK)
    return (w * scale[:, :, None, :, None]).view(e, n, k)


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["op"]
    if op == "route":
        return _plain_route(s)
    if op == "route_bwd":
        x, k, e = s["logits"].float(), s["topk"], s["experts"]
        kept = s["ids"] >= 0
        on = kept[:, :1]
        x = torch.where(on, x, torch.zeros_like(x))
        peak = x.amax(1, keepdim=True)
        ex = torch.exp(x - peak)
        total = ex.sum(1, keepdim=True)
        p, lse = ex / total, peak + torch.log(total)
        at = s["ids"].clamp(min=0).long()
        w = torch.where(kept, torch.gather(p, 1, at), torch.zeros((), device=x.device))
        if s["renormalize"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
        dw = torch.where(kept, s["dweights"], torch.zeros_like(s["dweights"]))
        n = s["live"].float().clamp(min=1)
        dp = (s["dlosses"][0] * e / (n * n * k) * s["counts"].float()).expand_as(p)
        d = p * (dp - (p * dp).sum(1, keepdim=True)) + 2 * s["dlosses"][1] / n * lse * p
        if s["renormalize"]:
            d = d.scatter_add(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
        else:
            d = d - p * (w * dw).sum(1, keepdim=True)
            d = d.scatter_add(1, at, w * dw)
        return torch.where(on, d, torch.zeros_like(d)).to(s["logits"].dtype)
    if op == "moe_fprop":
        w = _weight_values(s["wq"], s["w_scale"], s["n"], s["k"])
        x = _by_expert(s, _dequantize(s["xq"], s["x_scale"]))
        return _back(s, torch.bmm(x, w.transpose(1, 2)))
    if op == "moe_dgrad":
        wq = s["wqt"].view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn)
        w = _weight_values(wq, s["w_scale"], s["n"], s["k"])
        return _back(s, torch.bmm(_by_expert(s, _dequantize(s["gq"], s["g_scale"])), w))
    if op == "moe_wgrad":
        g = _by_expert(s, _dequantize(s["gqt"], s["g_scale_t"].t()).t())
        x = _by_expert(s, _dequantize(s["xqt"], s["x_scale_t"].t()).t())
        return torch.bmm(g.transpose(1, 2), x).to(torch.bfloat16)
    c = s["cols"]
    if op == "swiglu":
        gate, up = s["h"][:, :c].float(), s["h"][:, c:].float()
        y = gate / (1 + torch.exp(-gate)) * up
        got = {}
        if s["out"] == "rows":
            got["y"] = y.to(s["h"].dtype)
        else:
            got["yq"], got["y_scale"] = _quantize(y)
        if s["save"]:
            got["hq"], got["h_scale"] = _quantize_halves(s["h"])
        return got
    if s["save"]:
        tiles = -(-c // BLOCK)
        gate = _dequantize(s["hq"][:, :c], s["h_scale"][:, :tiles])
        up = _dequantize(s["hq"][:, c:], s["h_scale"][:, tiles:])
    else:
        gate, up = s["h"][:, :c].float(), s["h"][:, c:].float()
    dy = s["dy"].float()
    sig = 1 / (1 + torch.exp(-gate))
    act = gate * sig
    dgate = dy * up * (sig + act * (1 - sig))
    return {"dh": torch.cat([dgate, dy * act], 1).to(s["dy"].dtype),
            "y": (act * up).to(s["dy"].dtype)}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    s, op, f = prepare(case, seed), case["op"], torch.float64
    if op.startswith("route"):
        # by the library's softmax and, for the gradient, by autograd
        x = s["logits"].to(f)
        on = (s["mask"] & (x != -math.inf).any(1)) if op == "route" else s["ids"][:, 0] >= 0
        rows = torch.nonzero(on)[:, 0]
        n, e, k = max(1, rows.numel()), case["experts"], case["topk"]
        ids = _plain_route(s)["ids"] if op == "route" else s["ids"]
        at = ids[rows].clamp(min=0).long()
        kept = ids[rows] >= 0
        x = x[rows].requires_grad_(op == "route_bwd")
        p = torch.softmax(x, 1)
        w = p.gather(1, at) * kept
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        counts = torch.bincount(at[kept], minlength=e).to(f)
        balance = e * torch.dot(counts / (n * k), p.sum(0) / n)
        z = torch.logsumexp(x, 1).square().sum() / n
        if op == "route":
            weights = torch.zeros(case["tokens"], k, dtype=f, device="cuda")
            weights[rows] = w
            return {"ids": None, "weights": weights, "counts": None, "live": None,
                    "losses": torch.stack([balance, z])}
        loss = (w * s["dweights"][rows].to(f)).sum() + s["dlosses"][0].to(f) * balance
        loss = loss + s["dlosses"][1].to(f) * z
        d = torch.zeros(case["tokens"], e, dtype=f, device="cuda")
        d[rows], = torch.autograd.grad(loss, x)
        return d
    if op.startswith("moe"):
        n, k, cap = case["n"], case["k"], _capacity(case)
        at = s["offsets"].tolist()
        wide = lambda t, dim: t.to(f).repeat_interleave(BLOCK, dim)  # noqa: E731
        if op == "moe_wgrad":
            out = torch.zeros(case["experts"], n, k, dtype=f, device="cuda")
        else:
            out = torch.zeros(cap, n if op == "moe_fprop" else k, dtype=f, device="cuda")
        for e, (lo, hi) in enumerate(zip(at, at[1:])):  # expert by expert
            if hi == lo:
                continue
            if op == "moe_wgrad":
                b = slice(lo // BLOCK, hi // BLOCK)
                gt = s["gqt"][:, lo:hi].to(f) * wide(s["g_scale_t"][b], 0).t()
                xt = s["xqt"][:, lo:hi].to(f) * wide(s["x_scale_t"][b], 0).t()
                out[e] = gt @ xt.t()
                continue
            ws = wide(wide(s["w_scale"][e], 0), 1)
            if op == "moe_fprop":
                x = s["xq"][lo:hi].to(f) * wide(s["x_scale"][lo:hi], 1)
                out[lo:hi] = x @ (s["wq"][e].to(f) * ws).t()
            else:
                x = s["gq"][lo:hi].to(f) * wide(s["g_scale"][lo:hi], 1)
                out[lo:hi] = x @ (s["wqt"][:, e * n:(e + 1) * n].to(f) * ws.t()).t()
        return out
    c = case["cols"]
    tiles = -(-c // BLOCK)
    sizes = torch.full((tiles,), BLOCK, device="cuda")
    sizes[-1] = c - BLOCK * (tiles - 1)

    def largest(v):
        return torch.stack([t.abs().amax(1) for t in v.split(BLOCK, 1)], 1).clamp(min=1e-12)

    def spread(scale):  # a value for each column
        return torch.repeat_interleave(scale, sizes, dim=1)

    if op == "swiglu":
        gate, up = s["h"][:, :c].to(f), s["h"][:, c:].to(f)
        y = torch.nn.functional.silu(gate) * up
        got = {}
        if case["out"] == "rows":
            got["y"] = y
        else:
            a = largest(y)
            got["yq"], got["y_scale"] = y * spread(E4M3_MAX / a), a / E4M3_MAX
        if case["save"]:
            a, b = largest(gate), largest(up)
            got["hq"] = torch.cat([gate * spread(E4M3_MAX / a), up * spread(E4M3_MAX / b)], 1)
            got["h_scale"] = torch.cat([a, b], 1) / E4M3_MAX
        return got
    if case["save"]:
        scale = s["h_scale"].to(f)
        gate = s["hq"][:, :c].to(f) * spread(scale[:, :tiles])
        up = s["hq"][:, c:].to(f) * spread(scale[:, tiles:])
    else:
        gate, up = s["h"][:, :c].to(f), s["h"][:, c:].to(f)
    # silu and its slope by the hyperbolic tangent of half the argument
    half = torch.tanh(gate / 2)
    act = gate * (1 + half) / 2
    slope = (1 + half) / 2 + gate * (1 - half * half) / 4
    dy = s["dy"].to(f)
    return {"dh": torch.cat([dy * up * slope, dy * act], 1), "y": act * up}
