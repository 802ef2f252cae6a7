"""The router against its definition in 64 bits.  Ids and counts exactly;
probabilities within the roundings of the fp32 formula: l - peak is off by
2^-24 of its size, exp by two units, the sum of E terms by E + 1 halves, so
(E + |l - peak| + 16) 2^-24 relative covers a probability and a weight; sums
over T tokens add (T + 16) 2^-24 relative, as all their terms are positive.
The gradient's terms carry the same relative errors, so they are bounded by
(E + |l| + 32) 2^-23 of the sum of their magnitudes, plus half a unit of the
output's type."""
import math

import pytest
import torch

import scaled_linear_layers_gb300 as fp8

pytestmark = pytest.mark.gpu
BF, F, D = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
HALF = {BF: 2.0 ** -8, F: U}


def logits_of(tokens, experts, seed, dtype=F, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(tokens, experts, generator=g, device="cuda")).to(dtype)


def route(logits, topk, mask=None, renormalize=True, losses=True, stream=None):
    t, e = logits.shape
    i32 = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")  # noqa: E731
    out = {"ids": i32(t, topk), "weights": torch.full((t, topk), 9.0, device="cuda"),
           "counts": i32(e), "live": i32(1),
           "losses": torch.full((2,), 9.0, device="cuda") if losses else None}
    ws = torch.empty(fp8.fp8_moe_route_workspace_bytes(t, e), dtype=torch.uint8, device="cuda")
    fp8.fp8_moe_route(logits, **out, workspace=ws, mask=mask, renormalize=renormalize, stream=stream)
    return out


def plain(logits, topk, mask=None, renormalize=True):
    """The definition in 64 bits on the host (finite and -inf logits)."""
    x = logits.to(D).cpu()
    t, e = x.shape
    on = torch.ones(t, dtype=torch.bool) if mask is None else mask.cpu().bool().clone()
    on &= (x > -math.inf).any(1)
    ids = torch.full((t, topk), -1)
    w = torch.zeros(t, topk, dtype=D)
    p = torch.zeros(t, e, dtype=D)
    lse = torch.zeros(t, dtype=D)
    p[on] = torch.softmax(x[on], 1)
    lse[on] = torch.logsumexp(x[on], 1)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :topk]
    kept = (x.gather(1, order) > -math.inf) & on[:, None]
    ids[kept] = order[kept]
    w[kept] = p.gather(1, order)[kept]
    if renormalize:
        w = torch.where(kept, w / w.sum(1, keepdim=True).clamp(min=1e-300), w)
    counts = torch.bincount(ids[kept], minlength=e)
    n = max(1, int(on.sum()))
    balance = e / (n * n * topk) * (counts.to(D) * p.sum(0)).sum()
    return {"ids": ids, "weights": w, "counts": counts, "live": int(on.sum()),
            "losses": torch.stack([balance, lse.square().sum() / n]), "p": p, "lse": lse, "on": on}


def check(got, want, logits):
    t, e = logits.shape
    assert torch.equal(got["ids"].cpu().long(), want["ids"])
    assert torch.equal(got["counts"].cpu().long(), want["counts"])
    assert got["live"].item() == want["live"]
    finite = logits.double().cpu()
    finite = torch.where(finite > -math.inf, finite, torch.zeros_like(finite))
    spread = (finite.amax(1) - finite.amin(1)).max().item() if t else 0.0
    rel = (e + spread + 16) * U
    off = (got["weights"].cpu().double() - want["weights"]).abs()
    assert (off <= 2 * rel * want["weights"] + 1e-38).all()
    if got["losses"] is not None:
        # lse is off by its own rounding and its sum's, relative to max(|lse|, 1)
        off = (got["losses"].cpu().double() - want["losses"]).abs()
        assert off[0] <= (rel + (t + 32) * U) * want["losses"][0]
        big = want["lse"].abs().max().item() if t else 0.0
        assert off[1] <= (t + 32) * U * want["losses"][1] + 2 * big * rel * max(1.0, big) + 1e-38


@pytest.mark.parametrize("tokens, experts, topk", [
    (0, 8, 2), (1, 1, 1), (1, 64, 8), (3, 5, 5), (8, 64, 8), (257, 8, 2), (100, 61, 6),
    (513, 33, 1), (70, 160, 7), (40, 256, 8), (65, 300, 16), (33, 512, 32), (19, 1000, 10),
    (5, 1024, 32), (4099, 16, 4)])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route(tokens, experts, topk, dtype, renormalize):
    x = logits_of(tokens, experts, seed=tokens + experts, dtype=dtype)
    check(route(x, topk, renormalize=renormalize), plain(x, topk, renormalize=renormalize), x)


@pytest.mark.parametrize("mask_type", [torch.bool, torch.uint8])
def test_mask_closed_experts_and_rows_of_nothing(mask_type):
    x = logits_of(300, 40, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x[torch.rand(x.shape, generator=g, device="cuda") < 0.9] = -math.inf  # fewer open than topk
    x[7] = -math.inf
    mask = torch.rand(300, generator=g, device="cuda") < 0.7
    for renormalize in (True, False):
        got = route(x, 6, mask.to(mask_type), renormalize)
        check(got, plain(x, 6, mask, renormalize), x)
    assert (got["ids"][7] == -1).all() and (got["weights"][7] == 0).all()
    none = route(x, 6, torch.zeros(300, dtype=mask_type, device="cuda"))
    assert none["live"].item() == 0 and (none["counts"] == 0).all() and (none["losses"] == 0).all()


def test_ties_go_to_the_lowest_id_and_zeros_are_equal():
    x = torch.zeros(3, 70, device="cuda")
    x[0, 1::2] = -0.0
    x[1, 40:] = 1.0
    x[2] = torch.finfo(F).min
    got = route(x, 4)["ids"].cpu()
    assert got.tolist() == [[0, 1, 2, 3], [40, 41, 42, 43], [0, 1, 2, 3]]


def test_garbage_in_masked_rows_reaches_nothing():
    x = logits_of(50, 24, seed=8)
    mask = torch.ones(50, dtype=torch.bool, device="cuda")
    mask[10:20] = False
    want = route(x, 3, mask)
    x[10:15], x[15:20] = math.nan, math.inf
    got = route(x, 3, mask)
    for name in want:
        assert torch.equal(got[name], want[name]), name


def test_nan_and_infinite_logits_stay_in_their_rows_and_show_in_the_losses():
    x = logits_of(20, 24, seed=9)
    clean = route(x, 3)
    x[4, 5], x[6, 7] = math.nan, math.inf
    got = route(x, 3)
    assert got["ids"][4, 0].item() == 5 and got["ids"][6, 0].item() == 7
    assert got["weights"][4].isnan().all() and got["weights"][6].isnan().any()
    assert got["losses"].isnan().all()
    others = torch.tensor([i for i in range(20) if i not in (4, 6)], device="cuda")
    assert torch.equal(got["ids"][others], clean["ids"][others])
    assert torch.equal(got["weights"][others], clean["weights"][others])
    assert ((got["ids"] >= 0) & (got["ids"] < 24)).all()


def test_large_logits_do_not_overflow():
    x = logits_of(64, 48, seed=10, scale=3e4)
    check(route(x, 5, renormalize=False), plain(x, 5, renormalize=False), x)


@pytest.mark.parametrize("dtype", [BF, F])
def test_strided_rows_another_stream_and_the_same_bits(dtype):
    wide = logits_of(777, 100, seed=11, dtype=dtype)
    x = wide[:, 3:64]
    want = route(x.contiguous(), 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = route(x, 6, stream=s)
    s.synchronize()
    again = route(x, 6)
    for name in want:
        assert torch.equal(got[name], want[name]) and torch.equal(again[name], want[name])
    same = route(x[:1].expand(9, -1), 6)  # one row for all tokens: a row stride of 0
    assert (same["ids"] == want["ids"][0]).all() and same["live"].item() == 9
    assert route(x, 6, losses=False)["counts"].equal(want["counts"])


def backward(x, topk, seed, mask=None, renormalize=True, dweights=True, dlosses=True):
    fwd = route(x, topk, mask, renormalize)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dw = torch.randn(fwd["weights"].shape, generator=g, device="cuda") if dweights else None
    dl = torch.tensor([0.7, -0.3], device="cuda") if dlosses else None
    d = torch.full(x.shape, 9.0, dtype=x.dtype, device="cuda")
    fp8.fp8_moe_route_backward(x, fwd["ids"], fwd["counts"], fwd["live"], d, dw, dl, renormalize)
    return d, dw, dl


def plain_backward(x, topk, mask, renormalize, dw, dl):
    """The formula in 64 bits, and the sum of its terms' magnitudes."""
    want = plain(x, topk, mask, renormalize)
    t, e = x.shape
    p, on = want["p"], want["on"][:, None]
    n = max(1, want["live"])
    dl = torch.zeros(2, dtype=D) if dl is None else dl.cpu().double()
    dw = torch.zeros(t, topk, dtype=D) if dw is None else dw.cpu().double()
    kept = want["ids"] >= 0
    dw = torch.where(kept, dw, torch.zeros_like(dw))
    at = want["ids"].clamp(min=0)
    c = (dl[0] * e / (n * n * topk) * want["counts"].to(D)).expand(t, e)
    z = (2 * dl[1] / n * want["lse"])[:, None]
    d = p * (c - (p * c).sum(1, keepdim=True)) + z * p
    mag = p * (c.abs() + (p * c.abs()).sum(1, keepdim=True)) + z.abs() * p
    w = want["weights"]
    dot, mdot = (w * dw).sum(1, keepdim=True), (w * dw.abs()).sum(1, keepdim=True)
    if renormalize:
        d = d.scatter_add(1, at, w * (dw - dot) * kept)
        mag = mag.scatter_add(1, at, w * (dw.abs() + mdot) * kept)
    else:
        d = (d - p * dot).scatter_add(1, at, w * dw)
        mag = (mag + p * mdot).scatter_add(1, at, w * dw.abs())
    return torch.where(on, d, torch.zeros_like(d)), mag


def check_backward(got, want, mag, x):
    size = x.double().cpu()
    size = torch.where(size.abs() < math.inf, size.abs(), torch.zeros_like(size))
    size = size.max().item() if x.numel() else 0.0
    tol = HALF[x.dtype] * want.abs() + (x.shape[1] + 2 * size + 32) * 2 * U * (1 + HALF[x.dtype]) * mag
    assert ((got.cpu().double() - want).abs() <= tol + 1e-38).all()


@pytest.mark.parametrize("tokens, experts, topk", [
    (0, 8, 2), (1, 1, 1), (1, 64, 8), (8, 64, 8), (257, 8, 2), (100, 61, 6), (70, 160, 7),
    (40, 256, 8), (33, 512, 32), (5, 1024, 32), (4099, 16, 4)])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("renormalize", [True, False])
def test_backward(tokens, experts, topk, dtype, renormalize):
    x = logits_of(tokens, experts, seed=tokens + experts + 1, dtype=dtype)
    got, dw, dl = backward(x, topk, 3, None, renormalize)
    want, mag = plain_backward(x, topk, None, renormalize, dw, dl)
    check_backward(got, want, mag, x)


@pytest.mark.parametrize("renormalize", [True, False])
def test_backward_of_masked_rows_closed_experts_and_single_gradients(renormalize):
    x = logits_of(300, 40, seed=12)
    g = torch.Generator(device="cuda").manual_seed(13)
    x[torch.rand(x.shape, generator=g, device="cuda") < 0.9] = -math.inf
    mask = torch.rand(300, generator=g, device="cuda") < 0.7
    for kw in (dict(), dict(dweights=False), dict(dlosses=False), dict(dweights=False, dlosses=False)):
        got, dw, dl = backward(x, 6, 4, mask, renormalize, **kw)
        want, mag = plain_backward(x, 6, mask, renormalize, dw, dl)
        check_backward(got, want, mag, x)
        assert (got[~mask] == 0).all() and (got[x == -math.inf] == 0).all()
    x[~mask] = math.nan  # garbage in padding
    assert torch.equal(backward(x, 6, 4, mask, renormalize, dweights=False, dlosses=False)[0], got)


def test_backward_against_differences():
    """(f(x + h) - f(x - h)) / 2h of the 64-bit forward; its own error is h^2/6 of
    the third derivative (at most 6 of these sums' size) and 2^-52/h of f."""
    x = logits_of(6, 12, seed=14)
    h = 1e-4
    for renormalize in (True, False):
        got, dw, dl = backward(x, 3, 5, None, renormalize)
        base = plain(x, 3, None, renormalize)
        n = base["live"]

        def f(v):
            p = torch.softmax(v, 1)
            w = p.gather(1, base["ids"])
            w = w / w.sum(1, keepdim=True) if renormalize else w
            balance = 12 / (n * n * 3) * (base["counts"].to(D) * p.sum(0)).sum()
            z = torch.logsumexp(v, 1).square().sum() / n
            return (w * dw.cpu().double()).sum() + dl[0].item() * balance + dl[1].item() * z

        v = x.cpu().double()
        for t in range(6):
            for e in range(12):
                step = torch.zeros_like(v)
                step[t, e] = h
                want = (f(v + step) - f(v - step)) / (2 * h)
                assert abs(got[t, e].item() - want.item()) < 1e-6 * (1 + dw.abs().sum().item())


def test_backward_over_the_logits_and_from_a_graph():
    x = logits_of(600, 64, seed=15)
    want, dw, dl = backward(x, 8, 6)
    fwd = route(x, 8)
    own = x.clone()
    fp8.fp8_moe_route_backward(own, fwd["ids"], fwd["counts"], fwd["live"], own, dw, dl)
    assert torch.equal(own, want)
    # forward and backward captured, replayed on new logits
    out = {k: torch.empty_like(v) for k, v in fwd.items()}
    d, held = torch.empty_like(x), x.clone()
    ws = torch.empty(fp8.fp8_moe_route_workspace_bytes(600, 64), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.fp8_moe_route(held, **out, workspace=ws)
        fp8.fp8_moe_route_backward(held, out["ids"], out["counts"], out["live"], d, dw, dl)
    new = logits_of(600, 64, seed=16)
    held.copy_(new)
    graph.replay()
    graph.replay()
    eager = route(new, 8)
    for name in eager:
        assert torch.equal(out[name], eager[name]), name
    assert torch.equal(d, backward(new, 8, 6)[0])


def test_ids_out_of_range_are_left_out():
    x = logits_of(4, 8, seed=17)
    fwd = route(x, 2)
    dw = torch.ones(4, 2, device="cuda")
    ids = fwd["ids"].clone()
    ids[:, 1] = 8 + 1000000
    d = torch.empty_like(x)
    fp8.fp8_moe_route_backward(x, ids, fwd["counts"], fwd["live"], d, dw)
    assert d.isfinite().all()


def test_a_launch_that_fails_is_reported():
    x = logits_of(16, 8, seed=18)
    from scaled_linear_layers_gb300 import _LIB
    for n in (1, 2):
        # the forward has two launches: the first, or both, do not happen
        _LIB.fp8_inject_launch_failures(n)
        with pytest.raises(fp8.Fp8Error):
            route(x, 2)
        _LIB.fp8_inject_launch_failures(0)
    check(route(x, 2), plain(x, 2), x)


@pytest.mark.parametrize("tokens", [20, 40, 700])
def test_a_squared_log_sum_past_fp32_is_infinite(tokens):
    """(3e19)^2 is past fp32's 3.4e38: the loss is the infinity that rounding
    gives, in one block and over many, and the balance stays finite."""
    x = logits_of(tokens, 24, seed=30)
    x[tokens // 2] = 3e19
    got = route(x, 3)
    assert got["losses"][1].item() == math.inf and got["losses"][0].isfinite()


@pytest.mark.parametrize("tokens, experts, topk", [(3000, 96, 6), (5000, 300, 8), (64, 64, 8), (32, 64, 8)])
def test_replayed_with_new_logits_beside_other_streams(tokens, experts, topk):
    """One captured call (a launch, or two over many blocks) replayed with other
    logits and masks, while the same calls run on two more streams."""
    inputs = [(logits_of(tokens, experts, seed=40 + i),
               torch.rand(tokens, device="cuda") < (0.9, 0.1, 0.0)[i]) for i in range(3)]
    want = [route(x, topk, mask=m) for x, m in inputs]
    x, m = inputs[0][0].clone(), inputs[0][1].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = route(x, topk, mask=m)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, w in enumerate(want):
        x.copy_(inputs[i][0])
        m.copy_(inputs[i][1])
        torch.cuda.synchronize()
        others = []
        for s in streams:
            with torch.cuda.stream(s):
                others.append([route(*inputs[j][:1], topk, mask=inputs[j][1]) for j in range(3)])
        graph.replay()
        torch.cuda.synchronize()
        for name, value in w.items():
            assert torch.equal(held[name], value), name
            for got in others:
                assert torch.equal(got[i][name], value), name


def test_nan_rows_have_nan_gradients_and_no_other():
    """A NaN or +inf logit makes its token's gradient NaN, whichever lane and
    register holds it; a closed logit beside finite ones gets zero."""
    tokens, experts, topk = 200, 260, 4
    x = logits_of(tokens, experts, seed=50)
    bad = torch.arange(0, tokens, 7, device="cuda")
    x[bad, (bad * 13) % experts] = math.nan
    x[3, 5], x[4, 9] = math.inf, -math.inf
    clean = torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=-math.inf)
    ids = torch.argsort(clean, 1, descending=True)[:, :topk].int().contiguous()
    counts = torch.bincount(ids.reshape(-1), minlength=experts).int()
    live = torch.tensor([tokens], dtype=torch.int32, device="cuda")
    dw = torch.randn(tokens, topk, device="cuda")
    dl = torch.tensor([0.5, 0.25], device="cuda")
    d, ok = torch.empty_like(x), torch.empty_like(x)
    fp8.fp8_moe_route_backward(x, ids, counts, live, d, dw, dl)
    fp8.fp8_moe_route_backward(clean, ids, counts, live, ok, dw, dl)
    rows = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    rows[bad], rows[3] = True, True
    assert d[rows].isnan().all() and torch.equal(d[~rows], ok[~rows])
    assert d[4, 9] == 0 and ok.isfinite().all()
