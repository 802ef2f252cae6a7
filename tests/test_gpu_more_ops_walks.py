"""The gated activation and the router where a team or a warp takes several rows
one after the other: the next row's loads are held ahead, addresses move by a
step, and the last pass is ragged.  The grids hold at most 4 blocks of 16 teams an
SM (9728 teams), and 2 blocks of 16 warps (4864); every case here has more work
than that, and no multiple of it.  Bounds as in the tests of single rows."""
import pytest
import torch

import scaled_linear_layers_gb300 as fp8
import test_gpu_moe_route as router
import test_gpu_swiglu as gated

pytestmark = pytest.mark.gpu
BF, F, D = torch.bfloat16, torch.float32, torch.float64
empty, rnd = gated.empty, gated.rnd

# whole vectors of two tiles; two tiles and one element at a time; one ragged tile;
# more tiles than teams, so that a team goes on to the tiles a width further
SIZES = [(20001, 256), (20001, 250), (40009, 77), (3, 1400008), (2, 1400001)]


@pytest.mark.parametrize("rows, cols", SIZES)
@pytest.mark.parametrize("dtype", [BF, F])
def test_gated_forward(rows, cols, dtype):
    h = rnd(rows, 2 * cols, seed=rows, dtype=dtype)
    out = gated.forward(h)
    g, u, _, y = gated.plain(h)
    err = gated.rel_error(g, dtype) * y.abs() + 1e-37
    assert ((out["y"].to(D) - y).abs() <= err + gated.HALF[dtype] * y.abs() * (1 + 2.0 ** -8)).all()
    gated.check_scaled(out["yq"], out["y_scale"], y, err)
    n, zero = gated.tiles_of(cols), torch.zeros_like(y)
    gated.check_scaled(out["hq"][:, :cols], out["h_scale"][:, :n], g, zero, exact=True)
    gated.check_scaled(out["hq"][:, cols:], out["h_scale"][:, n:], u, zero, exact=True)
    for what in (("y",), ("yq",), ("hq",)):
        for name, t in gated.forward(h, what).items():
            assert torch.equal(t, out[name]), name


@pytest.mark.parametrize("rows, cols", SIZES)
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("saved", [True, False])
def test_gated_backward(rows, cols, dtype, saved):
    h = rnd(rows, 2 * cols, seed=rows + 1, dtype=dtype)
    dy = rnd(rows, cols, seed=5, dtype=dtype, scale=1e-3)
    dh, y = empty(dtype, rows, 2 * cols), empty(dtype, rows, cols)
    if saved:
        keep = gated.forward(h, ("hq",))
        fp8.fp8_swiglu_backward(dy, keep["hq"], dh, keep["h_scale"], y)
        gated.check_backward(dh, y, dy, gated.checkpoint_values(keep["hq"], keep["h_scale"], cols),
                             dtype)
        return
    fp8.fp8_swiglu_backward(dy, h, dh, y=y)
    gated.check_backward(dh, y, dy, h.to(D), dtype)
    own, again = h.clone(), torch.empty_like(y)
    fp8.fp8_swiglu_backward(dy, own, own, y=again)  # over its input
    assert torch.equal(own, dh) and torch.equal(again, y)


@pytest.mark.parametrize("rows, cols", SIZES[:3])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("live", [1, 9727, 9729, 13001])
def test_rows_that_end_inside_a_walk(rows, cols, dtype, live):
    h, dy = rnd(rows, 2 * cols, seed=6, dtype=dtype), rnd(rows, cols, seed=7, dtype=dtype)
    lv = torch.tensor([live], dtype=torch.int32, device="cuda")
    want = gated.forward(h)
    for name, t in gated.forward(h, live=lv, fill=3).items():
        assert torch.equal(t[:live], want[name][:live]) and (t[live:] == 3).all(), name
    for args in ((h, None), (want["hq"], want["h_scale"])):
        full = [empty(dtype, rows, 2 * cols), empty(dtype, rows, cols)]
        part = [torch.full_like(t, 3.0) for t in full]
        fp8.fp8_swiglu_backward(dy, args[0], full[0], args[1], full[1])
        fp8.fp8_swiglu_backward(dy, args[0], part[0], args[1], part[1], live=lv)
        for a, b in zip(full, part):
            assert torch.equal(b[:live], a[:live]) and (b[live:] == 3).all()


# 20 to 32 tokens: one block, two tokens to some or all of its warps
ROUTES = [(20, 64, 8), (32, 61, 6), (27, 256, 8), (31, 1024, 32), (10007, 16, 4), (10007, 61, 6),
          (10007, 128, 8), (10007, 256, 8), (15001, 250, 24), (5003, 512, 8), (6007, 1000, 10)]


@pytest.mark.parametrize("tokens, experts, topk", ROUTES)
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("renormalize", [True, False])
def test_router(tokens, experts, topk, dtype, renormalize):
    x = router.logits_of(tokens, experts, seed=tokens + experts, dtype=dtype)
    mask = torch.rand(tokens, device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(8)) < 0.8
    for m in (None, mask):
        got = router.route(x, topk, m, renormalize)
        router.check(got, router.plain(x, topk, m, renormalize), x)
    d, dw, dl = router.backward(x, topk, 9, mask, renormalize)
    want, mag = router.plain_backward(x, topk, mask, renormalize, dw, dl)
    router.check_backward(d, want, mag, x)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("experts, start, wide", [(61, 3, 100), (128, 0, 132), (128, 4, 300),
                                                  (256, 8, 264), (256, 2, 300), (512, 4, 1028),
                                                  (1000, 0, 1004)])
def test_router_of_rows_with_a_stride(dtype, experts, start, wide):
    """Rows on groups of four logits with others between them, and rows that are
    not: the bits of contiguous rows where the lanes share the experts alike."""
    x = router.logits_of(3001, wide, seed=10, dtype=dtype)[:, start:start + experts]
    own = x.contiguous()
    want, got = router.route(own, 6), router.route(x, 6)
    a, b = router.backward(own, 6, 11), router.backward(x, 6, 11)
    if start % 4 == 0 or experts % 4 != 0:
        for name in want:
            assert torch.equal(got[name], want[name]), name
        assert torch.equal(a[0], b[0])
    router.check(got, router.plain(own, 6), own)
    w, mag = router.plain_backward(own, 6, None, True, b[1], b[2])
    router.check_backward(b[0], w, mag, own)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("experts", [70, 300, 1024])
def test_ties_of_more_logits_than_are_dealt_out(dtype, experts):
    x = torch.zeros(5, experts, dtype=dtype, device="cuda")
    x[0, 1::2] = -0.0
    x[1, 40:] = 1.0
    x[2] = torch.finfo(dtype).min
    x[3, 5], x[3, 66] = 2.0, 2.0
    x[4, :3] = -torch.inf
    for topk in (4, 32):
        ids = router.route(x, topk)["ids"].tolist()
        # one value behind all others' bar: those above it first, then the lowest ids
        rest = [i for i in range(experts) if i not in (5, 66)]
        low = list(range(40, experts)) + list(range(40))
        assert ids[0] == list(range(topk)) and ids[2] == list(range(topk))
        assert ids[1] == low[:topk]
        assert ids[3] == ([5, 66] + rest)[:topk]
        assert ids[4] == list(range(3, topk + 3))


@pytest.mark.parametrize("experts", [24, 260])
def test_nan_and_infinite_bf16_logits(experts):
    """bf16 logits have numbers of their own in the top-k: NaN the largest, in its
    row alone; the gradient of such a row is NaN, whichever lane holds the logit."""
    tokens, topk = 210, 4
    x = router.logits_of(tokens, experts, seed=12, dtype=BF)
    clean = router.route(x, topk)
    bad = torch.arange(0, tokens, 7, device="cuda")
    at = (bad * 13) % experts
    x[bad, at] = torch.nan
    x[3, 5], x[4, 9] = torch.inf, -torch.inf
    got = router.route(x, topk)
    assert (got["ids"][bad, 0] == at).all() and got["ids"][3, 0] == 5
    assert got["weights"][bad].isnan().all() and got["weights"][3].isnan().any()
    assert got["losses"].isnan().all() and got["live"].item() == tokens
    same = torch.ones(tokens, dtype=torch.bool, device="cuda")
    same[bad], same[3], same[4] = False, False, False
    assert torch.equal(got["ids"][same], clean["ids"][same])
    assert torch.equal(got["weights"][same], clean["weights"][same])
    assert 9 not in got["ids"][4].tolist()
    dw = torch.randn(tokens, topk, device="cuda")
    dl = torch.tensor([0.5, 0.25], device="cuda")
    d = torch.empty_like(x)
    fp8.fp8_moe_route_backward(x, got["ids"], got["counts"], got["live"], d, dw, dl)
    rows = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    rows[bad], rows[3] = True, True
    assert d[rows].isnan().all() and d[~rows].isfinite().all() and d[4, 9] == 0
