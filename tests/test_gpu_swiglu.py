"""The gated activation and its gradient against the formula in 64 bits.

Rows: bf16 rows take the hardware's exponential and division, whose relative
errors are 2^-21 (1 + |x|/8) and 2^-22; with three products 2^-19 (1 + |x|/8)
covers y, and the same of the sum of its terms' magnitudes the gradient.  fp32
rows: exp within 2 units and 2^-24 |x| of its argument's rounding, a division
and three products, (16 + |x|) 2^-24.  Plus half a unit of the output's type.
Scales: those errors of y and two roundings; the checkpoint's are exact (its
maxima are inputs).  A cast is off by half a step of e4m3: 2^-4 of the value, or
2^-10 of the scale near zero, and a value that close to a border may take the
neighbour, which the same bound with y's error added covers."""
import math

import pytest
import torch

import scaled_linear_layers_gb300 as fp8

pytestmark = pytest.mark.gpu
BF, F, D = torch.bfloat16, torch.float32, torch.float64
HALF = {BF: 2.0 ** -8, F: 2.0 ** -24}
E4M3 = torch.float8_e4m3fn


def rnd(*shape, seed, dtype, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def rel_error(x, dtype):
    """Of s, y and the terms of the gradient, for gates x."""
    x = x.abs().clamp(max=200.0)
    return 2.0 ** -19 * (1 + x / 8) if dtype == BF else (16 + x) * 2.0 ** -24


def empty(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda")


def tiles_of(cols):
    return -(-cols // 128)


def forward(h, what=("y", "yq", "hq"), live=None, stream=None, fill=None):
    rows, c = h.shape[0], h.shape[1] // 2
    n = tiles_of(c)
    out = {}
    if "y" in what:
        out["y"] = empty(h.dtype, rows, c)
    if "yq" in what:
        out |= {"yq": empty(torch.uint8, rows, c), "y_scale": empty(F, rows, n)}
    if "hq" in what:
        out |= {"hq": empty(torch.uint8, rows, 2 * c), "h_scale": empty(F, rows, 2 * n)}
    if fill is not None:
        for t in out.values():
            t.fill_(fill)
    fp8.fp8_swiglu(h, **out, live=live, stream=stream)
    return out


def tile_max(x):
    return torch.stack([t.abs().amax(1) for t in x.split(128, 1)], 1) if x.shape[1] else x[:, :0]


def spread(scale, cols):
    return scale.repeat_interleave(128, 1)[:, :cols]


def plain(h):
    c = h.shape[1] // 2
    g, u = h[:, :c].to(D), h[:, c:].to(D)
    s = 1 / (1 + torch.exp(-g))
    return g, u, s, g * s * u


def check_scaled(q, scale, want, err, exact=False):
    """E4M3 bytes and their tiles' scales against 64-bit values off by `err`."""
    a = tile_max(want).clamp(min=1e-12)
    if want.numel():
        slack = torch.zeros_like(a) if exact else tile_max(err)
        assert ((scale.to(D) - a / 448).abs() <= (slack + a * 2.0 ** -23) / 448).all()
    got = q.view(E4M3).to(D) * spread(scale.to(D), want.shape[1])
    tol = 2.0 ** -4 * want.abs() + 2.0 ** -10 * spread(scale.to(D), want.shape[1]) * 1.01
    tol = tol * (1 + 2.0 ** -20) + 1.1 * err + spread(a, want.shape[1]) * 2.0 ** -22
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("rows, cols", [
    (0, 128), (1, 0), (1, 1), (1, 8), (3, 7), (5, 127), (4, 128), (9, 129), (7, 136), (33, 384),
    (2, 1001), (300, 250), (17, 2048), (1, 14336), (1000, 24), (129, 1032)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_forward(rows, cols, dtype):
    h = rnd(rows, 2 * cols, seed=rows + cols, dtype=dtype)
    out = forward(h)
    g, u, s, y = plain(h)
    err = rel_error(g, dtype) * y.abs() + 1e-37
    assert ((out["y"].to(D) - y).abs() <= err + HALF[dtype] * y.abs() * (1 + 2.0 ** -8)).all()
    check_scaled(out["yq"], out["y_scale"], y, err)
    n = tiles_of(cols)
    zero = torch.zeros_like(y)
    check_scaled(out["hq"][:, :cols], out["h_scale"][:, :n], g, zero, exact=True)
    check_scaled(out["hq"][:, cols:], out["h_scale"][:, n:], u, zero, exact=True)


@pytest.mark.parametrize("cols", [256, 384])
def test_the_checkpoint_is_the_block_recipe_of_the_halves(cols):
    """hq and h_scale are the bytes that fp8_quantize(BLOCK) makes of h."""
    h = rnd(64, 2 * cols, seed=3, dtype=BF)
    out = forward(h, ("hq",))
    q, s, si = empty(torch.uint8, 64, 2 * cols), empty(F, 64, cols // 64), empty(F, 64, cols // 64)
    fp8.fp8_quantize(h, fp8.BLOCK, s, si, q)
    assert torch.equal(out["hq"], q) and torch.equal(out["h_scale"], s)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("what", [("y",), ("yq",), ("hq",), ("y", "hq"), ("yq", "hq")])
def test_outputs_do_not_depend_on_each_other(dtype, what):
    for cols in (256, 133):
        h = rnd(40, 2 * cols, seed=4, dtype=dtype)
        full, some = forward(h), forward(h, what)
        for name, t in some.items():
            assert torch.equal(t, full[name]), name


def checkpoint_values(hq, h_scale, cols):
    n = tiles_of(cols)
    q = hq.view(E4M3).to(D)
    return torch.cat([q[:, :cols] * spread(h_scale[:, :n].to(D), cols),
                      q[:, cols:] * spread(h_scale[:, n:].to(D), cols)], 1)


def check_backward(dh, y, dy, h, dtype):
    """h: the 64-bit values of the forward's input."""
    c = dy.shape[1]
    g, u, s, want_y = plain(h)
    d = dy.to(D)
    act = g * s
    want = torch.cat([d * u * (s + act * (1 - s)), d * act], 1)
    # 1 - s cancels: the error of s enters act's term whole
    mag = torch.cat([(d * u).abs() * (s + 2 * act.abs()), (d * act).abs()], 1)
    err = rel_error(g, dtype).repeat(1, 2) * mag + 1e-37
    assert ((dh.to(D) - want).abs() <= err + HALF[dtype] * want.abs() * (1 + 2.0 ** -8)).all()
    if y is not None:
        err = rel_error(g, dtype) * want_y.abs() + 1e-37
        assert ((y.to(D) - want_y).abs() <= err + HALF[dtype] * want_y.abs() * (1 + 2.0 ** -8)).all()


@pytest.mark.parametrize("rows, cols", [
    (0, 128), (1, 0), (1, 1), (3, 7), (5, 127), (4, 128), (9, 129), (7, 136), (2, 1001), (300, 250),
    (17, 2048), (1, 14336), (1000, 24)])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("saved", [True, False])
def test_backward(rows, cols, dtype, saved):
    h = rnd(rows, 2 * cols, seed=rows + cols + 1, dtype=dtype)
    dy = rnd(rows, cols, seed=5, dtype=dtype, scale=1e-3)
    dh, y = empty(dtype, rows, 2 * cols), empty(dtype, rows, cols)
    if saved:
        keep = forward(h, ("hq",))
        fp8.fp8_swiglu_backward(dy, keep["hq"], dh, keep["h_scale"], y)
        # the bytes' values are products of two fp32 numbers: one rounding
        check_backward(dh, y, dy, checkpoint_values(keep["hq"], keep["h_scale"], cols), dtype)
    else:
        fp8.fp8_swiglu_backward(dy, h, dh, y=y)
        check_backward(dh, y, dy, h.to(D), dtype)
        assert torch.equal(y, forward(h, ("y",))["y"])
    again = torch.empty_like(dh)
    args = (keep["hq"], again, keep["h_scale"]) if saved else (h, again)
    fp8.fp8_swiglu_backward(dy, *args)  # without y
    assert torch.equal(again, dh)


def test_gradient_against_differences():
    """(f(x + h) - f(x - h)) / 2h of the 64-bit forward: off by h^2/6 of the third
    derivative (below 1 here) and by fp32's roundings of the kernel."""
    h, dy, step = rnd(2, 16, seed=6, dtype=F), rnd(2, 8, seed=7, dtype=F), 1e-4
    dh = empty(F, 2, 16)
    fp8.fp8_swiglu_backward(dy, h, dh)
    d = dy.to(D)
    for r in range(2):
        for c in range(16):
            e = torch.zeros(2, 16, dtype=D, device="cuda")
            e[r, c] = step
            want = ((plain(h.to(D) + e)[3] - plain(h.to(D) - e)[3]) * d).sum() / (2 * step)
            assert abs(dh[r, c].item() - want.item()) < 1e-5


@pytest.mark.parametrize("dtype", [BF, F])
def test_strides_and_unaligned_rows(dtype):
    wide = rnd(50, 600, seed=8, dtype=dtype)
    dwide = rnd(50, 300, seed=9, dtype=dtype)
    for start, cols in ((0, 128), (3, 128), (8, 136), (1, 77)):
        h, dy = wide[:, start:start + 2 * cols], dwide[:, start:start + cols]
        want, got = forward(h.contiguous()), forward(h)
        for name in want:
            assert torch.equal(got[name], want[name]), name
        a, b = empty(dtype, 50, 2 * cols), empty(dtype, 50, 2 * cols)
        fp8.fp8_swiglu_backward(dy.contiguous(), h.contiguous(), a)
        fp8.fp8_swiglu_backward(dy, h, b)
        assert torch.equal(a, b)
    one = wide[:1, :256].expand(20, -1)  # a row stride of 0
    assert torch.equal(forward(one)["yq"], forward(one.contiguous())["yq"])


def test_outputs_at_odd_addresses():
    h = rnd(6, 2 * 128, seed=10, dtype=BF)
    want = forward(h)
    room = torch.zeros(6 * 128 + 1, dtype=torch.uint8, device="cuda")
    yq = room[1:].view(6, 128)
    s = empty(F, 6, 1)
    fp8.fp8_swiglu(h, yq=yq, y_scale=s)
    assert torch.equal(yq, want["yq"]) and torch.equal(s, want["y_scale"]) and room[0] == 0


@pytest.mark.parametrize("live", [-3, 0, 1, 37, 50, 51, 1 << 30])
@pytest.mark.parametrize("cols", [256, 77])
def test_rows_behind_the_live_ones_are_left_as_they_were(live, cols):
    h = rnd(50, 2 * cols, seed=11, dtype=BF)
    n = min(50, max(0, live))
    want = forward(h)
    h[n:] = math.nan
    lv = torch.tensor([live], dtype=torch.int32, device="cuda")
    got = forward(h, live=lv, fill=3)
    for name, t in got.items():
        assert torch.equal(t[:n], want[name][:n]) and (t[n:] == 3).all(), name
    dy = rnd(50, cols, seed=12, dtype=BF)
    full, part = empty(BF, 50, 2 * cols), torch.full((50, 2 * cols), 3.0, dtype=BF, device="cuda")
    y = torch.full((50, cols), 3.0, dtype=BF, device="cuda")
    fp8.fp8_swiglu_backward(dy, want["hq"], full, want["h_scale"])
    fp8.fp8_swiglu_backward(dy, want["hq"], part, want["h_scale"], y, live=lv)
    assert torch.equal(part[:n], full[:n]) and (part[n:] == 3).all() and (y[n:] == 3).all()


def test_nan_and_infinities_stay_in_their_tiles():
    h = rnd(4, 2 * 256, seed=13, dtype=BF)
    clean = forward(h)
    h[1, 5] = math.nan
    h[2, 256 + 130] = math.inf
    out = forward(h)
    assert out["y_scale"][1, 0].isnan() and out["h_scale"][1, 0].isnan()
    assert out["y"][1, 5].isnan() and out["h_scale"][2, 3].isinf()
    for name in ("y", "yq", "y_scale", "hq", "h_scale"):
        assert torch.equal(out[name][0], clean[name][0]) and torch.equal(out[name][3], clean[name][3])
    assert torch.equal(out["yq"][1, 128:], clean["yq"][1, 128:])
    assert torch.equal(out["hq"][1, 128:], clean["hq"][1, 128:])
    # large gates of either sign: s is 0 or 1, nothing overflows
    big = torch.tensor([[-3e38, -200.0, -89.0, 3e38, 200.0, 0.0, -0.0, 1.0] + [1.0] * 8],
                       device="cuda")
    for dtype in (F, BF):
        y, dh = forward(big.to(dtype), ("y",))["y"], empty(dtype, 1, 16)
        assert y.isfinite().all() and (y[0, :2].abs() < 1e-30).all()
        fp8.fp8_swiglu_backward(torch.ones(1, 8, dtype=dtype, device="cuda"), big.to(dtype), dh)
        assert dh.isfinite().all()


def test_a_zero_tile_and_the_scale_floor():
    h = torch.zeros(2, 512, dtype=BF, device="cuda")
    h[1] = 1e-30
    out = forward(h)
    floor = torch.tensor(1e-12, device="cuda") / 448
    assert (out["y_scale"] == floor).all() and (out["h_scale"] == floor).all()
    assert (out["yq"] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("cols", [256, 77])
def test_gradient_over_its_input_another_stream_and_a_graph(dtype, cols):
    h, dy = rnd(70, 2 * cols, seed=14, dtype=dtype), rnd(70, cols, seed=15, dtype=dtype)
    want = empty(dtype, 70, 2 * cols)
    fp8.fp8_swiglu_backward(dy, h, want)
    own = h.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fp8.fp8_swiglu_backward(dy, own, own, stream=s)
    s.synchronize()
    assert torch.equal(own, want)
    held, keep, dh = h.clone(), forward(h), torch.empty_like(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.fp8_swiglu(held, **keep)
        fp8.fp8_swiglu_backward(dy, keep["hq"], dh, keep["h_scale"])
    held.copy_(rnd(70, 2 * cols, seed=16, dtype=dtype))
    graph.replay()
    eager, other = forward(held), torch.empty_like(dh)
    fp8.fp8_swiglu_backward(dy, eager["hq"], other, eager["h_scale"])
    for name in eager:
        assert torch.equal(keep[name], eager[name])
    assert torch.equal(dh, other)


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are those of a small call."""
    rows, cols = 70000, 16384  # h: 2.3e9 elements
    h = torch.zeros(rows, 2 * cols, dtype=BF, device="cuda")
    tail = rnd(3, 2 * cols, seed=17, dtype=BF)
    h[-3:] = tail
    out, small = forward(h, ("yq", "hq")), forward(tail, ("yq", "hq"))
    for name in small:
        assert torch.equal(out[name][-3:], small[name]), name
    dy = torch.zeros(rows, cols, dtype=BF, device="cuda")
    dy[-3:] = 1.0
    dh, one = empty(BF, rows, 2 * cols), empty(BF, 3, 2 * cols)
    fp8.fp8_swiglu_backward(dy, out["hq"], dh, out["h_scale"])
    fp8.fp8_swiglu_backward(dy[-3:], small["hq"], one, small["h_scale"])
    assert torch.equal(dh[-3:], one) and (dh[0] == 0).all()
