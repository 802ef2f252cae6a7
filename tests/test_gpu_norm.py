"""Layer norm against the formula in 64 bits.

Tolerances.  u = 2^-24.  A row's sum is formed by at most 16 (in the wide
kernel cols/1024) serial additions and 10 tree levels, so the mean is within
30 u mean|x| and, through the squares, rstd within about 30 u relative; with
the pointwise roundings 64 u times the terms' magnitudes bounds each output,
plus half a unit of the output's type (2^-8 relative in bf16).  Column sums:
each block adds rows/blocks values (at least 128 blocks once there are as many
rows), the blocks' sums are added by 8 warps.
"""
import numpy as np
import pytest
import torch

import scaled_linear_layers_gb300 as fp8

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5
OUT = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F = torch.bfloat16, torch.float32


def rnd(*shape, seed, dtype=F, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def f32(*shape):
    return torch.empty(shape, device="cuda")


def reference(x, w, b, eps=EPS):
    x = x.double()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1 / (xc.square().mean(1) + eps).sqrt()
    xhat = xc * rstd[:, None]
    w = torch.ones_like(x[0]) if w is None else w.double()
    b = torch.zeros_like(x[0]) if b is None else b.double()
    return mean, rstd, xhat, xhat * w + b, w, b


def check_forward(x, w, b, y, mean, rstd, eps=EPS):
    m, r, xhat, ref, wd, bd = reference(x, w, b, eps)
    xa = x.double().abs()
    assert ((mean.double() - m).abs() <= 32 * U * xa.mean(1) + 1e-38).all()
    # rstd is as uncertain as the spread is against the largest entry
    cond = 1 + (xa.amax(1) * r)
    assert ((rstd.double() - r).abs() <= 64 * U * r * cond).all()
    err = (y.double() - ref).abs()
    tol = 64 * U * (wd.abs() * ((r * xa.amax(1))[:, None] + xhat.abs() * cond[:, None]) + bd.abs()) \
        + OUT[y.dtype] * ref.abs() + 1e-38
    assert (err <= tol).all(), f"{(err / tol).max().item():.2f} x the tolerance"


SHAPES = [(1, 1), (1, 8), (1, 4096), (3, 7), (5, 512), (17, 513), (200, 64), (33, 1000),
          (64, 1023), (7, 2048), (301, 4096), (9, 5000), (4, 8192), (3, 16384), (2, 20001)]


@pytest.mark.parametrize("rows, cols", SHAPES)
@pytest.mark.parametrize("dtype, param", [(BF, BF), (BF, F), (F, F), (F, BF)])
def test_forward(rows, cols, dtype, param):
    x = rnd(rows, cols, seed=1, dtype=dtype, scale=2.0, shift=0.5)
    w, b = rnd(cols, seed=2, dtype=param, shift=1.0), rnd(cols, seed=3, dtype=param)
    y, mean, rstd = torch.empty_like(x), f32(rows), f32(rows)
    fp8.fp8_layer_norm(x, w, b, EPS, y, mean, rstd)
    check_forward(x, w, b, y, mean, rstd)


def test_forward_many_rows_more_than_a_wave():
    x = rnd(5003, 256, seed=4, dtype=BF)
    y, mean, rstd = torch.empty_like(x), f32(5003), f32(5003)
    fp8.fp8_layer_norm(x, None, None, EPS, y, mean, rstd)
    check_forward(x, None, None, y, mean, rstd)


@pytest.mark.parametrize("w, b", [(False, True), (True, False), (False, False)])
def test_forward_without_parameters(w, b):
    x = rnd(9, 96, seed=5, dtype=F)
    w = rnd(96, seed=6) if w else None
    b = rnd(96, seed=7) if b else None
    y, mean, rstd = torch.empty_like(x), f32(9), f32(9)
    fp8.fp8_layer_norm(x, w, b, EPS, y, mean, rstd)
    check_forward(x, w, b, y, mean, rstd)


def test_forward_large_mean_small_spread():
    # a sum of squares minus the square of the sum would lose every digit here
    x = rnd(8, 1024, seed=8, dtype=F, scale=1e-2, shift=1000.0)
    y, mean, rstd = torch.empty_like(x), f32(8), f32(8)
    fp8.fp8_layer_norm(x, None, None, 0.0, y, mean, rstd)
    check_forward(x, None, None, y, mean, rstd, eps=0.0)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("offset, width, stride", [(0, 64, 200), (1, 64, 200), (8, 128, 136),
                                                   (3, 77, 101)])
def test_forward_strided_rows_and_offsets(dtype, offset, width, stride):
    base = rnd(21, stride, seed=9, dtype=dtype)
    x = base[:, offset:offset + width]
    y, mean, rstd = torch.empty(21, width, dtype=dtype, device="cuda"), f32(21), f32(21)
    fp8.fp8_layer_norm(x, None, None, EPS, y, mean, rstd)
    check_forward(x, None, None, y, mean, rstd)
    # one row broadcast over all
    row = base[:1, :width].expand(21, width)
    fp8.fp8_layer_norm(row, None, None, EPS, y, mean, rstd)
    check_forward(row, None, None, y, mean, rstd)


@pytest.mark.parametrize("rows, cols", [(1, 16), (37, 4096), (300, 515), (2, 17000)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_forward_to_e4m3(rows, cols, dtype):
    x = rnd(rows, cols, seed=10, dtype=dtype)
    w, b = rnd(cols, seed=11, shift=1.0), rnd(cols, seed=12)
    y32 = f32(rows, cols)
    # fp32 rows give the unrounded y; the values are those of bf16 x
    fp8.fp8_layer_norm(x.float(), w, b, EPS, y32)
    si = torch.full((1,), 60.0, device="cuda")  # saturates some entries
    q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    y, amax, mean, rstd = torch.empty_like(x), f32(1).fill_(9e9), f32(rows), f32(rows)
    fp8.fp8_layer_norm(x, w, b, EPS, y, mean, rstd, yq=q, scale_inv=si, amax_out=amax)
    check_forward(x, w, b, y, mean, rstd)
    _, _, _, ref, wd, bd = reference(x, w, b)
    # the bytes are the cast of a value within the fp32 tolerance of y * 60
    tol = 64 * U * (wd.abs() * (8 + ref.abs()) + bd.abs() + ref.abs()) * 60
    lo = ((ref * 60) - tol).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    hi = ((ref * 60) + tol).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    assert ((q.float() >= lo) & (q.float() <= hi)).all()
    assert abs(amax.item() - ref.abs().max().item()) <= 64 * U * (8 + ref.abs().max().item()) * \
        (wd.abs().max().item() + 1)
    q2 = torch.empty_like(q)
    fp8.fp8_layer_norm(x, w, b, EPS, yq=q2, scale_inv=si)  # the bytes alone
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8))


def test_forward_nan_and_inf_stay_in_their_rows():
    x = rnd(6, 300, seed=13, dtype=BF)
    x[1, 7] = float("nan")
    x[4, 299] = float("inf")
    y, mean, rstd, amax = torch.empty_like(x), f32(6), f32(6), f32(1)
    q, si = torch.empty(6, 300, dtype=torch.uint8, device="cuda"), f32(1).fill_(1.0)
    fp8.fp8_layer_norm(x, None, None, EPS, y, mean, rstd, yq=q, scale_inv=si, amax_out=amax)
    ok = [0, 2, 3, 5]
    check_forward(x[ok], None, None, y[ok], mean[ok], rstd[ok])
    assert y[1].isnan().all() and y[4].isnan().any() and amax.isnan().all()


def backward_reference(dy, x, w, mean, rstd):
    dy, x, r = dy.double(), x.double(), rstd.double()[:, None]
    w = torch.ones_like(x[0]) if w is None else w.double()
    xhat = (x - mean.double()[:, None]) * r
    wdy = dy * w
    dx = r * (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True))
    mag = r * (wdy.abs() + wdy.abs().mean(1, keepdim=True)
               + xhat.abs() * (wdy * xhat).abs().mean(1, keepdim=True))
    return dx, mag, (dy * xhat), dy


def run_backward(x, dy, w, param, want=(True, True, True)):
    rows, cols = x.shape
    m64, r64 = reference(x, None, None)[:2]
    mean, rstd = m64.float(), r64.float()
    new = lambda dtype, *s: torch.full(s, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    dx = new(x.dtype, rows, cols) if want[0] else None
    dw = new(param, cols) if want[1] else None
    db = new(param, cols) if want[2] else None
    ws = torch.empty(fp8.fp8_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8,
                     device="cuda")
    fp8.fp8_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
    rdx, mag, tw, tb = backward_reference(dy, x, w, mean, rstd)
    if want[0]:
        err, tol = (dx.double() - rdx).abs(), 64 * U * mag + OUT[x.dtype] * rdx.abs() + 1e-38
        assert (err <= tol).all(), f"dx: {(err / tol).max().item():.2f} x the tolerance"
    n = rows / 128 + 256
    for got, terms, on in ((dw, tw, want[1]), (db, tb, want[2])):
        if on:
            ref = terms.sum(0)
            err = (got.double() - ref).abs()
            tol = n * U * terms.abs().sum(0) + OUT[param] * ref.abs() + 1e-38
            assert (err <= tol).all(), f"{(err / tol).max().item():.2f} x the tolerance"
    return dx, dw, db


@pytest.mark.parametrize("rows, cols", SHAPES + [(5003, 256), (2000, 1023), (700, 8200)])
@pytest.mark.parametrize("dtype, param", [(BF, BF), (BF, F), (F, F)])
def test_backward(rows, cols, dtype, param):
    x = rnd(rows, cols, seed=20, dtype=dtype, scale=2.0, shift=0.5)
    dy = rnd(rows, cols, seed=21, dtype=dtype, scale=1e-2)
    run_backward(x, dy, rnd(cols, seed=22, dtype=param, shift=1.0), param)


@pytest.mark.parametrize("want", [(True, False, False), (False, True, True), (False, False, True),
                                  (True, True, False)])
@pytest.mark.parametrize("cols", [64, 20001])
def test_backward_some_outputs(want, cols):
    x, dy = rnd(40, cols, seed=23, dtype=BF), rnd(40, cols, seed=24, dtype=BF)
    run_backward(x, dy, None, F, want)


def test_backward_strided_and_broadcast_inputs():
    base, gb = rnd(50, 300, seed=25), rnd(50, 270, seed=26)
    run_backward(base[:, 5:5 + 256], gb[:, 3:3 + 256], rnd(256, seed=27), F)
    # a gradient broadcast over the rows, as the gradient of a sum is
    run_backward(base[:, :256], gb[:1, :256].expand(50, 256), None, F)


# rows shared by two blocks or four (and wider): widths at both ends of each, one
# row to more than each has slots for
@pytest.mark.parametrize("rows, cols", [(1, 8200), (3, 9001), (400, 8208), (700, 12288), (900, 13256),
                                        (420, 16384), (350, 16383), (2, 16392), (5, 20001),
                                        (250, 32768), (260, 32767), (70, 32776), (2, 40001)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_backward_of_shared_rows(rows, cols, dtype):
    x = rnd(rows, cols, seed=50, dtype=dtype, scale=2.0, shift=0.5)
    dy = rnd(rows, cols, seed=51, dtype=dtype, scale=1e-2)
    run_backward(x, dy, rnd(cols, seed=52, dtype=F, shift=1.0), F)


def test_backward_of_shared_rows_strided_and_some_outputs():
    base, gb = rnd(300, 9100, seed=53), rnd(300, 9031, seed=54)
    x, dy = base[:, 3:3 + 9001], gb[:, 5:5 + 9001]
    run_backward(x, dy, rnd(9001, seed=55, dtype=BF), BF)
    run_backward(x, gb[:1, :9001].expand(300, 9001), None, F, (True, False, False))
    run_backward(x, dy, None, F, (False, True, True))
    a, b = run_backward(x, dy, None, F), run_backward(x, dy, None, F)
    for s, t in zip(a, b):
        assert torch.equal(s, t)


# enough rows for the ring, which 16-byte copies do not fit: odd widths, odd
# strides, starts between two elements' 16-byte groups
@pytest.mark.parametrize("rows, cols, stride, offset", [(9000, 1, 1, 0), (9000, 7, 11, 3),
                                                        (9001, 333, 333, 1), (3500, 1999, 2001, 5),
                                                        (1700, 3001, 3001, 7), (900, 8191, 8192, 1),
                                                        (500, 9001, 9001, 0)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_many_rows_of_odd_width(rows, cols, stride, offset, dtype):
    room = offset + rows * stride
    x = rnd(1, room, seed=56, dtype=dtype, shift=0.5)[0, offset:].view(rows, stride)[:, :cols]
    dy = rnd(1, room, seed=57, dtype=dtype)[0, offset:].view(rows, stride)[:, :cols]
    w, b = rnd(cols, seed=58, dtype=F, shift=1.0), rnd(cols, seed=59, dtype=F)
    y, mean, rstd = torch.empty(rows, cols, dtype=dtype, device="cuda"), f32(rows), f32(rows)
    fp8.fp8_layer_norm(x, w, b, EPS, y, mean, rstd)
    check_forward(x, w, b, y, mean, rstd)
    if cols > 1:
        run_backward(x, dy, w, F)


def test_backward_of_no_rows_is_zero():
    x = torch.empty(0, 96, dtype=BF, device="cuda")
    e = torch.empty(0, device="cuda")
    dw, db = f32(96).fill_(3.0), f32(96).fill_(3.0)
    fp8.fp8_layer_norm_backward(x, x, None, e, e, torch.empty_like(x), dw, db)
    assert (dw == 0).all() and (db == 0).all()
    fp8.fp8_layer_norm(x, None, None, EPS, torch.empty_like(x))


def test_backward_repeats_bit_for_bit():
    x, dy = rnd(3000, 1024, seed=28, dtype=BF), rnd(3000, 1024, seed=29, dtype=BF)
    a, b = run_backward(x, dy, None, F), run_backward(x, dy, None, F)
    for s, t in zip(a, b):
        assert torch.equal(s, t)


@pytest.mark.parametrize("cols", [40, 777])
def test_backward_against_differences(cols):
    """Central differences of the formula in 64 bits, along random directions:
    step h = 1e-6 leaves an error of order h^2 and 1e-16/h, well below 1e-6;
    the fp32 gradient itself is good for 64 u sqrt(rows cols) < 1e-4."""
    rows = 6
    x, dy, w = (rnd(rows, cols, seed=30), rnd(rows, cols, seed=31), rnd(cols, seed=32, shift=1.0))
    dx, dw, db = run_backward(x, dy, w, F)
    loss = lambda x, w, b: (reference(x, w, b)[3] * dy.double()).sum()  # noqa: E731
    zero = torch.zeros(cols, device="cuda", dtype=torch.float64)
    for seed in (33, 34):
        v, vw = rnd(rows, cols, seed=seed).double(), rnd(cols, seed=seed + 5).double()
        h = 1e-6
        args = (x.double(), w.double(), zero)
        for i, (grad, vec) in enumerate(((dx, v), (dw, vw), (db, vw))):
            hi, lo = list(args), list(args)
            hi[i], lo[i] = args[i] + h * vec, args[i] - h * vec
            num = ((loss(*hi) - loss(*lo)) / (2 * h)).item()
            got = (grad.double() * vec).sum().item()
            scale = (grad.double() * vec).abs().sum().item()
            assert abs(num - got) <= 1e-4 * scale


def test_another_stream_and_graph():
    x = rnd(64, 512, seed=40, dtype=BF)
    y, mean, rstd = torch.empty_like(x), f32(64), f32(64)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    fp8.fp8_layer_norm(x, None, None, EPS, y, mean, rstd, stream=s)
    s.synchronize()
    check_forward(x, None, None, y, mean, rstd)
    y.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp8.fp8_layer_norm(x, None, None, EPS, y, mean, rstd)
    x.copy_(rnd(64, 512, seed=41, dtype=BF))
    g.replay()
    torch.cuda.synchronize()
    check_forward(x, None, None, y, mean, rstd)


def test_python_refusals():
    x = rnd(4, 8, seed=50)
    y = torch.empty_like(x)
    ok = lambda **k: fp8.fp8_layer_norm(**{**dict(x=x, weight=None, bias=None, eps=EPS, y=y), **k})  # noqa: E731
    ok()
    for bad in (dict(x=x.half()), dict(x=x.t()), dict(x=x[0]), dict(y=y[:2]), dict(y=y.bfloat16()),
                dict(y=None), dict(weight=x[0].bfloat16(), bias=x[0]), dict(weight=x[0, :4]),
                dict(mean=y[0]), dict(yq=y), dict(x=x.cpu()),
                dict(yq=torch.empty(4, 8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fp8.Fp8Error):
            ok(**bad)


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    """A limit of 1 ns makes the waits for rows on their way give up; the call
    ends, the status says so, and nothing is left behind."""
    x, dy = rnd(6000, 1024, seed=60, dtype=BF), rnd(6000, 1024, seed=61, dtype=BF)
    y, mean, rstd = torch.empty_like(x), f32(6000), f32(6000)
    dw = f32(1024)
    ws = torch.empty(fp8.fp8_layer_norm_workspace_bytes(6000, 1024), dtype=torch.uint8,
                     device="cuda")
    fp8.fp8_check_device_status()
    old = fp8.fp8_set_wait_limit_ns(1)
    try:
        fp8.fp8_layer_norm(x, None, None, EPS, y, mean, rstd)
        fp8.fp8_layer_norm_backward(dy, x, None, mean, rstd, y, dw, None, ws)
        try:
            fp8.fp8_check_device_status()
        except fp8.Fp8Error as e:
            assert e.status == 6  # FP8_ERR_TIMEOUT
    finally:
        fp8.fp8_set_wait_limit_ns(old)
    fp8.fp8_layer_norm(x, None, None, EPS, y, mean, rstd)
    check_forward(x, None, None, y, mean, rstd)
    run_backward(x, dy, None, F)
    fp8.fp8_check_device_status()
