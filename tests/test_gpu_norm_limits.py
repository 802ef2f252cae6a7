"""Layer norm at the ends of its arguments' ranges.

The tolerances of the shared checks (32 and 64 units of 2^-24 a row, rows / 128 + 256
a column) for the kernels' shapes.  A row: a thread holds up to 32 elements, whose
squares are 16 additions of pairs and one of the two halves, and the sum over a team is up to
10 levels; the mean's terms cancel, so its leading bits and rests are added apart.  27
roundings in all; up to 40001 columns above the rings' widths: 40 and 10.  A column: its
rows of a block one after the other, at least 128 blocks or 38 clusters of at most 900
rows, 8 teams, and up to 512 blocks by 32 warps: 16 and 5 levels.
"""
import pytest
import torch

import scaled_linear_layers_gb300 as fp8
from scaled_linear_layers_gb300 import _lib
from test_gpu_norm import BF, EPS, F, check_forward, f32, rnd, run_backward

pytestmark = pytest.mark.gpu


@pytest.mark.slow
@pytest.mark.parametrize("cols", [2 ** 31 - 1, 2 ** 31 - 1024])
def test_the_widest_row(cols):
    """The last step of a thread's columns passes 2^31.  A thread adds 2^21 terms
    in fp32, whose roundings of random terms grow as their square root: 1448 * 2^-24
    = 1e-4 of a sum; 5e-4 is allowed, besides the output's 2^-8."""
    g = torch.Generator(device="cuda").manual_seed(80)
    x, dy = (torch.randn(1, cols, generator=g, device="cuda", dtype=BF) for _ in range(2))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd, db = f32(1), f32(1), torch.empty(cols, device="cuda", dtype=BF)
    chunks = [slice(lo, min(cols, lo + 2 ** 26)) for lo in range(0, cols, 2 ** 26)]

    def total(f):
        return sum(f(c).sum() for c in chunks)

    fp8.fp8_layer_norm(x, None, None, EPS, y, mean, rstd)
    m = total(lambda c: x[0, c].double()) / cols
    r = (total(lambda c: (x[0, c].double() - m).square()) / cols + EPS).rsqrt()
    assert abs(mean.item() - m.item()) <= 32 * 2.0 ** -24
    assert abs(rstd.item() - r.item()) <= 5e-4 * r.item()
    for c in chunks:
        ref = (x[0, c].double() - m) * r
        assert ((y[0, c].double() - ref).abs() <= (2.0 ** -8 + 5e-4) * ref.abs() + 1e-5).all()
    ws = torch.empty(fp8.fp8_layer_norm_workspace_bytes(1, cols), dtype=torch.uint8, device="cuda")
    fp8.fp8_layer_norm_backward(dy, x, None, mean, rstd, dx, None, db, ws)
    assert torch.equal(db, dy[0])
    m1 = total(lambda c: dy[0, c].double()) / cols
    m2 = total(lambda c: dy[0, c].double() * (x[0, c].double() - m) * r) / cols
    for c in chunks:
        xhat = (x[0, c].double() - m) * r
        ref = r * (dy[0, c].double() - m1 - xhat * m2)
        assert ((dx[0, c].double() - ref).abs() <= (2.0 ** -8 + 5e-4) * ref.abs()
                + 1e-4 * (1 + xhat.abs())).all()


@pytest.mark.parametrize("rows", [1, 1000, 300000])
def test_rows_without_columns_have_no_mean(rows):
    x = torch.empty(rows, 0, dtype=BF, device="cuda")
    mean, rstd, amax = f32(rows).fill_(3.0), f32(rows).fill_(3.0), f32(1).fill_(3.0)
    fp8.fp8_layer_norm(x, None, None, EPS, torch.empty_like(x), mean, rstd, amax_out=amax)
    assert mean.isnan().all() and rstd.isnan().all()  # 0 / 0, as the formula gives
    assert amax.item() == 0.0
    rstd.fill_(3.0)
    fp8.fp8_layer_norm(x, None, None, EPS, torch.empty_like(x), rstd=rstd)
    assert rstd.isnan().all()


@pytest.mark.parametrize("rows, cols", [(7, 96), (3000, 1024), (3000, 333), (400, 8208),
                                        (400, 9001), (3, 40001)])
@pytest.mark.parametrize("into", ["dy", "x"])
def test_gradient_written_over_its_input(rows, cols, into):
    x, dy = rnd(rows, cols, seed=70), rnd(rows, cols, seed=71)
    w, m = rnd(cols, seed=72), x.double().mean(1)
    r = ((x.double() - m[:, None]).square().mean(1) + EPS).rsqrt()
    ws = torch.empty(fp8.fp8_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8,
                     device="cuda")
    outs = []
    for over in (False, True):
        xi, gi, dw, db = x.clone(), dy.clone(), f32(cols), f32(cols)
        dx = (gi if into == "dy" else xi) if over else torch.empty_like(x)
        fp8.fp8_layer_norm_backward(gi, xi, w, m.float(), r.float(), dx, dw, db, ws)
        outs.append((dx, dw, db))
    for apart, over in zip(*outs):
        assert torch.equal(apart, over)


LIMIT_NS = 1_000_000


def lose_a_call(call):
    """`call` with its rows' copies left out: it ends, and the status says that
    its waits ran out."""
    lib = _lib.load()
    fp8.fp8_check_device_status()
    old = fp8.fp8_set_wait_limit_ns(LIMIT_NS)
    try:
        assert lib.fp8_inject_lost_copies(1) == 0
        call()
        with pytest.raises(fp8.Fp8Error) as e:
            fp8.fp8_check_device_status()
        assert e.value.status == 6  # FP8_ERR_TIMEOUT
    finally:
        lib.fp8_inject_lost_copies(0)
        fp8.fp8_set_wait_limit_ns(old)


# rows enough for the rings: teams of a warp and larger ones, rows that 16-byte
# copies fit and rows that they do not
@pytest.mark.parametrize("rows, cols, dtype", [(12000, 512, BF), (4000, 4096, BF), (12000, 333, BF),
                                               (3500, 1999, F)])
def test_rows_that_never_arrive_are_reported(rows, cols, dtype):
    x, dy = rnd(rows, cols, seed=73, dtype=dtype), rnd(rows, cols, seed=74, dtype=dtype)
    y, mean, rstd = torch.empty_like(x), f32(rows), f32(rows)
    lose_a_call(lambda: fp8.fp8_layer_norm(x, None, None, EPS, y, mean, rstd))
    fp8.fp8_layer_norm(x, None, None, EPS, y, mean, rstd)
    fp8.fp8_check_device_status()
    check_forward(x, None, None, y, mean, rstd)
    ws = torch.empty(fp8.fp8_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8,
                     device="cuda")
    dw = f32(cols)
    lose_a_call(lambda: fp8.fp8_layer_norm_backward(dy, x, None, mean, rstd, y, dw, None, ws))
    run_backward(x, dy, None, F)
    fp8.fp8_check_device_status()


# rows shared by two blocks and by four: the first block's part never arrives, and
# the others wait for its sums
@pytest.mark.parametrize("rows, cols, dtype", [(400, 12288, BF), (300, 16384, F), (400, 9001, BF),
                                               (200, 32768, BF)])
def test_shared_rows_that_never_arrive_are_reported(rows, cols, dtype):
    x, dy = rnd(rows, cols, seed=75, dtype=dtype), rnd(rows, cols, seed=76, dtype=dtype)
    mean, rstd = x.float().mean(1), f32(rows).fill_(1.0)
    ws = torch.empty(fp8.fp8_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8,
                     device="cuda")
    dx, dw = torch.empty_like(x), f32(cols)
    lose_a_call(lambda: fp8.fp8_layer_norm_backward(dy, x, None, mean, rstd, dx, dw, None, ws))
    run_backward(x, dy, None, F)
    fp8.fp8_check_device_status()


def test_lost_copies_refusal():
    assert _lib.load().fp8_inject_lost_copies(-1) == 2
