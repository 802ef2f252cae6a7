"""The experts' linears in one launch, against the products in 64 bits and
against one block-recipe call an expert.  The products of a block are exact in
fp32's range and added with at most a unit's error each, and a block's partial
takes three more roundings, so a result is off by half a unit of bf16 and
k 2^-23 of the sum of its terms' magnitudes (k terms, k >= 128).  One call an
expert adds the same numbers in the same order: equal bits."""
import pytest
import torch

import scaled_linear_layers_gb300 as fp8

pytestmark = pytest.mark.gpu
BF, F, D = torch.bfloat16, torch.float32, torch.float64
B = 128


@pytest.fixture(params=["chosen", "many", "few"])
def kernel(request, monkeypatch):
    """Runs a test on the kernel that the call chooses, and on both."""
    if request.param != "chosen":
        monkeypatch.setenv("FP8LINEAR_MOE_FEW", "1" if request.param == "few" else "0")
    return request.param


def rnd(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(BF)


def empty(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda")


def row_tiles(x):
    """q, scale, qt, scale_t of rows (a multiple of 128) by the block recipe."""
    r, c = x.shape
    q, qt = empty(torch.uint8, r, c), empty(torch.uint8, c, r)
    s, si, st, sit = (empty(F, *shape) for shape in ((r, c // B), (r, c // B), (r // B, c), (r // B, c)))
    fp8.fp8_quantize_transpose(x, fp8.BLOCK, s, si, q, qt, st, sit)
    return q, s, qt, st


def square_tiles(w):
    """wq [E, N, K], w_scale, and wqt [K, E N] of the stacked weights."""
    e, n, k = w.shape
    q, qt = empty(torch.uint8, e * n, k), empty(torch.uint8, k, e * n)
    s, si = empty(F, e * n // B, k // B), empty(F, e * n // B, k // B)
    fp8.fp8_quantize_transpose(w.reshape(e * n, k), fp8.BLOCK_2D, s, si, q, qt)
    return q.view(e, n, k), s.view(e, n // B, k // B), qt


def values(q, scale, rows=1):
    """The 64-bit values of E4M3 bytes under tiles of rows x 128."""
    s = scale.to(D).repeat_interleave(rows, 0).repeat_interleave(B, 1)
    return q.view(torch.float8_e4m3fn).to(D) * s[:q.shape[0]]


def offsets_of(counts, multiple):
    at = [0]
    for n in counts:
        at.append(at[-1] + -(-n // multiple) * multiple)
    return at, torch.tensor(at, dtype=torch.int32, device="cuda")


def near(got, a, b, k):
    """got against a · b^T in 64 bits."""
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    tol = 2.0 ** -8 * (1 + 2.0 ** -8) * want.abs() + (1 + 2.0 ** -7) * k * 2.0 ** -23 * mag
    off = (got.to(D) - want).abs()
    assert (off <= tol).all(), f"{(off > tol).sum().item()} of {off.numel()} outside"


SIZES = [
    # counts, multiple, N, K
    ([5], 1, 128, 128),
    ([0, 1, 0], 1, 256, 128),
    ([1, 2, 3, 4, 5, 6, 7, 8], 1, 384, 640),
    ([16, 0, 33, 128, 129, 7], 16, 256, 512),
    ([300, 0, 0, 511, 1], 128, 640, 384),
    ([128, 256, 384], 128, 512, 896),
    ([0, 0], 128, 128, 256),
    ([1] * 200, 1, 128, 256),
    ([700, 45], 1, 1152, 1024),
    ([9, 64, 65, 100], 1, 256, 4224),
]


def case(counts, multiple, seed, extra=0):
    at, offsets = offsets_of(counts, multiple)
    cap = -(-(at[-1] + extra) // B) * B
    return at, offsets, cap


@pytest.mark.parametrize("counts, multiple, N, K", SIZES)
@pytest.mark.parametrize("extra", [0, 300])
def test_fprop_and_dgrad(counts, multiple, N, K, extra, kernel):
    at, offsets, cap = case(counts, multiple, 1, extra)
    if cap == 0:
        cap = B
    e = len(counts)
    w = rnd(e, N, K, seed=2, scale=K ** -0.5)
    wq, ws, wqt = square_tiles(w)
    for which, wide, out in (("fprop", K, N), ("dgrad", N, K)):
        q, s, _, _ = row_tiles(rnd(cap, wide, seed=3))
        y = torch.full((cap, out), 7.0, dtype=BF, device="cuda")
        if which == "fprop":
            fp8.fp8_moe_linear_fprop(q, s, wq, ws, offsets, y)
        else:
            fp8.fp8_moe_linear_dgrad(q, s, wqt, ws, offsets, y)
        x = values(q, s)
        for i in range(e):
            wv = values(wq[i], ws[i], B)
            near(y[at[i]:at[i + 1]], x[at[i]:at[i + 1]], wv if which == "fprop" else wv.t(), wide)
        assert (y[at[-1]:] == 7.0).all()  # rows behind the last segment
    fp8.fp8_check_device_status()


@pytest.mark.parametrize("counts, N, K", [([300, 0, 0, 511, 1], 640, 384), ([128, 256, 384], 512, 896),
                                          ([0, 0], 128, 256), ([1, 1500], 256, 128),
                                          ([4, 5, 6] * 20, 128, 384)])
def test_wgrad(counts, N, K):
    at, offsets, cap = case(counts, B, 4, 200)
    g, x = rnd(cap, N, seed=5, scale=1e-3), rnd(cap, K, seed=6)
    _, _, gqt, gst = row_tiles(g)
    _, _, xqt, xst = row_tiles(x)
    dw = torch.full((len(counts), N, K), 7.0, dtype=BF, device="cuda")
    fp8.fp8_moe_linear_wgrad(gqt, gst, xqt, xst, offsets, dw)
    gv, xv = values(gqt, gst.t()), values(xqt, xst.t())
    for i in range(len(counts)):
        lo, hi = at[i], at[i + 1]
        if hi == lo:
            assert (dw[i] == 0).all()
        else:
            near(dw[i], gv[:, lo:hi], xv[:, lo:hi], max(B, hi - lo))
    fp8.fp8_check_device_status()


def test_the_bits_of_one_call_an_expert(kernel):
    counts, N, K = [128, 640, 0, 256], 512, 768
    at, offsets, cap = case(counts, B, 7)
    w, x, g = rnd(4, N, K, seed=8), rnd(cap, K, seed=9), rnd(cap, N, seed=10, scale=1e-3)
    wq, ws, wqt = square_tiles(w)
    xq, xs, xqt, xst = row_tiles(x)
    gq, gs, gqt, gst = row_tiles(g)
    y, dx, dw = empty(BF, cap, N), empty(BF, cap, K), empty(BF, 4, N, K)
    fp8.fp8_moe_linear_fprop(xq, xs, wq, ws, offsets, y)
    fp8.fp8_moe_linear_dgrad(gq, gs, wqt, ws, offsets, dx)
    fp8.fp8_moe_linear_wgrad(gqt, gst, xqt, xst, offsets, dw)
    for i in range(4):
        lo, hi = at[i], at[i + 1]
        if hi == lo:
            continue
        m = hi - lo
        one = empty(BF, m, N)
        fp8.fp8_linear_fprop(xq[lo:hi], xs[lo:hi], wq[i], ws[i], m, N, K, fp8.BLOCK, None, one)
        assert torch.equal(one, y[lo:hi])
        one = empty(BF, m, K)
        wt = wqt[:, i * N:(i + 1) * N].contiguous()
        fp8.fp8_linear_dgrad(gq[lo:hi], gs[lo:hi], wt, ws[i], m, N, K, fp8.BLOCK, one)
        assert torch.equal(one, dx[lo:hi])
        one = empty(BF, N, K)
        blocks = slice(lo // B, hi // B)
        fp8.fp8_linear_wgrad(gqt[:, lo:hi].contiguous(), gst[blocks].contiguous(),
                             xqt[:, lo:hi].contiguous(), xst[blocks].contiguous(), m, N, K,
                             fp8.BLOCK, one)
        assert torch.equal(one, dw[i])


def test_nan_outside_the_segments_reaches_nothing(kernel):
    counts, N, K = [40, 0, 200, 3], 256, 256
    at, offsets, cap = case(counts, B, 11, 130)
    wq, ws, wqt = square_tiles(rnd(4, N, K, seed=12))
    xq, xs, xqt, xst = row_tiles(rnd(cap, K, seed=13))
    gq, gs, gqt, gst = row_tiles(rnd(cap, N, seed=14))

    def all_three():
        y, dx = (torch.full((cap, c), 3.0, dtype=BF, device="cuda") for c in (N, K))
        dw = empty(BF, 4, N, K)
        fp8.fp8_moe_linear_fprop(xq, xs, wq, ws, offsets, y)
        fp8.fp8_moe_linear_dgrad(gq, gs, wqt, ws, offsets, dx)
        fp8.fp8_moe_linear_wgrad(gqt, gst, xqt, xst, offsets, dw)
        return y, dx, dw

    want = all_three()
    end = at[-1]
    for q, s in ((xq, xs), (gq, gs)):
        q[end:], s[end:] = 0x7F, float("nan")
    for q, s in ((xqt, xst), (gqt, gst)):
        q[:, end:], s[end // B:] = 0x7F, float("inf")
    for got, w in zip(all_three(), want):
        assert torch.equal(got, w)
    # one row's NaN stays in that row of y
    xq[5] = 0x7F
    y = all_three()[0]
    assert y[5].isnan().all() and torch.equal(y[:5], want[0][:5]) and torch.equal(y[6:], want[0][6:])


def test_wgrad_of_segments_off_the_blocks_is_nan():
    N, K, cap = 128, 256, 384
    _, _, gqt, gst = row_tiles(rnd(cap, N, seed=15))
    _, _, xqt, xst = row_tiles(rnd(cap, K, seed=16))
    offsets = torch.tensor([0, 128, 200, 384], dtype=torch.int32, device="cuda")
    dw = empty(BF, 3, N, K)
    fp8.fp8_moe_linear_wgrad(gqt, gst, xqt, xst, offsets, dw)
    assert dw[0].isfinite().all() and dw[1].isnan().all() and dw[2].isnan().all()


def test_offsets_outside_the_rows_are_held_inside(kernel):
    N, K, cap = 128, 128, 256
    wq, ws, _ = square_tiles(rnd(3, N, K, seed=17))
    xq, xs, xqt, xst = row_tiles(rnd(cap, K, seed=18))
    y = torch.full((cap, N), 3.0, dtype=BF, device="cuda")
    offsets = torch.tensor([-5, 100, 90, 1 << 30], dtype=torch.int32, device="cuda")
    fp8.fp8_moe_linear_fprop(xq, xs, wq, ws, offsets, y)
    x = values(xq, xs)
    near(y[:90], x[:90], values(wq[0], ws[0], B), K)
    near(y[100:], x[100:], values(wq[2], ws[2], B), K)
    dw = empty(BF, 3, K, K)
    fp8.fp8_moe_linear_wgrad(xqt, xst, xqt, xst, torch.tensor([-128, 0, 128, 1 << 30],
                                                              dtype=torch.int32, device="cuda"), dw)
    assert (dw[0] == 0).all() and dw[1:].isfinite().all()
    fp8.fp8_check_device_status()


def test_no_rows_at_all():
    wq, ws, wqt = square_tiles(rnd(2, 128, 128, seed=19))
    none = lambda dtype, *s: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    fp8.fp8_moe_linear_fprop(none(torch.uint8, 0, 128), none(F, 0, 1), wq, ws, offsets,
                             none(BF, 0, 128))
    fp8.fp8_moe_linear_dgrad(none(torch.uint8, 0, 128), none(F, 0, 1), wqt, ws, offsets,
                             none(BF, 0, 128))
    dw = torch.full((2, 128, 128), 7.0, dtype=BF, device="cuda")
    fp8.fp8_moe_linear_wgrad(none(torch.uint8, 128, 0), none(F, 0, 128), none(torch.uint8, 128, 0),
                             none(F, 0, 128), offsets, dw)
    assert (dw == 0).all()


def test_two_streams_and_a_replayed_graph_with_new_offsets(kernel):
    N, K, cap = 384, 512, 512
    wq, ws, _ = square_tiles(rnd(4, N, K, seed=20))
    xq, xs, _, _ = row_tiles(rnd(cap, K, seed=21))
    table = [[0, 100, 200, 300, 512], [0, 0, 0, 512, 512], [0, 1, 2, 3, 4]]

    def eager(at):
        y = torch.zeros(cap, N, dtype=BF, device="cuda")
        fp8.fp8_moe_linear_fprop(xq, xs, wq, ws, torch.tensor(at, dtype=torch.int32, device="cuda"), y)
        return y

    want = [eager(at) for at in table]
    held, y = torch.tensor(table[0], dtype=torch.int32, device="cuda"), torch.zeros_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y.zero_()
        fp8.fp8_moe_linear_fprop(xq, xs, wq, ws, held, y)
    for at, w in zip(table, want):
        held.copy_(torch.tensor(at, dtype=torch.int32))
        graph.replay()
        assert torch.equal(y, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in table]
    outs = [torch.zeros_like(w) for w in want]
    offs = [torch.tensor(at, dtype=torch.int32, device="cuda") for at in table]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, out in zip(streams, offs, outs):
            fp8.fp8_moe_linear_fprop(xq, xs, wq, ws, o, out, stream=s)
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out, w)


def test_a_wait_that_runs_out_is_reported(kernel):
    N, K, cap = 512, 1024, 1024
    wq, ws, _ = square_tiles(rnd(4, N, K, seed=22))
    xq, xs, _, _ = row_tiles(rnd(cap, K, seed=23))
    offsets = torch.tensor([0, 256, 512, 768, 1024], dtype=torch.int32, device="cuda")
    want, y = empty(BF, cap, N), empty(BF, cap, N)
    fp8.fp8_moe_linear_fprop(xq, xs, wq, ws, offsets, want)
    fp8.fp8_check_device_status()
    old = fp8.fp8_set_wait_limit_ns(1)
    try:
        fp8.fp8_moe_linear_fprop(xq, xs, wq, ws, offsets, y)
        torch.cuda.synchronize()
    finally:
        fp8.fp8_set_wait_limit_ns(old)
    try:  # waits that look at the clock give up; those already served do not
        fp8.fp8_check_device_status()
    except fp8.Fp8Error as e:
        assert e.status == 6
    fp8.fp8_moe_linear_fprop(xq, xs, wq, ws, offsets, y)
    fp8.fp8_check_device_status()
    assert torch.equal(y, want)


def test_a_tile_that_takes_longer_than_a_wait():
    """The search for tiles runs ahead of a tile of 2^14 blocks (9 ms or so),
    further than the 3 ms that every other wait is held to."""
    N, K, cap, experts = 128, 128, 1 << 21, 1024
    g = torch.Generator(device="cuda").manual_seed(24)
    gqt, xqt = (torch.randint(0, 120, (n, cap), generator=g, dtype=torch.uint8, device="cuda")
                for n in (N, K))
    gst, xst = (torch.rand(cap // B, n, generator=g, device="cuda") for n in (N, K))
    offsets = torch.full((experts + 1,), cap, dtype=torch.int32, device="cuda")
    offsets[0] = 0
    dw, one = empty(BF, experts, N, K), empty(BF, N, K)
    fp8.fp8_linear_wgrad(gqt, gst, xqt, xst, cap, N, K, fp8.BLOCK, one)
    torch.cuda.synchronize()
    old = fp8.fp8_set_wait_limit_ns(3000000)
    try:
        fp8.fp8_moe_linear_wgrad(gqt, gst, xqt, xst, offsets, dw)
        torch.cuda.synchronize()
    finally:
        fp8.fp8_set_wait_limit_ns(old)
    fp8.fp8_check_device_status()
    assert torch.equal(dw[0], one) and (dw[1:] == 0).all()


@pytest.mark.parametrize("N, K", [(384, 640), (128, 128), (256, 1152)])
def test_every_row_count_of_the_last_tile(N, K):
    """Outputs leave through boxes of eight rows: none behind a segment."""
    counts = [1, 7, 8, 9, 31, 32, 33, 63, 65, 96, 97, 127, 129, 161]
    at, offsets, cap = case(counts, 1, 25, 200)
    wq, ws, _ = square_tiles(rnd(len(counts), N, K, seed=26))
    xq, xs, _, _ = row_tiles(rnd(cap, K, seed=27))
    y = {}
    for few in "01":
        with pytest.MonkeyPatch.context() as env:
            env.setenv("FP8LINEAR_MOE_FEW", few)
            y[few] = torch.full((cap, N), 7.0, dtype=BF, device="cuda")
            fp8.fp8_moe_linear_fprop(xq, xs, wq, ws, offsets, y[few])
    assert torch.equal(y["0"], y["1"]) and (y["0"][at[-1]:] == 7.0).all()


@pytest.mark.parametrize("cap", [1, 5, 16, 17, 63, 100, 131])
def test_capacities_smaller_than_a_copy(cap, kernel):
    """Any number of rows: copies of 16 to 128 rows reach past the last."""
    N, K = 256, 640
    offsets = torch.tensor([0, cap // 3, cap // 3, cap], dtype=torch.int32, device="cuda")
    w = rnd(3, N, K, seed=28, scale=K ** -0.5)
    wq, ws, wqt = square_tiles(w)
    for which, wide, out in (("fprop", K, N), ("dgrad", N, K)):
        full = row_tiles(rnd(2 * B, wide, seed=29))
        # exactly cap rows, in memory of their own
        q, s = full[0][:cap].clone(), full[1][:cap].clone()
        y = torch.full((cap + 8, out), 7.0, dtype=BF, device="cuda")
        if which == "fprop":
            fp8.fp8_moe_linear_fprop(q, s, wq, ws, offsets, y[:cap])
        else:
            fp8.fp8_moe_linear_dgrad(q, s, wqt, ws, offsets, y[:cap])
        x = values(q, s)
        for i, (lo, hi) in enumerate(((0, cap // 3), (cap // 3, cap // 3), (cap // 3, cap))):
            wv = values(wq[i], ws[i], B)
            near(y[lo:hi], x[lo:hi], wv if which == "fprop" else wv.t(), wide)
        assert (y[cap:] == 7.0).all()
    fp8.fp8_check_device_status()
