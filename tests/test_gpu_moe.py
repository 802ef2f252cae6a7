"""Expert rows (sort, dispatch, combine and their gradients) against plain
definitions: the sort, the copies and the casts exactly; sums within (terms +
2) * 2^-24 of the terms' magnitudes, plus half a unit of the output's type."""
import numpy as np
import pytest
import torch

import scaled_linear_layers_gb300 as fp8

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
OUT = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F = torch.bfloat16, torch.float32


def rnd(*shape, seed, dtype=F, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def random_ids(tokens, topk, experts, seed, drop=0.1):
    r = np.random.default_rng(seed)
    ids = (r.random((tokens, topk)) ** 2 * experts).astype(np.int64)  # skewed to low experts
    ids[r.random((tokens, topk)) < drop] = -1
    return ids


def plain_sort(ids, experts, multiple, capacity):
    flat = ids.reshape(-1)
    row_of = np.full(flat.size, -1, np.int64)
    source = np.full(capacity, -1, np.int64)
    offsets, counts, at = [0], [], 0
    for e in range(experts):
        mine = np.flatnonzero(flat == e)
        row_of[mine] = at + np.arange(mine.size)
        source[at:at + mine.size] = mine
        at += -(-mine.size // multiple) * multiple
        offsets.append(at)
        counts.append(mine.size)
    return row_of.reshape(ids.shape), source, np.array(offsets), np.array(counts)


def sort(ids, experts, multiple, capacity=None, dtype=torch.int32):
    ids = torch.from_numpy(ids).to(dtype).cuda()
    n = ids.numel()
    cap = fp8.fp8_moe_capacity(n, experts, multiple) if capacity is None else capacity
    i32 = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")  # noqa: E731
    row_of, source, offsets, counts = i32(*ids.shape), i32(cap), i32(experts + 1), i32(experts)
    ws = torch.empty(fp8.fp8_moe_sort_workspace_bytes(n, experts), dtype=torch.uint8,
                     device="cuda")
    fp8.fp8_moe_sort(ids, experts, multiple, row_of, source, offsets, counts, ws)
    return row_of, source, offsets, counts


@pytest.mark.parametrize("tokens, topk, experts", [
    (0, 2, 4), (1, 1, 1), (1, 8, 64), (5, 3, 7), (33, 2, 8), (1000, 4, 32), (512, 8, 8),
    (513, 8, 33), (700, 6, 1024), (4097, 1, 5), (3000, 8, 160), (70001, 8, 64)])
@pytest.mark.parametrize("multiple", [1, 16, 128])
def test_sort(tokens, topk, experts, multiple):
    ids = random_ids(tokens, topk, experts, seed=tokens + topk)
    got = sort(ids, experts, multiple)
    want = plain_sort(ids, experts, multiple, got[1].shape[0])
    for g, w, name in zip(got, want, ("row_of", "source", "offsets", "counts")):
        assert np.array_equal(g.cpu().numpy(), w), name


@pytest.mark.parametrize("kind", ["all dropped", "one expert", "out of range", "large int64"])
def test_sort_odd_ids(kind):
    ids = {"all dropped": np.full((600, 8), -1), "one expert": np.full((600, 8), 3),
           "out of range": random_ids(600, 8, 20, seed=1) - 4,
           "large int64": random_ids(600, 8, 8, seed=2) + (1 << 32)}[kind].astype(np.int64)
    dtype = torch.int64 if kind == "large int64" else torch.int32
    got = sort(ids, 8, 16, dtype=dtype)
    kept = np.where((ids >= 0) & (ids < 8), ids, -1)
    want = plain_sort(kept, 8, 16, got[1].shape[0])
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)


def test_sort_int64_and_larger_capacity():
    ids = random_ids(900, 6, 24, seed=3)
    got = sort(ids, 24, 16, capacity=9000, dtype=torch.int64)
    want = plain_sort(ids, 24, 16, 9000)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)


def test_sort_dropped_duplicates_of_a_token_keep_their_order():
    ids = np.zeros((3, 4), np.int64)  # every assignment of every token to expert 0
    row_of = sort(ids, 2, 16)[0].cpu().numpy()
    assert np.array_equal(row_of, np.arange(12).reshape(3, 4))


CASES = [(1, 1, 1, 8, 1), (8, 8, 64, 256, 16), (5, 3, 7, 1, 1), (100, 2, 8, 33, 16),
         (300, 4, 32, 512, 128), (257, 6, 16, 1001, 16), (40, 2, 4, 4096, 16), (64, 1, 200, 250, 1),
         (2500, 2, 8, 64, 16), (30, 12, 16, 2056, 16)]


def route(tokens, topk, experts, multiple, seed=5):
    ids = random_ids(tokens, topk, experts, seed)
    if tokens > 2:
        ids[tokens // 2] = -1  # a token without any row
    return sort(ids, experts, multiple)


@pytest.mark.parametrize("tokens, topk, experts, hidden, multiple", CASES)
@pytest.mark.parametrize("dtype", [BF, F])
def test_dispatch(tokens, topk, experts, hidden, multiple, dtype):
    row_of, source, _, _ = route(tokens, topk, experts, multiple)
    x = rnd(tokens, hidden, seed=6, dtype=dtype)
    src = source.long()
    want = torch.where((src >= 0)[:, None], x[src.clamp(min=0) // topk],
                       torch.zeros((), dtype=dtype, device="cuda"))
    rows = torch.full((source.shape[0], hidden), float("nan"), dtype=dtype, device="cuda")
    fp8.fp8_moe_dispatch(x, row_of, source, rows)
    assert torch.equal(rows, want)
    si, amax = torch.full((1,), 150.0, device="cuda"), torch.full((1,), 9e9, device="cuda")
    q = torch.full(rows.shape, 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    fp8.fp8_moe_dispatch(x, row_of, source, q, scale_inv=si, amax_out=amax)
    wq = (want.float() * 150.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8))
    assert amax.item() == x.float().abs().max().item()


def test_dispatch_strided_offset_rows():
    row_of, source, _, _ = route(90, 2, 8, 16)
    base = rnd(90, 200, seed=7, dtype=BF)
    src = source.long()
    for lo, w in ((0, 128), (1, 128), (8, 64), (3, 99)):
        x = base[:, lo:lo + w]
        rows = torch.empty(source.shape[0], w, dtype=BF, device="cuda")
        fp8.fp8_moe_dispatch(x, row_of, source, rows)
        want = torch.where((src >= 0)[:, None], x[src.clamp(min=0) // 2], torch.zeros_like(rows))
        assert torch.equal(rows, want)


def test_dispatch_cast_equals_the_quantiser():
    row_of, source, _, _ = route(64, 1, 4, 16)
    x = rnd(64, 256, seed=8, dtype=BF, scale=3.0)
    si, amax, q = (torch.full((1,), 77.0, device="cuda"), torch.empty(1, device="cuda"),
                   torch.empty(64, 256, dtype=torch.uint8, device="cuda"))
    fp8.fp8_quantize(x, fp8.DELAYED, None, si, q, amax)
    rows = torch.empty(source.shape[0], 256, dtype=torch.uint8, device="cuda")
    fp8.fp8_moe_dispatch(x, row_of, source, rows, scale_inv=si)
    live = source >= 0
    assert torch.equal(rows[live], q[source[live].long()])


def gathered(rows, row_of):
    got = rows.double()[row_of.clamp(min=0).long()]
    return torch.where((row_of >= 0)[..., None], got, torch.zeros_like(got))


@pytest.mark.parametrize("tokens, topk, experts, hidden, multiple", CASES)
@pytest.mark.parametrize("dtype", [BF, F])
def test_combine_and_gradients(tokens, topk, experts, hidden, multiple, dtype):
    row_of, source, _, _ = route(tokens, topk, experts, multiple)
    cap = source.shape[0]
    rows = rnd(cap, hidden, seed=9, dtype=dtype)
    w = rnd(tokens, topk, seed=10)
    y = torch.full((tokens, hidden), float("nan"), dtype=dtype, device="cuda")
    terms = gathered(rows, row_of) * w.double()[..., None]
    for weights, t in ((w, terms), (None, gathered(rows, row_of))):
        fp8.fp8_moe_combine(rows, row_of, weights, y)
        ref = t.sum(1)
        tol = (topk + 2) * U * t.abs().sum(1) + OUT[dtype] * ref.abs()
        assert ((y.double() - ref).abs() <= tol).all()
    dx = torch.empty_like(y)
    fp8.fp8_moe_dispatch_backward(rows, row_of, dx)
    assert torch.equal(dx, y)  # the same sum

    dy = rnd(tokens, hidden, seed=11, dtype=dtype)
    drows = torch.full((cap, hidden), float("nan"), dtype=dtype, device="cuda")
    dw = torch.full((tokens, topk), float("nan"), device="cuda")
    fp8.fp8_moe_combine_backward(dy, rows, row_of, source, w, drows, dw)
    src = source.clamp(min=0).long()
    want = dy.float()[src // topk] * w.reshape(-1)[src][:, None]  # one rounding each in fp32
    want = torch.where((source >= 0)[:, None], want, torch.zeros_like(want)).to(dtype)
    assert torch.equal(drows, want)
    t = gathered(rows, row_of) * dy.double()[:, None, :]
    tol = (hidden / 32 + 34) * U * t.abs().sum(2)
    assert ((dw.double() - t.sum(2)).abs() <= tol).all()
    assert (dw[row_of < 0] == 0).all()
    drows2 = torch.empty_like(drows)
    fp8.fp8_moe_combine_backward(dy, rows, row_of, source, w, drows2)
    assert torch.equal(drows, drows2)


def test_combine_gradient_against_differences():
    """y is linear in rows and in the weights, so central differences in 64
    bits are exact to rounding; the fp32 results are within 1e-5."""
    row_of, source, _, _ = route(20, 3, 5, 16)
    cap, hidden = source.shape[0], 48
    rows, w, dy = rnd(cap, hidden, seed=12), rnd(20, 3, seed=13), rnd(20, hidden, seed=14)
    drows, dw = torch.empty_like(rows), torch.empty_like(w)
    fp8.fp8_moe_combine_backward(dy, rows, row_of, source, w, drows, dw)
    loss = lambda r, w: ((gathered(r, row_of) * w[..., None]).sum(1) * dy.double()).sum()  # noqa: E731
    r64, w64 = rows.double(), w.double()
    vr, vw = rnd(cap, hidden, seed=15).double(), rnd(20, 3, seed=16).double()
    for num, got in (((loss(r64 + vr, w64) - loss(r64 - vr, w64)) / 2, (drows.double() * vr)),
                     ((loss(r64, w64 + vw) - loss(r64, w64 - vw)) / 2, (dw.double() * vw))):
        assert abs(num.item() - got.sum().item()) <= 1e-5 * got.abs().sum().item()


def test_nothing_of_a_dropped_row_is_read():
    # rows without a source hold NaN; a dropped weight is NaN too
    row_of, source, _, _ = route(50, 2, 8, 16)
    rows = rnd(source.shape[0], 72, seed=17)
    rows[source < 0] = float("nan")
    w = rnd(50, 2, seed=18)
    w[row_of < 0] = float("nan")
    y, dw = torch.empty(50, 72, device="cuda"), torch.empty(50, 2, device="cuda")
    drows = torch.empty_like(rows)
    fp8.fp8_moe_combine(rows, row_of, w, y)
    fp8.fp8_moe_combine_backward(y, rows, row_of, source, w, drows, dw)
    assert y.isfinite().all() and dw.isfinite().all() and drows.isfinite().all()
    assert (y[25] == 0).all()  # the token without any row


def test_indices_outside_the_rows_count_as_dropped():
    row_of = torch.tensor([[0, 99], [5, -3]], dtype=torch.int32, device="cuda")
    source = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    rows, y = rnd(4, 16, seed=19), torch.empty(2, 16, device="cuda")
    fp8.fp8_moe_combine(rows, row_of, None, y)
    assert torch.equal(y[0], rows[0]) and (y[1] == 0).all()
    out = torch.empty_like(rows)
    fp8.fp8_moe_dispatch(y, row_of, source, out)
    assert (out[1:] == 0).all()


def test_no_tokens():
    row_of, source, offsets, counts = sort(np.zeros((0, 2), np.int64), 4, 16, capacity=32)
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    rows = torch.full((32, 64), 5.0, dtype=BF, device="cuda")
    fp8.fp8_moe_dispatch(x, row_of, source, rows)
    assert (rows == 0).all() and (offsets == 0).all() and (counts == 0).all()
    fp8.fp8_moe_combine(rows, row_of, None, torch.empty_like(x))


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31: the last of 600000 rows of 4096."""
    hidden, cap = 4096, 600000
    row_of = torch.tensor([[cap - 1, 2]], dtype=torch.int32, device="cuda")
    source = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    source[cap - 1], source[2] = 0, 1
    x = rnd(1, hidden, seed=20, dtype=BF)
    rows = torch.full((cap, hidden), 3.0, dtype=BF, device="cuda")
    fp8.fp8_moe_dispatch(x, row_of, source, rows)
    assert torch.equal(rows[cap - 1], x[0]) and torch.equal(rows[2], x[0])
    assert not rows[3:cap - 1].any()
    y = torch.empty_like(x)
    fp8.fp8_moe_combine(rows, row_of, None, y)
    assert torch.equal(y, (2 * x.float()).to(BF))


def test_another_stream():
    s = torch.cuda.Stream()
    x = rnd(70, 96, seed=21, dtype=BF)
    ids = torch.from_numpy(random_ids(70, 2, 8, seed=22)).int().cuda()
    cap = fp8.fp8_moe_capacity(140, 8, 16)
    i32 = lambda *v: torch.empty(v, dtype=torch.int32, device="cuda")  # noqa: E731
    row_of, source, offsets, counts = i32(70, 2), i32(cap), i32(9), i32(8)
    rows, y = torch.empty(cap, 96, dtype=BF, device="cuda"), torch.empty_like(x)
    torch.cuda.synchronize()
    fp8.fp8_moe_sort(ids, 8, 16, row_of, source, offsets, counts, stream=s)
    fp8.fp8_moe_dispatch(x, row_of, source, rows, stream=s)
    fp8.fp8_moe_combine(rows, row_of, None, y, stream=s)
    s.synchronize()
    want = (x.float() * (row_of >= 0).sum(1, keepdim=True)).to(BF)
    assert torch.equal(y, want)


def test_python_refusals():
    row_of, source, _, _ = route(10, 2, 4, 16)
    x = rnd(10, 32, seed=23, dtype=BF)
    rows = torch.empty(source.shape[0], 32, dtype=BF, device="cuda")
    w = rnd(10, 2, seed=24)
    bad = [lambda: fp8.fp8_moe_dispatch(x, row_of[:5], source, rows),
           lambda: fp8.fp8_moe_dispatch(x, row_of.long(), source, rows),
           lambda: fp8.fp8_moe_dispatch(x, row_of, source, rows.float()),
           lambda: fp8.fp8_moe_dispatch(x, row_of, source, rows[:-1]),
           lambda: fp8.fp8_moe_dispatch(x.t(), row_of, source, rows),
           lambda: fp8.fp8_moe_combine(rows, row_of, w.bfloat16(), x),
           lambda: fp8.fp8_moe_combine(rows, row_of, w[:, :1], x),
           lambda: fp8.fp8_moe_combine(rows, row_of, w, x[:5]),
           lambda: fp8.fp8_moe_combine(rows, row_of, w, x.float()),
           lambda: fp8.fp8_moe_combine_backward(x[:, :8], rows, row_of, source, w, rows),
           lambda: fp8.fp8_moe_combine_backward(x, rows, row_of, None, w, rows),
           lambda: fp8.fp8_moe_dispatch_backward(rows, row_of, x.cpu())]
    for call in bad:
        with pytest.raises(fp8.Fp8Error):
            call()


# widths that 16-byte groups do not fit, with enough tokens that few threads
# share a row, and with few; one and two elements; every share of threads
@pytest.mark.parametrize("tokens, topk, experts, hidden, multiple", [
    (3000, 3, 5, 1, 1), (900, 2, 4, 2, 1), (2500, 2, 8, 65, 1), (2000, 6, 16, 333, 16),
    (1500, 8, 64, 2047, 1), (1300, 2, 4, 7001, 16), (40, 3, 4, 4097, 1), (1400, 9, 16, 515, 16)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_rows_of_odd_width(tokens, topk, experts, hidden, multiple, dtype):
    test_dispatch(tokens, topk, experts, hidden, multiple, dtype)
    test_combine_and_gradients(tokens, topk, experts, hidden, multiple, dtype)
