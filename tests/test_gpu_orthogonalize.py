"""Newton-Schulz orthogonalisation against its formula in 64 bits, by way of
the singular values: U p(p(...p(sigma))) Vᵀ.

Tolerance.  A unit of bf16 is 2^-7 to 2^-8 of the value, so rounding a result
is 0.74 * 2^-7/sqrt(12) = 1.7e-3 in the 2-norm; of fp16, 0.74 * 2^-10/sqrt(12) = 2e-4;
four operands a step reach the result, each through the polynomial's slope (up
to 3.4 where the singular values still grow, around 1 after that), of which the
last two or three steps count: sqrt(12) * 2e-4 * 3.4 = 2.4e-3.  Together 2.9e-3;
5e-3 leaves room for small matrices, whose few entries average less.  Single
entries: 16 times that, in units of the root mean square.
"""
import pytest
import torch

import scaled_linear_layers_gb300 as fp8

pytestmark = pytest.mark.gpu
ABC = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
BF, F = torch.bfloat16, torch.float32


def rnd(*shape, seed, dtype=F, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def by_singular_values(g, coefficients, eps=EPS, scale=1.0):
    g = g.double().cpu()
    u, s, v = torch.linalg.svd(g, full_matrices=False)
    s = s / (s.square().sum(-1, keepdim=True).sqrt() + eps)
    for a, b, c in coefficients:
        s = a * s + b * s ** 3 + c * s ** 5
    return (scale * (u * s.unsqueeze(-2)) @ v).cuda()


def by_products(g, coefficients, eps=EPS):
    x = g.double()
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + eps)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    for a, b, c in coefficients:
        m = x @ x.mT
        x = a * x + b * (m @ x) + c * (m @ (m @ x))
    return x.mT if tall else x


def run(g, steps=5, coefficients=ABC, **k):
    batch = g.shape[0] if g.dim() == 3 else 1
    out = torch.full(g.shape, float("nan"), dtype=BF, device="cuda")
    n = fp8.fp8_orthogonalize_workspace_bytes(batch, *g.shape[-2:])
    # NaN in every byte of the workspace: nothing may be read before it is written
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    fp8.fp8_orthogonalize(g, out, ws, steps=steps, coefficients=coefficients, **k)
    fp8.fp8_check_device_status()
    return out


def check(out, ref, tol=5e-3):
    d = out.double() - ref
    assert torch.isfinite(d).all()
    assert (d.norm() / ref.norm()).item() <= tol
    rms = ref.square().mean().sqrt()
    assert (d.abs().max() / rms).item() <= 16 * tol


SHAPES = [(1, 1), (1, 50), (50, 1), (2, 3), (8, 8), (16, 40), (33, 97), (97, 33), (64, 64),
          (100, 333), (128, 128), (130, 129), (127, 500), (256, 256), (257, 511), (511, 257),
          (300, 64), (513, 520)]


@pytest.mark.parametrize("rows, cols", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F])
def test_one_matrix(rows, cols, dtype):
    g = rnd(rows, cols, seed=rows * 7 + cols, dtype=dtype, scale=1e-3)
    check(run(g), by_singular_values(g, [ABC] * 5))


@pytest.mark.parametrize("batch, rows, cols", [(2, 64, 64), (5, 100, 77), (3, 300, 130),
                                               (40, 96, 200), (8, 16, 16)])
def test_batch(batch, rows, cols):
    g = rnd(batch, rows, cols, seed=batch, dtype=BF)
    g *= torch.logspace(-4, 4, batch, device="cuda")[:, None, None].to(BF)  # own norms
    out, ref = run(g), by_singular_values(g, [ABC] * 5)
    for z in range(batch):
        check(out[z], ref[z])


@pytest.mark.parametrize("rows, cols", [(1024, 1024), (2000, 1100), (1100, 2307), (4096, 512),
                                        (640, 6000)])
def test_large(rows, cols):
    g = rnd(rows, cols, seed=3, dtype=BF)
    check(run(g), by_products(g, [ABC] * 5))


def test_many_tiles_of_both_kinds():
    # 3000 x 3200: 78 tiles of 256 on and below the diagonal, more than one
    # wave of pairs; rows, columns and the contraction all end inside a tile
    g = rnd(2999, 3201, seed=4)
    check(run(g), by_products(g, [ABC] * 5))


@pytest.mark.parametrize("batch, rows, cols", [
    (1, 64, 1024), (1, 100, 8000), (1, 8191, 130), (1, 128, 1100), (1, 200, 5001), (3, 257, 2049),
    (2, 3000, 300), (1, 640, 4097), (20, 50, 1500)])
def test_few_tiles_and_a_long_contraction(batch, rows, cols):
    """A's contraction is split over CTAs and its parts are added in order."""
    g = rnd(batch, rows, cols, seed=21, dtype=BF)
    out = run(g)
    check(out, by_products(g, [ABC] * 5))
    assert torch.equal(out, run(g))


@pytest.mark.parametrize("kind", ["low rank", "decay", "outlier"])
def test_spectra(kind):
    """Small singular values beside large ones, which the first steps raise."""
    m, n = 384, 512
    if kind == "low rank":
        g = rnd(m, 8, seed=5) @ rnd(8, n, seed=6) * 0.35 + 0.05 * rnd(m, n, seed=7)
    elif kind == "decay":
        u, v = torch.linalg.qr(rnd(m, m, seed=8))[0], torch.linalg.qr(rnd(n, m, seed=9))[0]
        g = (u / torch.arange(1, m + 1, device="cuda")) @ v.mT
    else:
        g = 0.01 * rnd(m, n, seed=10)
        g[17, 200] = 5.0
    check(run(g), by_singular_values(g, [ABC] * 5))


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_steps(steps):
    g = rnd(96, 160, seed=11)
    check(run(g, steps=steps), by_singular_values(g, [ABC] * steps))


def test_other_coefficients_each_step_and_scale():
    g = rnd(90, 200, seed=12)
    triples = [(3.4445, -4.7750, 2.0315), (2.5, -2.5, 1.0), (1.875, -1.25, 0.375),
               (1.875, -1.25, 0.375)]
    check(run(g, steps=4, coefficients=triples, scale=0.3),
          by_singular_values(g, triples, scale=0.3))


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_any_magnitude(scale):
    g = rnd(64, 80, seed=13, scale=scale)
    check(run(g, eps=0.0), by_singular_values(g, [ABC] * 5, eps=0.0))


def test_zero_matrix_is_zero_and_nan_stays_in_its_matrix():
    g = rnd(4, 48, 56, seed=14)
    g[1] = 0
    g[2, 5, 6] = float("nan")
    out, ref = run(g), by_singular_values(g[[0, 3]], [ABC] * 5)
    check(out[0], ref[0])
    check(out[3], ref[1])
    assert (out[1] == 0).all() and out[2].isnan().any()


def test_strided_input():
    base = rnd(3, 70, 200, seed=15, dtype=BF)
    for g in (base[:, 4:60, 8:136], base[:, :, 1:100], base[1, :, 3:], base[:1].expand(2, 70, 200)):
        check(run(g), by_singular_values(g, [ABC] * 5))


def test_odd_output_address():
    g = rnd(40, 64, seed=16)
    store = torch.zeros(40 * 64 + 2, dtype=BF, device="cuda")
    out = store[1:-1].view(40, 64)
    ws = torch.empty(fp8.fp8_orthogonalize_workspace_bytes(1, 40, 64), dtype=torch.uint8,
                     device="cuda")
    fp8.fp8_orthogonalize(g, out, ws)
    check(out, by_singular_values(g, [ABC] * 5))
    assert store[0] == 0 and store[-1] == 0


def test_repeats_bit_for_bit_and_on_another_stream():
    g = rnd(700, 900, seed=17, dtype=BF)
    a, b = run(g), run(g)
    assert torch.equal(a, b)
    s = torch.cuda.Stream()
    out, ws = torch.empty_like(a), torch.empty(
        fp8.fp8_orthogonalize_workspace_bytes(1, 700, 900), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    fp8.fp8_orthogonalize(g, out, ws, stream=s)
    s.synchronize()
    assert torch.equal(a, out)


def test_empty():
    for shape in ((0, 5), (5, 0), (0, 4, 4)):
        g = torch.empty(shape, dtype=BF, device="cuda")
        fp8.fp8_orthogonalize(g, torch.empty_like(g), None)


def test_python_refusals():
    g = rnd(16, 32, seed=18)
    out = torch.empty(16, 32, dtype=BF, device="cuda")
    ws = torch.empty(fp8.fp8_orthogonalize_workspace_bytes(1, 16, 32), dtype=torch.uint8,
                     device="cuda")
    for bad in (lambda: fp8.fp8_orthogonalize(g.t(), out, ws),
                lambda: fp8.fp8_orthogonalize(g.half(), out, ws),
                lambda: fp8.fp8_orthogonalize(g, out.float(), ws),
                lambda: fp8.fp8_orthogonalize(g, out[:8], ws),
                lambda: fp8.fp8_orthogonalize(g, out, ws[:-1]),
                lambda: fp8.fp8_orthogonalize(g, out, None),
                lambda: fp8.fp8_orthogonalize(g, out, ws, steps=0),
                lambda: fp8.fp8_orthogonalize(g, out, ws, steps=3, coefficients=[ABC] * 2),
                lambda: fp8.fp8_orthogonalize(g[None, None], out, ws)):
        with pytest.raises(fp8.Fp8Error):
            bad()


@pytest.mark.parametrize("rows, cols", [(600, 700), (4096, 1024)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(rows, cols):
    """A limit of 1 ns makes every wait give up: for copies, for products, for
    other tiles.  The call ends, the status says so, the next call is right."""
    g = rnd(rows, cols, seed=19, dtype=BF)
    out = torch.empty_like(g)
    ws = torch.empty(fp8.fp8_orthogonalize_workspace_bytes(1, rows, cols), dtype=torch.uint8,
                     device="cuda")
    fp8.fp8_check_device_status()
    old = fp8.fp8_set_wait_limit_ns(1)
    try:
        fp8.fp8_orthogonalize(g, out, ws)
        with pytest.raises(fp8.Fp8Error) as e:
            fp8.fp8_check_device_status()
        assert e.value.status == 6  # FP8_ERR_TIMEOUT
    finally:
        fp8.fp8_set_wait_limit_ns(old)
    check(run(g), by_products(g, [ABC] * 5))


def test_two_streams_at_once():
    """Two calls that may overlap, each with its own workspace: their resident
    CTAs wait for one another within a call only."""
    gs = [rnd(1500, 1500, seed=20 + i, dtype=BF) for i in range(2)]
    outs = [torch.empty_like(g) for g in gs]
    n = fp8.fp8_orthogonalize_workspace_bytes(1, 1500, 1500)
    wss = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, out, ws, s in zip(gs, outs, wss, streams):
            fp8.fp8_orthogonalize(g, out, ws, stream=s)
    torch.cuda.synchronize()
    fp8.fp8_check_device_status()
    for g, out in zip(gs, outs):
        check(out, by_products(g, [ABC] * 5))
