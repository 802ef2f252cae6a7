"""Orthogonalisation with operands of 22 bits (precise=True).

Tolerance.  A unit error e of a product is 2^-21 of its operands (two of 2^-22) and,
for the accumulator, 2^-23 for each 16 of a contraction of up to L = max(rows,
cols).  As with 11-bit operands, some twelve products' errors reach the result
through slopes of up to 3.4; here they may add up: 41 e (2-norm).  Beyond that the
result is the formula's, rounded once to bf16: its distance is at most that
rounding's own plus 41 e, single entries 16 times that plus half a unit.  An
entry goes to another bf16 value when the middle of two lies within its error:
of normal entries 444 times the error, 6 % at L = 384 (a third of them with 11
bits).
"""
import pytest
import torch

import scaled_linear_layers_gb300 as fp8
from test_gpu_orthogonalize import ABC, BF, EPS, F, by_products, by_singular_values, rnd

pytestmark = pytest.mark.gpu


def run(g, steps=5, coefficients=ABC, **k):
    batch = g.shape[0] if g.dim() == 3 else 1
    out = torch.full(g.shape, float("nan"), dtype=BF, device="cuda")
    n = fp8.fp8_orthogonalize_workspace_bytes(batch, *g.shape[-2:], precise=True)
    # NaN in every byte of the workspace: nothing may be read before it is written
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    fp8.fp8_orthogonalize(g, out, ws, steps=steps, coefficients=coefficients, precise=True, **k)
    fp8.fp8_check_device_status()
    return out


def error(g):
    return 41 * (2.0 ** -21 + max(g.shape[-2:]) / 16 * 2.0 ** -23)


def check(g, out, ref):
    rounded, delta, rms = ref.to(BF).double(), error(g), ref.square().mean().sqrt()
    d = out.double() - ref
    assert torch.isfinite(d).all()
    assert d.norm() <= (rounded - ref).norm() + delta * ref.norm()
    assert (d.abs() <= 2.0 ** -8 * ref.abs() + 16 * delta * rms).all()


@pytest.mark.parametrize("rows, cols", [
    (1, 1), (1, 50), (50, 1), (2, 3), (8, 8), (33, 97), (97, 33), (64, 64), (100, 333), (128, 128),
    (130, 129), (127, 500), (257, 511), (511, 257), (300, 64), (513, 520)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_one_matrix(rows, cols, dtype):
    g = rnd(rows, cols, seed=rows * 7 + cols, dtype=dtype, scale=1e-3)
    check(g, run(g), by_singular_values(g, [ABC] * 5))


@pytest.mark.parametrize("batch, rows, cols", [(5, 100, 77), (40, 96, 200), (3, 257, 2049),
                                               (20, 50, 1500)])
def test_batch(batch, rows, cols):
    g = rnd(batch, rows, cols, seed=batch, dtype=BF)
    g *= torch.logspace(-4, 4, batch, device="cuda")[:, None, None].to(BF)  # own norms
    out, ref = run(g), by_products(g, [ABC] * 5)
    for z in range(batch):
        check(g, out[z], ref[z])


# tiles of 256 and of 128, more than one wave, split contractions, both ways round
@pytest.mark.parametrize("rows, cols", [(1024, 1024), (2000, 1100), (1100, 2307), (4096, 512),
                                        (128, 8000), (8191, 130), (2999, 3201)])
def test_large(rows, cols):
    g = rnd(rows, cols, seed=3, dtype=BF)
    out = run(g)
    check(g, out, by_products(g, [ABC] * 5))
    assert torch.equal(out, run(g))


@pytest.mark.parametrize("rows, cols", [(256, 384), (384, 256)])
def test_entries_are_the_rounded_formula(rows, cols):
    g = rnd(rows, cols, seed=4)
    assert (run(g) != by_products(g, [ABC] * 5).to(BF)).double().mean() <= 0.06


def in_32_bits(g, coefficients):
    x = g / (g.square().sum().sqrt() + EPS)
    for a, b, c in coefficients:
        m = x @ x.mT
        x = a * x + (b * m + c * (m @ m)) @ x
    return x


# On [1e-3, 1], then on the range of values of the step before, the odd quintic with
# the least largest distance from 1: the ends of the ranges are where its slope is
# largest, 26 in the first step.
EDGE = [(8.470329, -25.108078, 18.629279), (4.182834, -3.108701, 0.580607),
        (3.961856, -2.954063, 0.562976), (3.286584, -2.464719, 0.507358),
        (2.273748, -1.644659, 0.416191), (1.888716, -1.265157, 0.376519)]


@pytest.mark.parametrize("safety", [1.0, 1.01])
@pytest.mark.parametrize("noise", [1e-2, 1e-3, 1e-4])
def test_a_singular_value_where_the_slope_is_largest(safety, noise):
    """A nearly rank-one matrix's is at the end of the first range, and roundings
    grow by the product of the slopes.  Units of 2^-22 against 2^-24: at most four
    times as far from the rounded formula as 32-bit products are (11 bits: 19 times
    at a noise of 1e-4)."""
    g = rnd(256, 1, seed=5) @ rnd(1, 384, seed=6) + noise * rnd(256, 384, seed=7)
    coefficients = [(a / safety, b / safety ** 3, c / safety ** 5) for a, b, c in EDGE]
    want = by_products(g, coefficients).to(BF).double()
    far = (in_32_bits(g, coefficients).to(BF).double() - want).norm()
    near = (run(g, steps=6, coefficients=coefficients).double() - want).norm()
    assert near <= 4 * far + 1e-4 * want.norm()


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 8])
def test_steps_and_scale(steps):
    g = rnd(96, 160, seed=11)
    check(g, run(g, steps=steps, scale=0.3), by_singular_values(g, [ABC] * steps, scale=0.3))


@pytest.mark.parametrize("scale", [6e37, 1e-42])
def test_entries_at_the_ends_of_fp32(scale):
    g = rnd(64, 81, seed=13, scale=scale)
    check(g, run(g, eps=0.0), by_singular_values(g, [ABC] * 5, eps=0.0))


def test_zero_matrix_is_zero_and_nan_stays_in_its_matrix():
    g = rnd(4, 48, 56, seed=14)
    g[1] = 0
    g[2, 5, 6] = float("nan")
    out, ref = run(g), by_singular_values(g[[0, 3]], [ABC] * 5)
    check(g, out[0], ref[0])
    check(g, out[3], ref[1])
    assert (out[1] == 0).all() and out[2].isnan().any()


def test_strided_input_and_odd_output_address():
    base = rnd(3, 70, 200, seed=15, dtype=BF)
    for g in (base[:, 4:60, 8:136], base[1, :, 3:], base[:1].expand(2, 70, 200)):
        check(g, run(g), by_singular_values(g, [ABC] * 5))
    g = rnd(40, 64, seed=16)
    store = torch.zeros(40 * 64 + 2, dtype=BF, device="cuda")
    out = store[1:-1].view(40, 64)
    n = fp8.fp8_orthogonalize_workspace_bytes(1, 40, 64, precise=True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    fp8.fp8_orthogonalize(g, out, ws, precise=True)
    check(g, out, by_singular_values(g, [ABC] * 5))
    assert store[0] == 0 and store[-1] == 0


def test_two_streams_and_a_graph():
    gs = [rnd(700, 900, seed=20 + i, dtype=BF) for i in range(2)]
    outs = [torch.empty_like(g) for g in gs]
    n = fp8.fp8_orthogonalize_workspace_bytes(1, 700, 900, precise=True)
    wss = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    torch.cuda.synchronize()
    for g, out, ws, s in zip(gs, outs, wss, streams):
        fp8.fp8_orthogonalize(g, out, ws, stream=s, precise=True)
    torch.cuda.synchronize()
    for g, out in zip(gs, outs):
        check(g, out, by_products(g, [ABC] * 5))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.fp8_orthogonalize(gs[0], outs[1], wss[0], precise=True)
    outs[1].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])


def test_a_workspace_of_the_other_form_is_refused():
    g = rnd(256, 256, seed=18)
    out = torch.empty(256, 256, dtype=BF, device="cuda")
    ws = torch.empty(fp8.fp8_orthogonalize_workspace_bytes(1, 256, 256), dtype=torch.uint8,
                     device="cuda")
    with pytest.raises(fp8.Fp8Error) as e:
        fp8.fp8_orthogonalize(g, out, ws, precise=True)
    assert e.value.status == 2  # FP8_ERR_SHAPE


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    g = rnd(600, 700, seed=19, dtype=BF)
    out = torch.empty_like(g)
    ws = torch.empty(fp8.fp8_orthogonalize_workspace_bytes(1, 600, 700, precise=True),
                     dtype=torch.uint8, device="cuda")
    fp8.fp8_check_device_status()
    old = fp8.fp8_set_wait_limit_ns(1)
    try:
        fp8.fp8_orthogonalize(g, out, ws, precise=True)
        with pytest.raises(fp8.Fp8Error) as e:
            fp8.fp8_check_device_status()
        assert e.value.status == 6  # FP8_ERR_TIMEOUT
    finally:
        fp8.fp8_set_wait_limit_ns(old)
    check(g, run(g), by_products(g, [ABC] * 5))
