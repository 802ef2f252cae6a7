"""Orthogonalisation at the ends of its range: coefficients and singular values
whose polynomial is large, few steps, entries near the ends of fp32."""
import pytest
import torch

from test_gpu_orthogonalize import ABC, by_products, by_singular_values, check, rnd, run

pytestmark = pytest.mark.gpu


# |b s^2 + c s^4|, plus a where the step multiplies by (a I + B), is the largest
# entry of the matrix that a step multiplies X by.  Singular values equal to one
# another leave no cancellation: the largest error is the rounding of the operands,
# 2e-4 (2-norm) each, through the slope of the polynomial, 2.2 relative at s = 3.5
# (t (b + 2 c t) / (a + b t + c t^2) at t = 12.25); the bound of 5e-3 stays.
@pytest.mark.parametrize("n, coefficients", [
    (64, [(28.0, 0.0, 0.0), ABC]),                     # s = 3.5: 250 in the last step
    (64, [(20.0, 0.0, 0.0), ABC]),                     # s = 2.5: 53
    (1024, [(100.0, 0.0, 0.0), (0.5, 0.0, 0.0)]),      # 100 on the diagonal
    (1024, [(-28.0, 131072.0, 0.0)] + [(0.5, 0.0, 0.0)] * 3),  # 128 in an early step
    (1024, [(1.0, 0.0, 0.0)] * 3 + [(100.0, 0.0, 0.0), (0.5, 0.0, 0.0)]),  # 100 in a late one
])
def test_polynomials_of_large_values(n, coefficients):
    q = torch.linalg.qr(rnd(n, n, seed=31).double().cpu())[0].float().contiguous().cuda()
    out = run(q, steps=len(coefficients), coefficients=coefficients)
    check(out, by_products(q, coefficients))


@pytest.mark.parametrize("scale", [6e37, 1e-42])
@pytest.mark.parametrize("cols", [80, 81])
def test_entries_at_the_ends_of_fp32(scale, cols):
    g = rnd(64, cols, seed=32, scale=scale)
    assert g.isfinite().all() and g.count_nonzero() > 0.9 * g.numel()
    check(run(g, eps=0.0), by_singular_values(g, [ABC] * 5, eps=0.0))


@pytest.mark.parametrize("steps", [1, 2, 3])
@pytest.mark.parametrize("scale", [1.0, 0.3])
def test_few_steps_keep_the_input_to_its_own_rounding(steps, scale):
    """With (1, 0, 0) the result is X itself.  Held to 22 bits and rounded once
    to bf16's 8, it differs from the 64-bit X's rounding where X lies within 2^-22
    of the middle of two values 2^-8 apart, one entry in 2^13; 11 bits differ in
    one of 30."""
    g = rnd(96, 160, seed=33)
    out = run(g, steps=steps, coefficients=[(1.0, 0.0, 0.0)] * steps, scale=scale)
    want = (scale * by_products(g, [(1.0, 0.0, 0.0)] * steps)).to(torch.bfloat16)
    assert (out != want).double().mean().item() <= 0.005


def test_a_batch_of_many_small_matrices():
    """More matrices than one launch of the scaling takes, with few parts each."""
    g = rnd(70000, 5, 3, seed=34)
    out = run(g)
    ref = by_products(g, [ABC] * 5)
    check(out, ref)
    check(out[-1], ref[-1])


# The first steps' errors grow with the slopes of the later ones: 2.4e-3 to 2.9e-3
# (2-norm) in these cases besides the output's 1.7e-3, together 3.4e-3; 5e-3 as for
# the others.
@pytest.mark.parametrize("rank", [1, 2, 8])
@pytest.mark.parametrize("noise", [1e-3, 1e-4])
@pytest.mark.parametrize("coefficients", ["usual", "own interval a step"])
def test_nearly_low_rank(rank, noise, coefficients):
    g = rnd(256, rank, seed=35) @ rnd(rank, 384, seed=36) / rank ** 0.5
    g += noise * rnd(256, 384, seed=37)
    triples = [ABC] * 5
    if coefficients != "usual":
        # the odd quintics nearest to 1 on [1e-3, 1] and the ranges after it, with
        # 1 % between the largest singular value and the end
        triples = [(a / 1.01, b / 1.01 ** 3, c / 1.01 ** 5) for a, b, c in (
            (8.470329, -25.108078, 18.629279), (4.182834, -3.108701, 0.580607),
            (3.961856, -2.954063, 0.562976), (3.286584, -2.464719, 0.507358),
            (2.273748, -1.644659, 0.416191), (1.888716, -1.265157, 0.376519))]
    check(run(g, steps=len(triples), coefficients=triples), by_products(g, triples))


@pytest.mark.parametrize("steps", [8, 10])
def test_many_steps(steps):
    g = rnd(256, 384, seed=38)
    check(run(g, steps=steps), by_products(g, [ABC] * steps))
