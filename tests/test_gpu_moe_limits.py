"""Expert rows at the ends of their arguments' ranges."""
import pytest
import torch

import scaled_linear_layers_gb300 as fp8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden", [64, 33])
def test_amax_of_tokens_without_rows(hidden):
    """max |x| is over all tokens, whatever becomes of them: also without a row
    to write."""
    x = torch.randn(9, hidden, device="cuda").bfloat16()
    row_of = torch.full((9, 2), -1, dtype=torch.int32, device="cuda")
    for capacity in (0, 4):
        source = torch.full((capacity,), -1, dtype=torch.int32, device="cuda")
        rows = torch.empty(capacity, hidden, dtype=torch.uint8, device="cuda")
        amax = torch.full((1,), 9e9, device="cuda")
        fp8.fp8_moe_dispatch(x, row_of, source, rows, scale_inv=torch.ones(1, device="cuda"),
                             amax_out=amax)
        assert amax.item() == x.float().abs().max().item()
        assert (rows == 0).all()


@pytest.mark.slow
def test_a_segment_that_ends_at_the_last_row():
    """Padding up to row 2^31 - 2, the last that a place of 32 bits reaches."""
    capacity = 2 ** 31 - 1
    i32 = lambda *s: torch.full(s, 7, dtype=torch.int32, device="cuda")  # noqa: E731
    row_of, source, offsets, counts = i32(3, 1), i32(capacity), i32(2), i32(1)
    ids = torch.tensor([[0], [-1], [0]], dtype=torch.int32, device="cuda")
    fp8.fp8_moe_sort(ids, 1, capacity - 2, row_of, source, offsets, counts)
    torch.cuda.synchronize()
    assert row_of.flatten().tolist() == [0, -1, 1] and source[:2].tolist() == [0, 2]
    assert offsets.tolist() == [0, capacity - 2] and counts.tolist() == [2]
    assert all((part == -1).all() for part in source[2:].split(2 ** 28))
