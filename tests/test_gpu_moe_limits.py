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
