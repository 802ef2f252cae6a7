"""The router over many blocks is two launches.  Whichever does not happen is
reported; what the first alone writes are ids and weights."""
import pytest
import torch

import scaled_linear_layers_gb300 as fp8
from scaled_linear_layers_gb300 import _lib
from test_gpu_moe_route import check, logits_of, plain, route

pytestmark = pytest.mark.gpu
TOKENS, EXPERTS, TOPK = 600, 24, 3


@pytest.mark.parametrize("after", [0, 1])
def test_a_launch_that_fails_is_reported(after):
    lib, x = _lib.load(), logits_of(TOKENS, EXPERTS, seed=70)
    want = route(x, TOPK)
    out = {k: torch.full_like(v, -7) for k, v in want.items()}
    ws = torch.empty(fp8.fp8_moe_route_workspace_bytes(TOKENS, EXPERTS), dtype=torch.uint8,
                     device="cuda")
    assert lib.fp8_inject_later_launch_failure(after) == 0
    try:
        with pytest.raises(fp8.Fp8Error) as e:
            fp8.fp8_moe_route(x, **out, workspace=ws)
        assert e.value.status == 5  # FP8_ERR_CUDA
    finally:
        lib.fp8_inject_launch_failures(0)
    for name, t in out.items():
        if after == 1 and name in ("ids", "weights"):
            assert torch.equal(t, want[name])
        else:
            assert (t == -7).all(), name
    check(route(x, TOPK), plain(x, TOPK), x)


def test_later_launch_failure_refusal():
    assert _lib.load().fp8_inject_later_launch_failure(-1) == 2  # FP8_ERR_SHAPE
