"""The experts' linears when a copy never arrives: the wait for it runs out, the
products and copies in flight are settled, the status says so, and the next call
is right."""
import pytest
import torch

import scaled_linear_layers_gb300 as fp8
from scaled_linear_layers_gb300 import _lib

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
B = 128
LIMIT_NS = 1_000_000


def lose_a_call(call):
    """`call` with copies left out; its time on the device in ms."""
    lib = _lib.load()
    fp8.fp8_check_device_status()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    old = fp8.fp8_set_wait_limit_ns(LIMIT_NS)
    try:
        assert lib.fp8_inject_lost_copies(1) == 0
        begin.record()
        call()
        end.record()
        with pytest.raises(fp8.Fp8Error) as e:
            fp8.fp8_check_device_status()
        assert e.value.status == 6  # FP8_ERR_TIMEOUT
    finally:
        lib.fp8_inject_lost_copies(0)
        fp8.fp8_set_wait_limit_ns(old)
    return begin.elapsed_time(end)


def bytes_of(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 120, shape, generator=g, dtype=torch.uint8, device="cuda")


def scales(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(shape, generator=g, device="cuda")


# enough tiles for every block to have several, contractions of three hand-offs
# and more: of 128 elements, or of 512 where there are few rows
COUNTS, N, K = [600, 0, 300, 129, 1, 1400], 2560, 2048


def products(which, env, monkeypatch):
    """The call, and its output."""
    if env is not None:
        monkeypatch.setenv("FP8LINEAR_MOE_FEW", env)
    e, at = len(COUNTS), [0]
    for n in COUNTS:
        at.append(at[-1] + -(-n // B) * B)
    cap, offsets = at[-1], torch.tensor(at, dtype=torch.int32, device="cuda")
    if which == "wgrad":
        out = torch.empty(e, N, K, dtype=BF, device="cuda")
        args = (bytes_of(N, cap, seed=1), scales(cap // B, N, seed=2), bytes_of(K, cap, seed=3),
                scales(cap // B, K, seed=4), offsets, out)
    else:
        wide, cols = (K, N) if which == "fprop" else (N, K)
        out = torch.zeros(cap, cols, dtype=BF, device="cuda")
        w = bytes_of(e, N, K, seed=5) if which == "fprop" else bytes_of(K, e * N, seed=5)
        args = (bytes_of(cap, wide, seed=6), scales(cap, wide // B, seed=7), w,
                scales(e, N // B, K // B, seed=8), offsets, out)
    return (lambda: getattr(fp8, f"fp8_moe_linear_{which}")(*args)), out


KINDS = [("fprop", "0"), ("fprop", "1"), ("dgrad", "0"), ("dgrad", "1"), ("wgrad", None)]


@pytest.mark.parametrize("which, few", KINDS)
def test_a_copy_that_never_arrives_is_reported(which, few, monkeypatch):
    call, out = products(which, few, monkeypatch)
    call()
    fp8.fp8_check_device_status()
    want = out.clone()
    for _ in range(2):
        lose_a_call(call)
        out.zero_()
        call()
        fp8.fp8_check_device_status()
        assert torch.equal(out, want)


@pytest.mark.parametrize("which, few", KINDS)
def test_a_lost_copy_is_reported_soon(which, few, monkeypatch):
    """A wait ends within two polls (1 ms each) of its limit of 1 ms, and the last
    wait for the copy that is lost after 10 ms more; 64 polls between two looks at
    the clock took 62 ms and more."""
    call, _ = products(which, few, monkeypatch)
    call()
    assert lose_a_call(call) < 40
