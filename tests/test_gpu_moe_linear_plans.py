"""dgrad and wgrad of the experts' linears replayed from a graph with other
offsets, and beside the same calls on other streams: the bits of calls alone."""
import pytest
import torch

import scaled_linear_layers_gb300 as fp8

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
B, N, K, CAP, EXPERTS = 128, 384, 512, 1024, 4
TABLES = {"dgrad": [[0, 100, 200, 300, 1024], [0, 0, 0, 700, 700], [0, 1, 2, 3, 4]],
          "wgrad": [[0, 128, 256, 512, 1024], [0, 0, 0, 896, 896], [0, 0, 0, 0, 0]]}


def operands(which):
    g = torch.Generator(device="cuda").manual_seed(1)
    q = lambda *s: torch.randint(0, 120, s, generator=g, dtype=torch.uint8, device="cuda")  # noqa: E731
    f = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    if which == "dgrad":
        return (q(CAP, N), f(CAP, N // B), q(K, EXPERTS * N), f(EXPERTS, N // B, K // B)), (CAP, K)
    return (q(N, CAP), f(CAP // B, N), q(K, CAP), f(CAP // B, K)), (EXPERTS, N, K)


def offsets(at):
    return torch.tensor(at, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("which, few", [("dgrad", "0"), ("dgrad", "1"), ("wgrad", "0")])
def test_replayed_with_new_offsets_beside_other_streams(which, few, monkeypatch):
    monkeypatch.setenv("FP8LINEAR_MOE_FEW", few)
    args, shape = operands(which)
    run = getattr(fp8, f"fp8_moe_linear_{which}")

    def alone(at):
        out = torch.full(shape, 7.0, dtype=BF, device="cuda")
        run(*args, offsets(at), out)
        return out

    tables = TABLES[which]
    want = [alone(at) for at in tables]
    if which == "wgrad":
        assert (want[2] == 0).all() and (want[1][:2] == 0).all()
    else:
        assert (want[1][700:] == 7).all() and (want[2][4:] == 7).all()
    held, out = offsets(tables[0]), torch.empty(shape, dtype=BF, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out.fill_(7.0)
        run(*args, held, out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, w in enumerate(want):
        held.copy_(offsets(tables[i]))
        others = [[torch.full(shape, 7.0, dtype=BF, device="cuda") for _ in tables] for _ in streams]
        at = [offsets(t) for t in tables]
        torch.cuda.synchronize()
        for s, outs in zip(streams, others):
            for o, a in zip(outs, at):
                run(*args, a, o, stream=s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
        for outs in others:
            for o, v in zip(outs, want):
                assert torch.equal(o, v)
    fp8.fp8_check_device_status()
