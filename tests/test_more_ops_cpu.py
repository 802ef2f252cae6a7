"""Host-side argument checks of the router, the experts' linears and the gated
activation: every rejection happens before the device is touched, so these run
on a CPU-only machine (the fake addresses are never dereferenced)."""
import pytest
import torch

import __graft_entry__

OK, NULL, SHAPE, ALIGN, UNSUPPORTED = 0, 1, 2, 3, 4
A, ODD = 0x10000, 0x10001  # aligned, misaligned
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    from scaled_linear_layers_gb300 import _lib
    return _lib.load()


def route(lib, logits=A, ldl=64, lt=BF16, mask=None, tokens=4, experts=64, topk=8, renorm=1, ids=A,
          weights=A, counts=A, live=A, losses=A, ws=A):
    return lib.fp8_moe_route(logits, ldl, lt, mask, tokens, experts, topk, renorm, ids, weights,
                             counts, live, losses, ws, None)


@pytest.mark.parametrize("kw, status", [
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL),
    (dict(counts=None), NULL), (dict(live=None), NULL), (dict(ws=None), NULL),
    (dict(lt=2), SHAPE), (dict(tokens=-1), SHAPE), (dict(experts=0), SHAPE), (dict(topk=0), SHAPE),
    (dict(topk=65), SHAPE), (dict(ldl=-1), SHAPE), (dict(tokens=1 << 29), SHAPE),
    (dict(experts=1025), UNSUPPORTED), (dict(topk=33), UNSUPPORTED),
    (dict(logits=ODD), ALIGN), (dict(logits=A + 2, lt=F32), ALIGN), (dict(ids=A + 2), ALIGN),
    (dict(weights=A + 1), ALIGN), (dict(counts=A + 2), ALIGN), (dict(live=A + 2), ALIGN),
    (dict(losses=A + 2), ALIGN), (dict(ws=A + 2), ALIGN),
])
def test_route_refusals(lib, kw, status):
    assert route(lib, **kw) == status
    assert "fp8_moe_route" in lib.fp8_last_error().decode()


def route_bwd(lib, logits=A, ldl=64, lt=BF16, tokens=4, experts=64, topk=8, ids=A, counts=A, live=A,
              dw=A, dlosses=A, dlogits=A):
    return lib.fp8_moe_route_backward(logits, ldl, lt, tokens, experts, topk, 1, ids, counts, live,
                                      dw, dlosses, dlogits, None)


@pytest.mark.parametrize("kw, status", [
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(dlogits=None), NULL),
    (dict(counts=None), NULL), (dict(live=None), NULL), (dict(topk=65), SHAPE),
    (dict(lt=-1), SHAPE), (dict(experts=2000), UNSUPPORTED), (dict(dlogits=ODD), ALIGN),
    (dict(dw=A + 2), ALIGN), (dict(dlosses=A + 1), ALIGN),
])
def test_route_backward_refusals(lib, kw, status):
    assert route_bwd(lib, **kw) == status


def test_route_workspace(lib):
    f = lib.fp8_moe_route_workspace_bytes
    assert f(-1, 8) == f(4, 0) == f(4, 1025) == 0
    assert 0 < f(0, 8) <= f(1, 8) <= f(1 << 20, 8) <= 512 * 2 * 9 * 4


def linear(lib, which, a=A, sa=A, b=A, sb=A, offsets=A, experts=4, capacity=512, N=256, K=384, d=A):
    return getattr(lib, f"fp8_moe_linear_{which}")(a, sa, b, sb, offsets, experts, capacity, N, K, d,
                                                   None)


@pytest.mark.parametrize("which", ["fprop", "dgrad", "wgrad"])
@pytest.mark.parametrize("kw, status", [
    (dict(a=None), NULL), (dict(sa=None), NULL), (dict(b=None), NULL), (dict(sb=None), NULL),
    (dict(offsets=None), NULL), (dict(d=None), NULL), (dict(experts=0), SHAPE),
    (dict(capacity=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=-128), SHAPE),
    (dict(capacity=1 << 31), SHAPE), (dict(experts=1024, N=1 << 21), SHAPE),
    (dict(experts=1025), UNSUPPORTED), (dict(N=192), ALIGN), (dict(K=64), ALIGN),
    (dict(a=A + 8), ALIGN), (dict(sa=A + 4), ALIGN), (dict(b=ODD), ALIGN), (dict(sb=A + 8), ALIGN),
    (dict(offsets=A + 2), ALIGN), (dict(d=A + 8), ALIGN),
])
def test_moe_linear_refusals(lib, which, kw, status):
    assert linear(lib, which, **kw) == status
    assert f"fp8_moe_linear_{which}" in lib.fp8_last_error().decode()


def test_moe_wgrad_takes_whole_blocks_of_rows(lib):
    assert linear(lib, "wgrad", capacity=500) == ALIGN


def swiglu(lib, h=A, ldh=256, ht=BF16, rows=4, cols=128, live=None, y=A, yq=None, ys=None, hq=None,
           hs=None):
    return lib.fp8_swiglu(h, ldh, ht, rows, cols, live, y, yq, ys, hq, hs, None)


@pytest.mark.parametrize("kw, status", [
    (dict(h=None), NULL), (dict(y=None), NULL), (dict(yq=A), NULL), (dict(hq=A), NULL),
    (dict(ht=3), SHAPE), (dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE), (dict(cols=1 << 30), SHAPE),
    (dict(ldh=-1), SHAPE), (dict(h=ODD), ALIGN), (dict(ht=F32, y=A + 2), ALIGN),
    (dict(yq=A, ys=A + 2), ALIGN), (dict(hq=A, hs=A + 1), ALIGN), (dict(live=A + 2), ALIGN),
])
def test_swiglu_refusals(lib, kw, status):
    assert swiglu(lib, **kw) == status
    assert "fp8_swiglu" in lib.fp8_last_error().decode()


def swiglu_bwd(lib, dy=A, lddy=128, t=BF16, h=A, ldh=256, hs=None, rows=4, cols=128, live=None, dh=A,
               y=None):
    return lib.fp8_swiglu_backward(dy, lddy, t, h, ldh, hs, rows, cols, live, dh, y, None)


@pytest.mark.parametrize("kw, status", [
    (dict(dy=None), NULL), (dict(h=None), NULL), (dict(dh=None), NULL), (dict(t=2), SHAPE),
    (dict(lddy=-1), SHAPE), (dict(ldh=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(dy=ODD), ALIGN),
    (dict(h=ODD), ALIGN), (dict(dh=ODD), ALIGN), (dict(y=ODD), ALIGN), (dict(hs=A + 2), ALIGN),
])
def test_swiglu_backward_refusals(lib, kw, status):
    assert swiglu_bwd(lib, **kw) == status


def test_python_checks_refuse_host_tensors_and_odd_halves():
    import scaled_linear_layers_gb300 as fp8
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    q = torch.zeros(128, 128, dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: fp8.fp8_moe_route(x, x.int(), x, x, x, None, None),
                 lambda: fp8.fp8_moe_route_backward(x, x.int(), x, x, x),
                 lambda: fp8.fp8_moe_linear_fprop(q, q, q, q, off, q),
                 lambda: fp8.fp8_moe_linear_dgrad(q, q, q, q, off, q),
                 lambda: fp8.fp8_moe_linear_wgrad(q, q, q, q, off, q),
                 lambda: fp8.fp8_moe_linear_fprop(q, q, q, q, x, q),
                 lambda: fp8.fp8_swiglu(x, x),
                 lambda: fp8.fp8_swiglu_backward(x, x, x)):
        with pytest.raises(fp8.Fp8Error):
            call()
