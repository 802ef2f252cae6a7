"""Host-side argument checks of the layer-norm, expert-row and orthogonalising
entry points: every rejection happens before the device is touched, so these
run on a CPU-only machine (the fake addresses are never dereferenced)."""
import ctypes

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


def norm(lib, x=A, ldx=64, xt=BF16, w=A, b=A, wt=BF16, rows=4, cols=64, eps=1e-5, y=A, yq=None,
         si=None, amax=None, mean=A, rstd=A):
    return lib.fp8_layer_norm(x, ldx, xt, w, b, wt, rows, cols, eps, y, yq, si, amax, mean, rstd,
                              None)


@pytest.mark.parametrize("kw, status", [
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(y=None, yq=A), NULL),
    (dict(xt=7), SHAPE), (dict(wt=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE),
    (dict(cols=1 << 31), SHAPE), (dict(ldx=-64), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(x=ODD), ALIGN), (dict(y=ODD), ALIGN),
    (dict(xt=F32, x=A + 2), ALIGN), (dict(w=ODD), ALIGN), (dict(mean=A + 2), ALIGN),
    (dict(amax=A + 1), ALIGN),
])
def test_layer_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status
    assert "fp8_layer_norm" in lib.fp8_last_error().decode()


def norm_bwd(lib, dy=A, x=A, xt=BF16, w=A, wt=F32, mean=A, rstd=A, rows=4, cols=64, dx=A, dw=A,
             db=A, ws=A, lddy=64, ldx=64):
    return lib.fp8_layer_norm_backward(dy, lddy, x, ldx, xt, w, wt, mean, rstd, rows, cols, dx, dw,
                                       db, ws, None)


@pytest.mark.parametrize("kw, status", [
    (dict(dy=None), NULL), (dict(mean=None), NULL), (dict(rstd=None), NULL),
    (dict(dx=None, dw=None, db=None), NULL), (dict(ws=None), NULL), (dict(ws=A + 8), ALIGN),
    (dict(rows=-2), SHAPE), (dict(lddy=-1), SHAPE), (dict(dw=A + 2), ALIGN), (dict(wt=2), SHAPE),
])
def test_layer_norm_backward_refusals(lib, kw, status):
    assert norm_bwd(lib, **kw) == status


def test_layer_norm_workspace(lib):
    f = lib.fp8_layer_norm_workspace_bytes
    assert f(0, 64) == 0 and f(4, 0) == 0 and f(-1, 4) == 0
    assert f(3, 100) == 2 * 3 * 100 * 4
    assert f(1 << 20, 100) == 2 * 512 * 100 * 4


def test_moe_capacity(lib):
    f = lib.fp8_moe_capacity
    assert f(0, 8, 16) == 0
    assert f(3, 8, 16) == 3 * 16          # three experts of one row each at most
    assert f(100, 8, 16) == 100 + 8 * 15
    assert f(100, 8, 1) == 100
    assert f(-1, 8, 1) == f(1, 0, 1) == f(1, 1, 0) == -1


def sort(lib, ids=A, n=64, experts=8, multiple=16, capacity=64 + 8 * 15, row_of=A, source=A,
         offsets=A, counts=A, ws=None, ids_64=0):
    return lib.fp8_moe_sort(ids, ids_64, n, experts, multiple, capacity, row_of, source, offsets,
                            counts, ws, None)


@pytest.mark.parametrize("kw, status", [
    (dict(ids=None), NULL), (dict(source=None), NULL), (dict(offsets=None), NULL),
    (dict(n=-1), SHAPE), (dict(experts=0), SHAPE), (dict(multiple=0), SHAPE),
    (dict(capacity=100), SHAPE), (dict(capacity=1 << 31), SHAPE),
    (dict(experts=1025, capacity=1 << 20), UNSUPPORTED),
    (dict(n=5000, capacity=1 << 20), NULL),  # a workspace is needed from 4097 assignments
    (dict(ids=A + 2), ALIGN), (dict(ids=A + 4, ids_64=1), ALIGN), (dict(row_of=A + 1), ALIGN),
])
def test_moe_sort_refusals(lib, kw, status):
    assert sort(lib, **kw) == status


def dispatch(lib, x=A, ldx=64, xt=BF16, tokens=4, topk=2, hidden=64, row_of=A, source=A,
             capacity=16, rows=A, rows_q=None, si=None, amax=None):
    return lib.fp8_moe_dispatch(x, ldx, xt, tokens, topk, hidden, row_of, source, capacity, rows,
                                rows_q, si, amax, None)


@pytest.mark.parametrize("kw, status", [
    (dict(x=None), NULL), (dict(rows=None), NULL), (dict(source=None), NULL),
    (dict(row_of=None), NULL), (dict(rows=None, rows_q=A), NULL),
    (dict(rows_q=A, si=A), UNSUPPORTED), (dict(amax=A), UNSUPPORTED),
    (dict(topk=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(hidden=-1), SHAPE),
    (dict(capacity=-1), SHAPE), (dict(ldx=-1), SHAPE), (dict(tokens=1 << 30, topk=4), SHAPE),
    (dict(xt=3), SHAPE), (dict(rows=ODD), ALIGN),
])
def test_moe_dispatch_refusals(lib, kw, status):
    assert dispatch(lib, **kw) == status


def test_moe_combine_refusals(lib):
    def combine(rows=A, ldr=64, y=A, w=A, row_of=A, topk=2):
        return lib.fp8_moe_combine(rows, ldr, BF16, 4, topk, 64, row_of, 16, w, y, None)
    assert combine(rows=None) == combine(y=None) == combine(row_of=None) == NULL
    assert combine(ldr=-1) == combine(topk=0) == SHAPE
    assert combine(w=A + 1) == combine(y=ODD) == ALIGN
    assert lib.fp8_moe_dispatch_backward(None, 64, BF16, 4, 2, 64, A, 16, A, None) == NULL
    assert "fp8_moe_dispatch_backward" in lib.fp8_last_error().decode()

    def bwd(dy=A, lddy=64, ldr=64, drows=A, source=A, dw=A):
        return lib.fp8_moe_combine_backward(dy, lddy, A, ldr, F32, 4, 2, 64, A, source, 16, A,
                                            drows, dw, None)
    assert bwd(dy=None) == bwd(drows=None) == bwd(source=None) == NULL
    assert bwd(lddy=-1) == bwd(ldr=-1) == SHAPE
    assert bwd(dy=A + 2) == bwd(dw=A + 2) == ALIGN


def ortho(lib, g=A, ldg=64, bsg=4096, gt=BF16, batch=1, rows=64, cols=64, steps=5, coef=True,
          eps=1e-7, out=A, ws=A):
    c = (ctypes.c_float * (3 * max(1, steps)))()
    return lib.fp8_orthogonalize(g, ldg, bsg, gt, batch, rows, cols, steps, c if coef else None,
                                 eps, 1.0, out, ws, None)


@pytest.mark.parametrize("kw, status", [
    (dict(g=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL), (dict(coef=False), NULL),
    (dict(steps=0), SHAPE), (dict(steps=65), SHAPE), (dict(rows=-1), SHAPE),
    (dict(cols=65537), SHAPE), (dict(batch=-1), SHAPE), (dict(batch=1 << 31), SHAPE),
    (dict(ldg=-1), SHAPE), (dict(bsg=-1), SHAPE), (dict(eps=-1e-7), SHAPE), (dict(gt=2), SHAPE),
    (dict(g=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(ws=A + 8), ALIGN),
])
def test_orthogonalize_refusals(lib, kw, status):
    assert ortho(lib, **kw) == status


def test_orthogonalize_workspace(lib):
    f = lib.fp8_orthogonalize_workspace_bytes
    assert f(0, 4, 4) == f(1, 0, 4) == f(-1, 4, 4) == f(1, 70000, 4) == 0
    assert f(1, 256, 512) >= 8 * 256 * 512 + 4 * 256 * 256
    assert f(3, 256, 512) > 2.9 * f(1, 256, 512)


def test_python_checks_refuse_host_tensors():
    import scaled_linear_layers_gb300 as fp8
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: fp8.fp8_layer_norm(x, None, None, 1e-5, x),
                 lambda: fp8.fp8_moe_dispatch(x, x, x, x),
                 lambda: fp8.fp8_moe_sort(x.int(), 4, 1, None, torch.zeros(4), None, None),
                 lambda: fp8.fp8_orthogonalize(x, x, None)):
        with pytest.raises(fp8.Fp8Error):
            call()
