"""Sizes of workspaces and their borders: host arithmetic only."""
import ctypes

import pytest

import __graft_entry__


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    from scaled_linear_layers_gb300 import _lib
    return _lib.load()


def pad(v, m):
    return -(-v // m) * m


@pytest.mark.parametrize("batch, rows, cols", [(1, 1, 1), (1, 256, 256), (8, 1531, 1000),
                                               (1, 4096, 14336), (3, 200, 5001), (100000, 16, 16),
                                               (1000, 128, 64)])
def test_orthogonalize_workspace_is_what_the_header_says(lib, batch, rows, cols):
    s, l = min(rows, cols), max(rows, cols)
    x, t, u = batch * rows * pad(cols, 64), pad(s, 128) // 128, pad(l, 128) // 128
    parts = 2 * x if s <= 2048 <= l else 0
    want = 8 * x + 4 * batch * s * pad(s, 64) + parts \
        + 12 * batch * min(rows, max(16, 2048 // batch)) + 4 * batch * (5 * t * (t + 1) + t * u)
    got = lib.fp8_orthogonalize_workspace_bytes(batch, rows, cols)
    assert want <= got <= want + 10 * 256  # ten regions, each from a multiple of 256
    precise = lib.fp8_orthogonalize_precise_workspace_bytes(batch, rows, cols)
    assert want + 4 * batch * s * pad(s, 64) <= precise <= got + 4 * batch * s * pad(s, 64) + 512


def test_orthogonalize_tiles(lib):
    f = lib.fp8_orthogonalize_workspace_bytes
    assert f(2 ** 23 - 1, 1, 1) > 0 and f(2 ** 23, 1, 1) == 0
    assert f(2 ** 23 // 4, 129, 129) == 0 and f(2 ** 23 // 4 - 1, 129, 129) > 0
    assert lib.fp8_orthogonalize_precise_workspace_bytes(2 ** 23, 1, 1) == 0


def test_precise_refusals_name_their_entry_point(lib):
    a, abc = 0x10000, (ctypes.c_float * 3)(1, 0, 0)
    call = lib.fp8_orthogonalize_precise
    assert call(a, 64, 4096, 0, 1, 64, 64, 0, abc, 0.0, 1.0, a, a, None) == 2   # steps
    assert "fp8_orthogonalize_precise" in lib.fp8_last_error().decode()
    assert call(a, 64, 4096, 0, 1, 64, 64, 1, None, 0.0, 1.0, a, a, None) == 1  # coefficients
    assert call(a, 64, 4096, 0, 1, 64, 64, 1, abc, 0.0, 1.0, a, a + 8, None) == 3  # workspace


def test_sort_needs_a_workspace_from_1025_assignments(lib):
    assert lib.fp8_moe_sort_workspace_bytes(1024, 8) == 0
    assert lib.fp8_moe_sort_workspace_bytes(1025, 8) > 0
    a = 0x10000  # never dereferenced: the refusal comes first
    assert lib.fp8_moe_sort(a, 0, 1025, 8, 16, 1 << 20, a, a, a, a, None, None) == 1  # FP8_ERR_NULL


def test_current_stream_without_the_private_call(lib, monkeypatch):
    import scaled_linear_layers_gb300 as fp8
    import torch

    class Stream:
        cuda_stream = 0x1234

    monkeypatch.setattr(fp8, "_current_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream)
    assert fp8._stream(None) == 0x1234
    assert fp8._stream(Stream) == 0x1234
