"""The vocabulary operators refuse bad arguments before any device work.

No GPU is needed: every call here returns (or raises) before it touches the
device.  Pointers are made-up addresses that nothing follows."""
import ctypes

import pytest
import torch

from trie_constrained_beam_fr_b200 import build, fr

P = ctypes.c_void_p
BAD = fr.FR_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_null_handles():
    L, a = fr.libfr(), P(256)
    assert L.fr_embed_lookup(None, a, 8, 0, a, 1, 1.0, a, 8, 0, None) == BAD
    assert L.fr_embed_grad(None, a, 8, 0, a, 1, 1.0, a, 8, 0, 0, None) == BAD
    assert L.fr_embed_status(None) == BAD
    assert L.fr_embed_clear_status(None, None) == BAD
    assert L.fr_ce_loss(None, a, 8, a, 8, a, 1, a, a, None) == BAD
    assert L.fr_ce_grad(None, a, 8, a, 8, a, a, a, 1, a, 8, a, 8, None) == BAD
    assert L.fr_ce_status(None) == BAD
    assert L.fr_ce_clear_status(None, None) == BAD
    assert L.fr_ce_set_wait_test(None, 1000000, 1) == BAD
    assert L.fr_i8_matmul(None, a, 16, a, 1, a, 8, 0, None) == BAD
    assert L.fr_i8_lse(None, a, 16, a, 1, a, a, None) == BAD
    assert L.fr_i8_status(None) == BAD
    assert L.fr_i8_clear_status(None, None) == BAD
    assert L.fr_i8_set_wait_test(None, 1000000, 1) == BAD
    L.fr_embed_destroy(None)
    L.fr_ce_destroy(None)
    L.fr_i8_destroy(None)


@pytest.mark.parametrize("V,d,n", [(0, 8, 8), (8, 0, 8), (8, 8, 0), (-1, 8, 8), (8, 8, 1 << 30), ((1 << 30) + 1, 8, 8),
                                    (8, (1 << 24) + 1, 8)])
def test_embed_init_sizes(V, d, n):
    out = P(7)
    assert fr.libfr().fr_embed_init(V, d, n, ctypes.byref(out)) == BAD
    assert out.value is None


@pytest.mark.parametrize("V,d,rows", [(0, 8, 8), (8, 0, 8), (8, 8, 0), (8, 8, (1 << 24) + 1), ((1 << 24) + 1, 8, 8)])
def test_ce_init_sizes(V, d, rows):
    out = P(7)
    assert fr.libfr().fr_ce_init(V, d, rows, ctypes.byref(out)) == BAD
    assert out.value is None


def test_init_without_an_out_pointer():
    L = fr.libfr()
    assert L.fr_embed_init(8, 8, 8, None) == BAD
    assert L.fr_ce_init(8, 8, 8, None) == BAD
    assert L.fr_i8_init(P(256), 16, P(256), 8, 8, 8, 0, 0, None) == BAD


@pytest.mark.parametrize("w,ldw,ws,N,d,rows,base,span", [
    (None, 16, 256, 8, 8, 8, 0, 0), (256, 16, None, 8, 8, 8, 0, 0), (256, 16, 256, 0, 8, 8, 0, 0),
    (256, 16, 256, 8, 0, 8, 0, 0), (256, 131088, 256, 8, 131072, 8, 0, 0), (256, 16, 256, 8, 17, 8, 0, 0),
    (256, 24, 256, 8, 8, 8, 0, 0), (264, 16, 256, 8, 8, 8, 0, 0), (256, 16, 258, 8, 8, 8, 0, 0),
    (256, 16, 256, 8, 8, 0, 0, 0), (256, 16, 256, 8, 8, 8, -1, 0), (256, 16, 256, 8, 8, 8, 4, 5),
    (256, 16, 256, 8, 8, 8, 0, -1), (256, 16, 256, (1 << 24) + 1, 8, 8, 0, 0), (256, 16, 256, 8, 8, (1 << 24) + 1, 0, 0),
])
def test_i8_init_arguments(w, ldw, ws, N, d, rows, base, span):
    out = P(7)
    assert fr.libfr().fr_i8_init(P(w), ldw, P(ws), N, d, rows, base, span, ctypes.byref(out)) == BAD
    assert out.value is None


def test_i8_quantize_arguments():
    L, a = fr.libfr(), P(256)
    for x, ldx, dtype, rows, d, q, ldq, s in (
            (None, 8, 0, 1, 8, a, 8, a), (a, 8, 0, 1, 8, None, 8, a), (a, 8, 0, 1, 8, a, 8, None), (a, 7, 0, 1, 8, a, 8, a),
            (a, 8, 0, 1, 8, a, 7, a), (a, 8, 2, 1, 8, a, 8, a), (a, 8, 0, -1, 8, a, 8, a), (a, 8, 0, 1, 0, a, 8, a),
            (P(258), 8, 0, 1, 8, a, 8, a), (P(257), 8, 1, 1, 8, a, 8, a), (a, 8, 0, 1, 8, a, 8, P(257)),
            (a, 1 << 31, 0, 1, (1 << 30) + 1, a, 1 << 31, a)):
        assert L.fr_i8_quantize(x, ldx, dtype, rows, d, q, ldq, s, None) == BAD
    assert L.fr_i8_quantize(a, 8, 0, 0, 8, a, 8, a, None) == fr.FR_OK  # no rows: nothing to do


def test_the_binding_checks_shapes_types_and_devices():
    """Tensors on the CPU are refused by every call (they are the easiest wrong
    device), and the shape checks work without a GPU."""
    f, b, q = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.int8)
    fr_matrix = fr._matrix
    assert fr_matrix(f, "x", fr._FLOATS, 4, 8) == 8
    assert fr_matrix(f[:1], "x", fr._FLOATS, 1, 8) == 8
    assert fr_matrix(torch.zeros(4, 16)[:, :8], "x", fr._FLOATS, 4, 8) == 16
    for t, rows, cols in ((f, 5, 8), (f, 4, 7), (f[0], 4, 8), (f.t().contiguous().t(), 4, 8), (f[:1].expand(4, 8), 4, 8),
                          (f.half(), 4, 8), (q, 4, 8)):
        with pytest.raises(ValueError):
            fr_matrix(t, "x", fr._FLOATS, rows, cols)
    with pytest.raises(ValueError):
        fr._vector(torch.zeros(8)[::2], "v", torch.float32, 4)
    with pytest.raises(ValueError):
        fr._vector(torch.zeros(4, dtype=torch.int64), "v", torch.int32, 4)
    assert b.dtype in fr._FLOATS


