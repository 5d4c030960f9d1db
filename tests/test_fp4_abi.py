"""The 4-bit entry points' argument checks that need no GPU: what is empty is done, what is
missing is refused before any device call."""
import ctypes

import pytest

import block_wise_w8a8_b200 as w8
import block_wise_w8a8_b200.build as b

OK, INVALID, SHAPE = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    b.build()
    return w8.lib()


def _linear(L, M, K, rec):
    path = ctypes.c_int(-1)
    return L.w8a8_fp4_linear(None, M, K, ctypes.byref(rec), None, None, None, 0, ctypes.byref(path), None), path.value


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("K", [0, 40, 64])
def test_a_weight_without_rows_gives_nothing(L, fmt, K):
    """N = 0 with the null pointers that empty tensors have."""
    rec = w8._FP4Weight(0, K, fmt, None, None, None, None)
    for M in (0, 1, 3, 7):
        assert _linear(L, M, K, rec) == (OK, w8.PATH_NONE)
        want = OK if K and K % 32 == 0 else SHAPE
        assert L.w8a8_fp4_linear_prequant(None, None, None, M, K, ctypes.byref(rec), None, None, None) == want


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_weight_with_rows_needs_its_buffers(L, fmt):
    rec = w8._FP4Weight(8, 64, fmt, None, None, None, None)
    assert _linear(L, 0, 64, rec)[0] == INVALID and _linear(L, 3, 64, rec)[0] == INVALID
    assert L.w8a8_fp4_linear_prequant(None, None, None, 3, 64, ctypes.byref(rec), None, None, None) == INVALID
    rec = w8._FP4Weight(0, 64, 2, None, None, None, None)              # no such format
    assert _linear(L, 3, 64, rec)[0] == INVALID
    rec = w8._FP4Weight(0, 64, fmt, None, None, None, None)            # another K than the activations'
    assert _linear(L, 3, 32, rec)[0] == INVALID
