"""The block-scaled FP8 layer's limits, and what its build and binding decide
without a GPU."""

import ctypes

import pytest

import rotation_bit_ptq_b200 as rbq

FAKE = ctypes.c_void_p(0x10000)                  # never dereferenced
BF, NONE, GELU = rbq.RBQ_BF16, rbq.RBQ_ACT_NONE, rbq.RBQ_ACT_GELU
MOST = 1 << 30


@pytest.fixture(scope="module")
def lib():
    return rbq.lib()


# ---- sizes: no count of blocks leaves 32 bits ---------------------------------------

# the first above the limit, and those whose number of blocks of 128 would wrap
@pytest.mark.parametrize("n", [MOST + 16, (1 << 31) - 128, (1 << 31) - 112, (1 << 31) - 16])
def test_widths_above_the_limit_are_refused(lib, n):
    for rc in (lib.quantize_fp8(FAKE, BF, 1, n, NONE, FAKE, FAKE, None, None, None),
               lib.quantize_fp8(FAKE, BF, 0, n, GELU, FAKE, FAKE, FAKE, FAKE, None),
               lib.quantize_weights_fp8(FAKE, BF, 16, n, FAKE, FAKE, None, None, None),
               lib.quantize_weights_fp8(FAKE, BF, n, 16, FAKE, FAKE, FAKE, FAKE, None),
               lib.qlinear_fp8(FAKE, FAKE, FAKE, FAKE, 1, 8, n, FAKE, None),
               lib.qlinear_fp8(FAKE, FAKE, FAKE, FAKE, 0, 8, n, FAKE, None),
               lib.qlinear_fp8_wgrad(FAKE, FAKE, FAKE, 1, 8, n, FAKE, BF, None),
               lib.gelu_backward_fp8(FAKE, FAKE, FAKE, 1, n, FAKE, None, None, None)):
        assert rc == rbq.RBQ_EINVAL


def test_the_limit_itself_is_allowed(lib):
    """(No rows, so that nothing is launched.)"""
    assert lib.quantize_fp8(None, BF, 0, MOST, NONE, None, None, None, None, None) == rbq.RBQ_OK
    assert lib.quantize_weights_fp8(None, BF, 0, MOST, None, None, None, None, None) == rbq.RBQ_OK
    assert lib.qlinear_fp8(None, None, None, None, 0, MOST, MOST, None, None) == rbq.RBQ_OK
    assert lib.qlinear_fp8_wgrad(None, None, None, MOST, 0, MOST, None, BF, None) == rbq.RBQ_OK
    assert lib.gelu_backward_fp8(None, None, None, 0, MOST, None, None, None, None) == rbq.RBQ_OK
