"""Which overlaps of outputs with inputs the 8-bit layer and the rotary
positions refuse, by addresses that are never read: the device is declared
another architecture, so that a call which passes its checks launches nothing."""

import pytest

import bit_w4a4_quantized_nvfp4_b200 as svdq
from bit_w4a4_quantized_nvfp4_b200 import build as svdq_build

S = svdq.Status
FAR = 1 << 30
PASSED = (S.UNSUPPORTED_ARCH, S.CUDA)   # (CUDA: no device here at all)


@pytest.fixture(scope="module")
def lib():
    svdq_build.build()
    L = svdq.load()
    svdq.debug_force_arch(9, 0)
    yield L
    svdq.debug_force_arch(0, 0)


def rope(lib, M, x, ldx, y, ldy, heads=2):
    return S(lib.svdq_rope_apply(M, heads, 128, 64, 0, 1, 1 << 20, 5 * FAR, None, 1.0, x, ldx, y, ldy, None))


def norm(lib, M, x, ldx, r, ldr, ro, ldo, K=256):
    return S(lib.svdq_fp8_norm_quantize(M, K, x, ldx, r, ldr, 5 * FAR, 1e-6, ro, ldo, 6 * FAR, 7 * FAR, None))


def test_one_row_in_place_whatever_the_strides(lib):
    """The stride of a single row says nothing."""
    assert rope(lib, 1, FAR, 512, FAR, 256) in PASSED
    assert rope(lib, 2, FAR, 512, FAR, 256) is S.INVALID_ARG
    assert rope(lib, 2, FAR, 512, FAR, 512) in PASSED
    assert norm(lib, 1, FAR, 512, 2 * FAR, 1024, FAR, 256) in PASSED
    assert norm(lib, 1, FAR, 512, 2 * FAR, 1024, 2 * FAR, 256) in PASSED
    assert norm(lib, 2, FAR, 512, 2 * FAR, 1024, FAR, 256) is S.INVALID_ARG
    assert norm(lib, 2, FAR, 512, 2 * FAR, 1024, 2 * FAR, 1024) in PASSED
    # a part of the row is not the row
    assert rope(lib, 1, FAR, 512, FAR + 16, 512) is S.INVALID_ARG
    assert norm(lib, 1, FAR, 512, 2 * FAR, 1024, FAR + 16, 512) is S.INVALID_ARG


def test_column_ranges_of_one_tensor(lib):
    """Two column ranges of the same rows (one stride) that share no column do
    not overlap; those that share one, or whose strides differ, do."""
    for M in (1, 2, 9):
        assert rope(lib, M, FAR, 1024, FAR + 2 * 256, 1024) in PASSED
        assert rope(lib, M, FAR + 2 * 768, 1024, FAR, 1024) in PASSED
        assert rope(lib, M, FAR, 1024, FAR + 2 * 248, 1024) is S.INVALID_ARG
        assert rope(lib, M, FAR + 2 * 248, 1024, FAR, 1024) is S.INVALID_ARG
        assert norm(lib, M, FAR, 1024, FAR + 2 * 256, 1024, FAR + 2 * 512, 1024) in PASSED
        assert norm(lib, M, FAR, 1024, FAR + 2 * 256, 1024, FAR + 2 * 504, 1024) is S.INVALID_ARG
        assert norm(lib, M, FAR + 2 * 512, 1024, FAR + 2 * 256, 1024, FAR + 2 * 264, 1024) is S.INVALID_ARG
    # one range ends in the row after the one it starts in
    assert rope(lib, 2, FAR, 1024, FAR + 2 * 776, 1024) is S.INVALID_ARG
    assert rope(lib, 2, FAR, 1024, FAR + 2 * 768, 1024) in PASSED
    # ranges a row apart, and rows of other strides in between
    assert rope(lib, 2, FAR, 1024, FAR + 2 * (1024 + 256), 1024) in PASSED
    assert rope(lib, 2, FAR, 1024, FAR + 2 * 1024, 1024) is S.INVALID_ARG
    assert rope(lib, 4, FAR, 1024, FAR + 2 * 256, 2048) is S.INVALID_ARG
