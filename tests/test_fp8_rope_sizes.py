"""The largest sizes of the 8-bit layer and the rotary positions: what the
kernels' 32-bit sizes do not hold is refused, never cut short. By addresses
that are never read (the device is declared another architecture) and by
tensors without memory."""

import pytest
import torch

import bit_w4a4_quantized_nvfp4_b200 as svdq
from bit_w4a4_quantized_nvfp4_b200 import build as svdq_build

S = svdq.Status
PASSED = (S.UNSUPPORTED_ARCH, S.CUDA)
A = [(i + 1) << 42 for i in range(6)]
MOST = 2 ** 31 - 256


@pytest.fixture(scope="module")
def lib():
    svdq_build.build()
    L = svdq.load()
    svdq.debug_force_arch(9, 0)
    yield L
    svdq.debug_force_arch(0, 0)


def test_sizes_near_two_to_the_31(lib):
    """Blocks of 128 and 256 are counted in 32 bits: sizes up to 2^31 - 256."""
    def quant(M, K):
        return S(lib.svdq_fp8_quantize_act(M, K, A[0], K, A[1], A[2], None))

    def linear(M, K, N):
        return S(lib.svdq_fp8_linear(M, K, N, A[0], A[1], A[2], A[3], None, A[4], 0, None))

    def pack(K, N):
        return S(lib.svdq_fp8_pack_weight(K, N, A[0], A[1], A[2], None))

    def norm(M, K):
        return S(lib.svdq_fp8_norm_quantize(M, K, A[0], K, None, 0, A[3], 1e-6, None, 0, A[1], A[2], None))

    for big in (MOST + 16, 2 ** 31 - 16):
        assert quant(1, big) is S.SHAPE
        assert quant(0, big) is S.SHAPE
        assert linear(1, big, 8) is S.SHAPE
        assert linear(1, 16, big) is S.SHAPE
        assert linear(big, 16, 8) is S.SHAPE
        assert pack(big, 8) is S.SHAPE
        assert quant(big, 16) is S.SHAPE
        assert norm(big, 16) is S.SHAPE
    assert quant(1, MOST) in PASSED and quant(MOST, 16) in PASSED and norm(MOST, 16) in PASSED
    assert linear(1, MOST, 8) in PASSED and linear(1, 16, MOST) in PASSED and linear(MOST, 16, 8) in PASSED
    assert pack(MOST, 8) in PASSED


def test_tensors_past_32_bits():
    """Sizes that a C int would wrap to a small one."""
    wrap = 2 ** 32 + 16
    fr = svdq.rope_freqs(32, device="cpu")

    def meta(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")

    def refused(fn, *a, **kw):
        with pytest.raises(ValueError, match="2\\^31"):
            fn(*a, **kw)

    refused(svdq.fp8_quantize_act, meta(wrap, 16))
    refused(svdq.fp8_quantize_act, meta(1, wrap))
    refused(svdq.fp8_norm_quantize, meta(wrap, 16), meta(16), 1e-6)
    refused(svdq.fp8_pack_weight, meta(wrap, 16, dtype=torch.float32))
    refused(svdq.fp8_pack_weight, meta(16, wrap, dtype=torch.float32))
    refused(svdq.rope_apply, meta(wrap, 32), 1, 32, meta(wrap, dtype=torch.int64), fr)
    refused(svdq.rope_tables, meta(wrap, dtype=torch.int64), fr)
    refused(svdq.rope_tables, meta(4, dtype=torch.int64), svdq.RopeFreqs(meta(wrap, dtype=torch.float64)))
    refused(svdq.rope_tables, meta(4, wrap, dtype=torch.int64), fr)
    for M, K, N in ((wrap, 16, 8), (1, wrap, 8), (1, 16, wrap)):
        f8 = torch.float8_e4m3fn
        qa = svdq.Fp8Act(M, K, meta(M, K, dtype=f8), meta((K + 127) // 128, M, dtype=torch.float32))
        w = svdq.Fp8Weight(K, N, meta(N, K, dtype=f8), meta((N + 127) // 128, (K + 127) // 128, dtype=torch.float32))
        refused(svdq.fp8_linear, qa, w)
