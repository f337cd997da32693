"""The norm of the 8-bit layer at the ends of fp32's range, against 64 bits.

bf16 values reach from 2^-133 to 2^128, so that a row's squares, its mean
square's root and the products with the weight can each leave fp32 although the
result lies within it."""

import pytest
import torch

import bit_w4a4_quantized_nvfp4_b200 as svdq
from tests import _plain as plain

pytestmark = pytest.mark.gpu

BF16_MAX = torch.finfo(torch.bfloat16).max
# as for rows of ordinary size: a sum of up to 32768 squares (chains of at most
# 128 + 20 additions), its mean, root and two products, under 2^8 roundings of
# 2^-24 (one more where a factor is subnormal in fp32: it keeps 21 bits or more)
NORM_DELTA = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_w4a4_quantized_nvfp4_b200 import build

    build.build()
    svdq.load()


def _acts(M, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)


def _norm(x, w, eps, residual):
    """The kernel's codes and scales for x, split as x + 0 where residual is asked for."""
    res = torch.zeros_like(x) if residual else None
    qa, _ = svdq.fp8_norm_quantize(x, w, eps, residual=res)
    torch.cuda.synchronize()
    assert svdq.device_error() == 0
    return qa


# few rows (spread over several warps) and many (a row a warp), short and long
SIZES = [(6, 16), (6, 400), (6, 4096), (5, 32768), (3700, 400)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_rows_at_the_top_of_the_range(M, K, residual):
    """Rows whose sum of squares leaves fp32 however few of their columns are
    large, up to a row of the largest bf16 value."""
    x = _acts(M, K, K)
    sign = torch.where(_acts(1, K, 1)[0] < 0, -1.0, 1.0)
    x[0] = (1e37 * sign).to(torch.bfloat16)
    x[1] = (2.5e38 * sign).to(torch.bfloat16)
    x[2] = BF16_MAX
    x[3, :] = 1.0
    x[3, 3], x[3, -2] = 3e38, -3e38
    x[4] = (x[4].float() * 2e18).to(torch.bfloat16)
    w = (1 + 0.2 * _acts(1, K, 2)[0].float()).to(torch.bfloat16)
    qa = _norm(x, w, 1e-6, residual)
    v, _ = plain.norm64(x, w, 1e-6)
    plain.check_codes(qa.codes, qa.scales, v, NORM_DELTA)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_rows_at_the_bottom_of_the_range(M, K, residual):
    """eps = 0 (or too small to count): rows of bf16 subnormals, whose inverse
    root leaves fp32, one column among zeros, and weights that bring products
    back to ordinary size."""
    x = _acts(M, K, K + 1)
    w = (1 + 0.2 * _acts(1, K, 2)[0].float()).to(torch.bfloat16)
    x[0] = 2.0 ** -133
    x[1] = (x[1].float() * 2.0 ** -128).to(torch.bfloat16)
    x[2] = (x[2].float() * 2.0 ** -118).to(torch.bfloat16)
    x[3] = 0.0
    x[3, -1] = 2.0 ** -133
    x[4] = (x[4].float() * 2.0 ** -50).to(torch.bfloat16)
    for eps in (0.0, 2.0 ** -140):
        qa = _norm(x, w, eps, residual)
        v, _ = plain.norm64(x, w, eps)
        plain.check_codes(qa.codes, qa.scales, v, NORM_DELTA)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_a_value_past_fp32_spoils_its_block(M, K, residual):
    """Weights near the largest value: where r / rms * w leaves fp32 (r w stays
    within) the block holds an infinity, so all of it stands for NaN; a block
    that stays within is as ever, however near."""
    x = (_acts(M, K, K + 2).float().clamp(-1.5, 1.5) / 64).to(torch.bfloat16)
    x[:, 5] = 2.0 / 64
    x[1] = 1.0 / 64
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    w[:8] = 3e38
    if K > 256:
        w[128:256] = 1e38
    qa = _norm(x, w, 1e-6, residual)
    v, _ = plain.norm64(x, w, 1e-6)
    top = plain.scales64(v) * 448.0
    limit = torch.finfo(torch.float32).max
    gone = top > limit
    # none of the inputs is within the norm's error of the border
    assert ((top - limit).abs() > 1e-3 * limit).all() and gone[0, 0] and not gone[0, 1]
    got = qa.codes.float() * plain.spread(qa.scales, K)
    assert torch.equal(got.isnan(), plain.spread(gone, K))
    rows = ~gone.any(0)
    plain.check_codes(qa.codes[rows], qa.scales[:, rows], v[rows], NORM_DELTA)
    assert (((qa.scales.double() - top / 448.0).abs() <= NORM_DELTA * top / 448.0) | gone).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_products_with_the_weight_below_fp32(M, K, residual):
    """Small rows under small weights (eps = 0): r w rounds to zero in fp32
    over a whole block while r / rms * w does not. Blocks of zeros beside them
    stay zeros."""
    x = _acts(M, K, K + 3)
    w = (1 + 0.2 * _acts(1, K, 2)[0].float()).to(torch.bfloat16)
    w[:128] = 2.0 ** -75
    w[-16:] = 2.0 ** -132
    x[0] = (x[0].float() * 2.0 ** -90).to(torch.bfloat16)
    x[1] = (x[1].float() * 2.0 ** -30).to(torch.bfloat16)
    x[2] = (x[2].float() * 2.0 ** -99).to(torch.bfloat16)
    x[2, :8] = 0.0
    if K > 256:
        x[2, :256] = 0.0
    qa = _norm(x, w, 0.0, residual)
    v, _ = plain.norm64(x, w, 0.0)
    plain.check_codes(qa.codes, qa.scales, v, NORM_DELTA)
    if K > 256:
        assert (qa.codes[2, :256].float() == 0).all() and (qa.scales[:2, 2] == plain.MIN_SCALE).all()


def test_rows_of_zeros_among_small_ones():
    """A padded batch at an eps that counts for nothing else: zeros stay zeros
    at the smallest scale beside rows of any size."""
    x = _acts(300, 400, 9)
    x[100:200] = 0.0
    x[200:] = (x[200:].float() * 1e-7).to(torch.bfloat16)
    x[250, 128:256] = 0.0
    w = torch.ones(400, dtype=torch.bfloat16, device="cuda")
    for eps in (1e-12, 1e-30):
        qa = _norm(x, w, eps, False)
        v, _ = plain.norm64(x, w, eps)
        plain.check_codes(qa.codes, qa.scales, v, NORM_DELTA)
        assert (qa.codes[100:200].float() == 0).all() and (qa.scales[:, 100:200] == plain.MIN_SCALE).all()


@pytest.mark.parametrize("residual", [False, True])
def test_products_below_fp32_with_an_eps(residual):
    """As above where eps alone sets the norm and the row's squares vanish
    beside it: v = 2^-84 * 1e6 * 2^-70, some 2^-134, a code of some 2^-8."""
    x = torch.full((40, 400), 2.0 ** -84, dtype=torch.bfloat16, device="cuda")
    w = torch.full((400,), 2.0 ** -70, dtype=torch.bfloat16, device="cuda")
    qa = _norm(x, w, 1e-12, residual)
    v, _ = plain.norm64(x, w, 1e-12)
    plain.check_codes(qa.codes, qa.scales, v, NORM_DELTA)
    assert (qa.codes.float() > 0).all()
