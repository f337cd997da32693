"""Every variant of the 8-bit layer's kernels (tests/_fp8_plans.py) against 64
bits: sums that are exact in fp32 over the whole output, ordinary values on
rows of the first and last tiles and some between."""

import math

import pytest
import torch

import bit_w4a4_quantized_nvfp4_b200 as svdq
from tests import _fp8_plans as plans
from tests import _plain as plain

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
# as in the other tests of the norm: under 2^8 roundings of 2^-24; of the pass
# without it, a rounded reciprocal and a product
NORM_DELTA, QUANT_DELTA = 2.0 ** -16, 2.0 ** -22


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_w4a4_quantized_nvfp4_b200 import build

    build.build()
    svdq.load()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ok():
    torch.cuda.synchronize()
    assert svdq.device_error() == 0


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


LINEAR = [(k, s) for k, shapes in plans.LINEAR.items() for s in shapes]
ACT = [(k, s) for k, shapes in plans.ACT.items() for s in shapes]


@pytest.mark.parametrize("plan,shape", LINEAR)
def test_linear_exact_sums(plan, shape):
    """Whole codes up to 8 and scales that are powers of two from 1/2 to 2: every
    partial sum is a whole number of quarters, a term at most 64 * 4 of them
    times 4 = 2^10, so that 4096 terms stay below 2^24; past that codes up to
    4, whose terms are at most 2^8 quarters (17472 of them: 2^22.1)."""
    M, K, N = shape
    assert svdq.probe_fp8_linear_plan(M, K, N, _sms()) == plan
    G, nb = math.ceil(K / 128), math.ceil(N / 128)
    top = 8 if K <= 4096 else 4
    g = _gen(M)
    a = torch.randint(-top, top + 1, (M, K), generator=g, device="cuda").float().to(F8)
    c = torch.randint(-top, top + 1, (N, K), generator=g, device="cuda").float().to(F8)
    sa = torch.exp2(torch.randint(-1, 2, (G, M), generator=g, device="cuda").float())
    sw = torch.exp2(torch.randint(-1, 2, (nb, G), generator=g, device="cuda").float())
    bias = torch.randint(-8, 9, (N,), generator=g, device="cuda").to(torch.bfloat16)
    qa, w = svdq.Fp8Act(M, K, a, sa), svdq.Fp8Weight(K, N, c, sw)
    f = svdq.fp8_linear(qa, w, bias, out_dtype="f32")
    h = svdq.fp8_linear(qa, w, bias)
    _ok()
    W = (c.double() * sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]).t()
    for r in range(0, M, 4096):
        rows = slice(r, min(M, r + 4096))
        y64 = a[rows].double() * sa[:, rows].double().t().repeat_interleave(128, 1)[:, :K] @ W + bias.double()
        assert torch.equal(f[rows].double(), y64)
        assert torch.equal(h[rows], y64.float().to(torch.bfloat16))


@pytest.mark.parametrize("plan,shape", LINEAR)
def test_linear(plan, shape):
    """Both outputs, with and without bias; called again the same bits."""
    M, K, N = shape
    G, nb = math.ceil(K / 128), math.ceil(N / 128)
    g = _gen(M + 1)
    a = torch.randn(M, K, generator=g, device="cuda").mul(60.0).clamp(-448, 448).to(F8)
    c = torch.randn(N, K, generator=g, device="cuda").mul(60.0).clamp(-448, 448).to(F8)
    sa = torch.rand(G, M, generator=g, device="cuda") * 0.02 + 1e-3
    sw = torch.rand(nb, G, generator=g, device="cuda") * 0.02 + 1e-3
    bias = torch.randn(N, generator=g, device="cuda").to(torch.bfloat16)
    qa, w = svdq.Fp8Act(M, K, a, sa), svdq.Fp8Weight(K, N, c, sw)
    some = torch.randint(0, M, (48,), generator=g, device="cuda")
    rows = torch.cat([torch.arange(M, device="cuda")[:8], torch.arange(M, device="cuda")[-8:], some]).unique()
    for b in (bias, None):
        f = svdq.fp8_linear(qa, w, b, out_dtype="f32")
        h = svdq.fp8_linear(qa, w, b)
        again = svdq.fp8_linear(qa, w, b, out_dtype="f32")
        _ok()
        assert torch.equal(f.to(torch.bfloat16), h) and torch.equal(f, again)
        y64, mag = plain.linear64(a[rows], sa[:, rows], c, sw, b)
        assert ((f[rows].double() - y64).abs() <= plain.linear_bound(mag, K)).all()


@pytest.mark.parametrize("plan,shape", ACT)
def test_act(plan, shape):
    """Every row; without the norm also the bits that fewer rows, which take
    another variant, give."""
    norm, residual, *want = plan
    M, K = shape
    assert svdq.probe_fp8_act_plan(M, K, norm, residual, _sms()) == tuple(want)
    g = _gen(M + K)
    wide = torch.where(torch.rand(K, generator=g, device="cuda") < 0.02, 20.0, 1.0)
    x = (torch.randn(M, K, generator=g, device="cuda") * wide).to(torch.bfloat16)
    x[M // 2, K // 2:] = 0.0
    if not norm:
        qa = svdq.fp8_quantize_act(x)
        _ok()
        plain.check_codes(qa.codes, qa.scales, x.double(), QUANT_DELTA)
        for r in range(0, M, 997):
            rows = slice(r, min(M, r + 50))
            part = svdq.fp8_quantize_act(x[rows])
            assert torch.equal(part.codes.view(torch.uint8), qa.codes[rows].view(torch.uint8))
            assert torch.equal(part.scales, qa.scales[:, rows])
        return
    w = (1 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)
    res = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16) if residual else None
    qa, r = svdq.fp8_norm_quantize(x, w, 1e-6, residual=res)
    _ok()
    v, r64 = plain.norm64(x, w, 1e-6, res)
    plain.check_codes(qa.codes, qa.scales, v, NORM_DELTA)
    if residual:
        assert torch.equal(r, r64)
