"""The 8-bit GEMM's bounded waits: a limit so short that waits run out makes
the call report it and nothing else go wrong. The calls behind it, on the same
multiprocessors, give the bits that they always give."""

import math

import pytest
import torch

import bit_w4a4_quantized_nvfp4_b200 as svdq

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
DEFAULT_NS = 2_000_000_000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_w4a4_quantized_nvfp4_b200 import build

    build.build()
    svdq.load()


def _layer(M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    G, nb = math.ceil(K / 128), math.ceil(N / 128)
    code = lambda r: torch.randn(r, K, generator=g, device="cuda").mul(60.0).clamp(-448, 448).to(F8)  # noqa: E731
    scale = lambda *s: torch.rand(*s, generator=g, device="cuda") * 0.02 + 1e-3  # noqa: E731
    return svdq.Fp8Act(M, K, code(M), scale(G, M)), svdq.Fp8Weight(K, N, code(N), scale(nb, G))


def _status():
    torch.cuda.synchronize()
    try:
        svdq.device_error()
        return svdq.Status.OK
    except svdq.SvdqError as e:
        return e.status


def _runs_out(M, K, N, out, sure):
    """sure: whether the first blocks' way from HBM is certain to outlast a limit of nothing."""
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")   # twice the L2
    qa, w = _layer(M, K, N)
    want = svdq.fp8_linear(qa, w, out_dtype=out)
    assert _status() == svdq.Status.OK
    seen = []
    for limit in (0, 0, 300, 1000, 3000, 10_000):
        cold.fill_(1)
        torch.cuda.synchronize()
        try:
            svdq.set_wait_limit_ns(limit)
            svdq.fp8_linear(qa, w, out_dtype=out)
        finally:
            svdq.set_wait_limit_ns(DEFAULT_NS)
        # behind it at once, so that it takes over the first call's shared memory
        got = svdq.fp8_linear(qa, w, out_dtype=out)
        seen.append(_status())
        assert seen[-1] in (svdq.Status.OK, svdq.Status.TIMEOUT)
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
        assert torch.equal(svdq.fp8_linear(qa, w, out_dtype=out).view(torch.uint8), want.view(torch.uint8))
        assert _status() == svdq.Status.OK
    assert svdq.Status.TIMEOUT in seen or not sure


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N,sure", [(1, 512, 2048, False), (1, 4096, 9216, True), (16, 12288, 4096, True),
                                        (24, 2064, 1000, False), (64, 4112, 5120, False), (77, 2064, 1000, False),
                                        (256, 4096, 4096, False), (1, 16384, 32768, True), (64, 16384, 16384, True)])
def test_few_rows(M, K, N, sure, out):
    """Parts of K of one block, of as many as there are stages and of more."""
    _runs_out(M, K, N, out, sure)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N,sure", [(2560, 512, 4096, False), (4608, 640, 12288, False), (1100, 2064, 4104, False),
                                        (4608, 1152, 4096, False), (8192, 8192, 8192, True)])
def test_many_rows(M, K, N, sure, out):
    """As many blocks of K as there are stages and fewer, tiles for some of the
    multiprocessors and for each several."""
    _runs_out(M, K, N, out, sure)
