"""Outputs that are views of the inputs: the 8-bit norm's residual and the
rotary positions, in place and beside the input in the same rows."""

import pytest
import torch

import bit_w4a4_quantized_nvfp4_b200 as svdq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_w4a4_quantized_nvfp4_b200 import build

    build.build()
    svdq.load()


def _x(M, W, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(M, W, generator=g, device="cuda").to(torch.bfloat16)


def _ok():
    torch.cuda.synchronize()
    assert svdq.device_error() == 0


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("rot", [128, 64])
@pytest.mark.parametrize("M", [1, 2, 40])
def test_rope_in_place_through_a_view(M, rot, layout):
    """out = the heads' columns of x itself: the same as in place without out."""
    fr = svdq.rope_freqs(rot)
    pos = torch.arange(M, device="cuda") + 70
    x = _x(M, 7 * 128, 1)
    a, b = x.clone(), x.clone()
    svdq.rope_apply(a, 5, 128, pos, fr, layout=layout)
    y = svdq.rope_apply(b, 5, 128, pos, fr, layout=layout, out=b[:, :5 * 128])
    _ok()
    assert y.data_ptr() == b.data_ptr()
    assert torch.equal(a, b) and torch.equal(b[:, 5 * 128:], x[:, 5 * 128:]) and not torch.equal(a, x)


@pytest.mark.parametrize("M", [1, 2, 40])
def test_norm_in_place_through_views(M):
    """residual_out = a column range of the wider tensor that holds the residual."""
    x, wide = _x(M, 256, 2), _x(M, 1024, 3)
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    qa, r = svdq.fp8_norm_quantize(x, w, 1e-6, residual=wide[:, 256:512])
    work = wide.clone()
    qb, s = svdq.fp8_norm_quantize(x, w, 1e-6, residual=work[:, 256:512], residual_out=work[:, 256:512])
    _ok()
    assert torch.equal(r, s) and torch.equal(qa.codes.view(torch.uint8), qb.codes.view(torch.uint8))
    assert torch.equal(work[:, :256], wide[:, :256]) and torch.equal(work[:, 512:], wide[:, 512:])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("M", [1, 3, 700])
def test_rope_into_another_column_range(M, layout):
    """From one column range of a tensor into another, nothing beside it written."""
    fr = svdq.rope_freqs(64)
    pos = torch.arange(M, device="cuda")
    wide = _x(M, 1024, 4)
    want = svdq.rope_apply(wide[:, :256].clone(), 2, 128, pos, fr, layout=layout)
    work = wide.clone()
    svdq.rope_apply(work[:, :256], 2, 128, pos, fr, layout=layout, out=work[:, 512:768])
    _ok()
    assert torch.equal(work[:, 512:768], want)
    assert torch.equal(work[:, :512], wide[:, :512]) and torch.equal(work[:, 768:], wide[:, 768:])


@pytest.mark.parametrize("M", [1, 3, 700])
def test_norm_between_column_ranges(M):
    """x, the residual and its output as three column ranges of one tensor."""
    wide = _x(M, 1024, 5)
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    qa, r = svdq.fp8_norm_quantize(wide[:, :256].clone(), w, 1e-6, residual=wide[:, 256:512].clone())
    work = wide.clone()
    qb, s = svdq.fp8_norm_quantize(work[:, :256], w, 1e-6, residual=work[:, 256:512], residual_out=work[:, 768:])
    _ok()
    assert torch.equal(r, s) and torch.equal(qa.codes.view(torch.uint8), qb.codes.view(torch.uint8))
    assert torch.equal(work[:, :768], wide[:, :768])
