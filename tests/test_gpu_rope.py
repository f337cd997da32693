"""Rotary positions on the GPU against their definition in 64 bits."""

import math

import pytest
import torch

import bit_w4a4_quantized_nvfp4_b200 as svdq
from tests import _plain as plain

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


def _check(y, x, heads, D, t, factor, layout):
    """Rotated columns: the tables' error and two fp32 roundings of the sum's
    terms, then half a step of bf16; the columns past them unchanged."""
    y64, mag = plain.rope64(x, heads, D, t, factor, layout)
    err = (y.double() - y64).abs()
    bound = (plain.TABLE_TOL + 2.0 ** -23) * factor * mag
    bound = bound + 2.0 ** -8 * (y64.abs() + bound)
    assert (err <= bound).all(), float((err - bound).max())
    R = 2 * t.shape[1]
    rest = slice(R, D)
    M = x.shape[0]
    assert torch.equal(y.reshape(M, heads, D)[:, :, rest], x[:, :heads * D].reshape(M, heads, D)[:, :, rest])


CASES = [(1, 1, 8, 2), (1, 48, 128, 128), (3, 5, 64, 64), (2, 3, 80, 40), (17, 2, 96, 48), (33, 7, 128, 64), (5, 1, 256, 256),
         (4, 2, 192, 96), (100, 16, 32, 32), (2, 1, 1024, 1024), (9, 3, 72, 70), (300, 9, 128, 128), (7, 2, 48, 6),
         (2, 96, 128, 128), (1030, 4, 64, 32)]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("M,heads,D,rot", CASES)
def test_rope_apply(M, heads, D, rot, layout):
    """Into another tensor and in place, from rows wider than the heads; what
    lies beside the heads stays as it was."""
    fr = svdq.rope_freqs(rot, scaling="yarn", factor=4.0, original_len=2048)
    pos = torch.arange(M, device="cuda") * 37 + 100003
    t = plain.angles64(pos, fr.freq)
    W = heads * D + 8
    x = _x(M, W, M + D)
    keep = x.clone()
    out = torch.empty(M, heads * D, dtype=torch.bfloat16, device="cuda")
    y = svdq.rope_apply(x, heads, D, pos, fr, layout=layout, out=out)
    _ok()
    assert y is out and torch.equal(x, keep)
    _check(y, keep, heads, D, t, fr.factor, layout)
    z = svdq.rope_apply(x, heads, D, pos, fr, layout=layout)
    _ok()
    assert z is x
    assert torch.equal(x[:, :heads * D], y) and torch.equal(x[:, heads * D:], keep[:, heads * D:])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("M,heads,D,rot", [(1300, 40, 128, 128), (1210, 96, 128, 64), (700, 300, 64, 64), (1300, 33, 72, 70),
                                           (5000, 6, 128, 128), (2600, 12, 96, 48), (1190, 2, 1024, 1000)])
def test_rope_many_wide_rows(M, heads, D, rot, layout):
    """As above, at rows enough that each has a CTA of its own or shares one,
    shorter and longer than a CTA takes at once."""
    test_rope_apply(M, heads, D, rot, layout)


@pytest.mark.parametrize("axes,rot", [((16, 56, 56), 128), ((2, 2), 4), ((8, 24), 32)])
def test_axes_and_tables(axes, rot):
    """Several position axes; the tables against 64 bits, and the rotation by
    them the same as rope_apply's."""
    fr = svdq.rope_freqs(axes, base=500.0)
    M = 77
    g = torch.Generator(device="cuda").manual_seed(1)
    pos = torch.randint(-300, 4000, (M, len(axes)), generator=g, device="cuda")
    c, s = svdq.rope_tables(pos, fr)
    _ok()
    t = plain.angles64(pos, fr.freq, fr.axis)
    assert c.shape == s.shape == (M, rot // 2)
    assert ((c.double() - t.cos()).abs() <= plain.TABLE_TOL).all()
    assert ((s.double() - t.sin()).abs() <= plain.TABLE_TOL).all()
    x = _x(M, 2 * rot + 8, 2)[:, :2 * rot] if rot % 8 == 0 else None
    if x is not None:
        y = svdq.rope_apply(x, 2, rot, pos, fr, out=torch.empty(M, 2 * rot, dtype=torch.bfloat16, device="cuda"))
        _ok()
        _check(y, x, 2, rot, t, 1.0, "interleaved")


@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 8.0), ("ntk", 8.0), ("yarn", 8.0)])
def test_far_positions(scaling, factor):
    """Angles keep their bits at positions up to 2^40 and below zero."""
    fr = svdq.rope_freqs(128, scaling=scaling, factor=factor, original_len=4096)
    pos = torch.tensor([0, 1, -1, 4095, 1 << 20, -(1 << 20), (1 << 31) - 1, 1 << 31, 1 << 33, (1 << 40) + 12345],
                       device="cuda")
    c, s = svdq.rope_tables(pos, fr)
    _ok()
    t = plain.angles64(pos, fr.freq)
    tol = plain.TABLE_TOL * fr.factor
    assert ((c.double() - t.cos() * fr.factor).abs() <= tol).all()
    assert ((s.double() - t.sin() * fr.factor).abs() <= tol).all()
    assert (c[0] == torch.tensor(fr.factor, device="cuda", dtype=torch.float32)).all() and (s[0] == 0).all()


def test_rotation_by_the_opposite_position_undoes_it():
    x = _x(9, 384, 3)
    pos = torch.arange(9, device="cuda") * 1000
    fr = svdq.rope_freqs(128)
    y = svdq.rope_apply(x.clone(), 3, 128, pos, fr, layout="half")
    z = svdq.rope_apply(y.clone(), 3, 128, -pos, fr, layout="half")
    _ok()
    # two roundings of half a bf16 step each, of values no larger than a pair's length
    a, b = x.view(9, 3, 128)[:, :, :64].double(), x.view(9, 3, 128)[:, :, 64:].double()
    length = (a.square() + b.square()).sqrt().repeat(1, 1, 2).view(9, 384)
    assert ((z.double() - x.double()).abs() <= 2.0 ** -8 * 2.5 * length).all()


def test_scores_depend_on_the_distance_alone():
    """q at position p and k at position s: their product is that of p - s."""
    fr = svdq.rope_freqs(64)
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k = (torch.randn(1, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    got = []
    for p, s in ((5, 3), (100005, 100003), (2, 0)):
        a = svdq.rope_apply(q.clone(), 1, 64, torch.tensor([p], device="cuda"), fr)
        b = svdq.rope_apply(k.clone(), 1, 64, torch.tensor([s], device="cuda"), fr)
        got.append(float((a.double() * b.double()).sum()))
    # both factors are rounded to bf16 (2^-8 of their size)
    tol = 2 * 2.0 ** -8 * 1.01 * float(q.double().norm() * k.double().norm())
    assert max(got) - min(got) <= 2 * tol


def test_the_fused_epilogue_takes_the_tables():
    """rope_tables -> pack_rope and qkv_norm_rope: the framework's own rotary
    calls on tables made here turn heads as rope_apply does (unit norm weights,
    rows of unit mean square)."""
    M, heads = 40, 2
    fr = svdq.rope_freqs((16, 56, 56))
    g = torch.Generator(device="cuda").manual_seed(7)
    pos = torch.randint(0, 64, (M, 3), generator=g, device="cuda")
    cos, sin = svdq.rope_tables(pos, fr)
    packed = svdq.pack_rope(cos, sin)
    sign = torch.where(torch.rand(M, 3 * heads * 128, generator=g, device="cuda") < 0.5, -1.0, 1.0).to(torch.bfloat16)
    one = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    y = svdq.qkv_norm_rope(sign.clone(), heads, one, one, 0.0, cos, sin)
    _ok()
    assert packed.M == M
    t = plain.angles64(pos, fr.freq, fr.axis)
    y64, mag = plain.rope64(sign, 2 * heads, 128, t, 1.0, "interleaved")
    bound = 2.0 ** -20 * mag + 2.0 ** -8 * y64.abs()
    assert ((y[:, :2 * heads * 128].double() - y64).abs() <= bound + 2.0 ** -8 * bound).all()


def test_edges():
    fr = svdq.rope_freqs(64)
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert svdq.rope_apply(e, 2, 64, none, fr).shape == (0, 128)
    c, s = svdq.rope_tables(none, fr)
    assert c.shape == (0, 32)
    # an axis that is not there is read as axis 0, never past the positions
    pos = torch.arange(5, device="cuda")
    bad = svdq.RopeFreqs(fr.freq, 1.0, torch.full((32,), 7, dtype=torch.int32, device="cuda"))
    assert torch.equal(svdq.rope_tables(pos, bad)[0], svdq.rope_tables(pos, fr)[0])
    # NaN and infinity stay in their pair
    x = _x(2, 128, 1)
    x[0, 3], x[1, 70] = float("nan"), float("inf")
    y = svdq.rope_apply(x.clone(), 2, 64, pos[:2] + 1, fr)
    _ok()
    gone = torch.zeros(2, 128, dtype=torch.bool)
    gone[0, 2:4] = True
    gone[1, 70:72] = True
    assert torch.equal(~y.isfinite().cpu(), gone)


def test_offsets_past_32_bits():
    M, W = 70000, 32768
    x = torch.zeros(M, W, dtype=torch.bfloat16, device="cuda")
    x[-2:] = _x(2, W, 1)
    keep = x[-2:].clone()
    fr = svdq.rope_freqs(128)
    pos = torch.arange(M, device="cuda")
    svdq.rope_apply(x, 256, 128, pos, fr)
    _ok()
    _check(x[-2:], keep, 256, 128, plain.angles64(pos[-2:], fr.freq), 1.0, "interleaved")
    assert (x[:64] == 0).all()


def test_stream_and_graph():
    fr = svdq.rope_freqs(128)
    x = _x(33, 512, 1)
    pos = torch.arange(33, device="cuda")
    want = svdq.rope_apply(x.clone(), 4, 128, pos, fr)
    side = torch.cuda.Stream()
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    svdq.rope_apply(x, 4, 128, pos, fr, out=y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    z = torch.empty_like(x)
    with torch.cuda.graph(g):
        svdq.rope_apply(x, 4, 128, pos, fr, out=z)
    for k in range(3):
        pos.add_(1000)
        g.replay()
        _ok()
        assert torch.equal(z, svdq.rope_apply(x.clone(), 4, 128, pos, fr))
    assert math.isfinite(float(z.float().sum()))
