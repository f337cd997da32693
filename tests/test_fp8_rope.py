"""Argument checks of the 8-bit layer and the rotary positions, and the
rotary frequencies' formulas. No kernel is launched here."""

import math

import pytest
import torch

import bit_w4a4_quantized_nvfp4_b200 as svdq
from bit_w4a4_quantized_nvfp4_b200 import build as svdq_build

S = svdq.Status
FAKE = 1 << 20   # never dereferenced: every call below fails validation first
FAR = 1 << 30


@pytest.fixture(scope="module")
def lib():
    svdq_build.build()
    return svdq.load()


def _call(fn, names, ok):
    def f(**kw):
        args = list(ok)
        for k, v in kw.items():
            args[names.index(k)] = v
        return fn(*args)
    return f


def test_quantize_act_validation(lib):
    c = _call(lib.svdq_fp8_quantize_act, ["M", "K", "x", "ldx", "codes", "scales", "s"],
              [4, 256, FAKE, 256, FAR, 2 * FAR, None])
    assert c(M=-1) == S.INVALID_ARG
    assert c(K=0) == S.INVALID_ARG
    assert c(K=100, ldx=104) == S.SHAPE          # K % 16
    assert c(ldx=248) == S.SHAPE                 # rows overlap
    assert c(ldx=257) == S.SHAPE                 # row stride % 8
    assert c(x=None) == S.INVALID_ARG
    assert c(codes=None) == S.INVALID_ARG
    assert c(scales=None) == S.INVALID_ARG
    assert c(x=FAKE + 8) == S.ALIGN
    assert c(codes=FAR + 4) == S.ALIGN
    assert c(codes=FAKE + 16) == S.INVALID_ARG   # codes overlap x
    assert c(scales=FAR + 512) == S.INVALID_ARG  # scales overlap codes
    assert c(M=0, x=None, codes=None, scales=None) == S.OK


def test_norm_quantize_validation(lib):
    c = _call(lib.svdq_fp8_norm_quantize,
              ["M", "K", "x", "ldx", "res", "ldr", "w", "eps", "ro", "ldo", "codes", "scales", "s"],
              [4, 256, FAKE, 256, 2 * FAR, 256, 3 * FAR, 1e-6, 4 * FAR, 256, 5 * FAR, 6 * FAR, None])
    assert c(K=32768 + 16, ldx=32768 + 16, ldr=32768 + 16, ldo=32768 + 16) == S.SHAPE
    assert c(eps=-1.0) == S.INVALID_ARG
    assert c(eps=float("nan")) == S.INVALID_ARG
    assert c(w=None) == S.INVALID_ARG
    assert c(ro=None) == S.INVALID_ARG           # residual without its output
    assert c(res=None) == S.INVALID_ARG          # and the other way round
    assert c(ldr=128) == S.SHAPE
    assert c(ldo=260) == S.SHAPE
    assert c(ro=4 * FAR + 2) == S.ALIGN
    assert c(ro=FAKE, ldo=512) == S.INVALID_ARG  # x itself, but at another stride
    assert c(ro=FAKE + 512) == S.INVALID_ARG     # overlaps x by a row
    assert c(codes=2 * FAR) == S.INVALID_ARG     # codes over the residual
    assert c(scales=3 * FAR) == S.INVALID_ARG    # scales over the weight
    assert c(M=0, x=None, res=None, w=None, ro=None, codes=None, scales=None) == S.OK


def test_pack_and_linear_validation(lib):
    p = _call(lib.svdq_fp8_pack_weight, ["K", "N", "W", "codes", "scales", "s"], [256, 64, FAKE, FAR, 2 * FAR, None])
    assert p(K=0) == S.INVALID_ARG
    assert p(K=24) == S.SHAPE
    assert p(N=12) == S.SHAPE
    assert p(N=1 << 23) == S.SHAPE
    assert p(W=None) == S.INVALID_ARG
    assert p(codes=FAR + 8) == S.ALIGN
    c = _call(lib.svdq_fp8_linear, ["M", "K", "N", "xc", "xs", "wc", "ws", "b", "y", "out", "s"],
              [4, 256, 64, FAKE, FAR, 2 * FAR, 3 * FAR, 4 * FAR, 5 * FAR, 0, None])
    assert c(M=-1) == S.INVALID_ARG
    assert c(N=0) == S.INVALID_ARG
    assert c(K=264) == S.SHAPE
    assert c(N=60) == S.SHAPE
    assert c(out=2) == S.INVALID_ARG
    assert c(out=3) == S.INVALID_ARG
    assert c(wc=None) == S.INVALID_ARG
    assert c(y=None) == S.INVALID_ARG
    assert c(xc=FAKE + 8) == S.ALIGN
    assert c(xs=FAR + 2) == S.ALIGN
    assert c(b=4 * FAR + 2) == S.ALIGN
    assert c(y=FAKE) == S.INVALID_ARG            # y over the activations
    assert c(y=2 * FAR + 64) == S.INVALID_ARG    # y over the weight
    assert c(M=0, xc=None, xs=None, wc=None, ws=None, b=None, y=None) == S.OK


def test_rope_validation(lib):
    t = _call(lib.svdq_rope_tables, ["M", "axes", "pairs", "pos", "freq", "axis", "f", "c", "n", "s"],
              [4, 1, 64, FAKE, FAR, None, 1.0, 2 * FAR, 3 * FAR, None])
    assert t(M=-1) == S.INVALID_ARG
    assert t(axes=0) == S.INVALID_ARG
    assert t(axes=9) == S.INVALID_ARG
    assert t(pairs=0) == S.INVALID_ARG
    assert t(pairs=513) == S.SHAPE
    assert t(pos=None) == S.INVALID_ARG
    assert t(freq=FAR + 4) == S.ALIGN
    assert t(n=2 * FAR + 512) == S.INVALID_ARG   # the tables overlap
    assert t(c=FAR) == S.INVALID_ARG             # cos over the frequencies
    assert t(M=0, pos=None, freq=None, c=None, n=None) == S.OK
    a = _call(lib.svdq_rope_apply, ["M", "heads", "D", "pairs", "layout", "axes", "pos", "freq", "axis", "f", "x",
                                    "ldx", "y", "ldy", "s"],
              [4, 2, 128, 64, 0, 1, FAKE, FAR, None, 1.0, 2 * FAR, 256, 3 * FAR, 256, None])
    assert a(heads=0) == S.INVALID_ARG
    assert a(layout=2) == S.INVALID_ARG
    assert a(pairs=65) == S.SHAPE                # 2 pairs > head_dim
    assert a(D=132) == S.SHAPE
    assert a(ldx=248) == S.SHAPE
    assert a(ldy=260) == S.SHAPE
    assert a(heads=1 << 14, ldx=1 << 21, ldy=1 << 21) == S.SHAPE
    assert a(x=2 * FAR + 8) == S.ALIGN
    assert a(y=2 * FAR, ldy=512) == S.INVALID_ARG   # x itself, but at another stride
    assert a(y=2 * FAR + 256) == S.INVALID_ARG      # partly over x
    assert a(y=FAKE) == S.INVALID_ARG               # over the positions
    assert a(M=0, pos=None, freq=None, x=None, y=None) == S.OK


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_binding_checks_fp8(lib):
    x, w = _bf(8, 256), _bf(256)
    _raises("CUDA", svdq.fp8_quantize_act, x)                              # well formed
    _raises("x: expected", svdq.fp8_quantize_act, torch.zeros(8, 256))
    _raises("x: expected", svdq.fp8_quantize_act, _bf(256))
    _raises("unit stride", svdq.fp8_quantize_act, _bf(256, 8).t())
    _raises("row stride", svdq.fp8_quantize_act, _bf(1, 256).expand(8, 256))
    _raises("CUDA", svdq.fp8_norm_quantize, x, w, 1e-6)
    _raises("weight: shape", svdq.fp8_norm_quantize, x, _bf(128), 1e-6)
    _raises("weight: dtype", svdq.fp8_norm_quantize, x, torch.zeros(256), 1e-6)
    _raises("K = 128", svdq.fp8_linear, svdq.Fp8Act(8, 128, None, None), svdq.Fp8Weight(256, 64, None, None))
    f8 = torch.float8_e4m3fn
    qa = svdq.Fp8Act(8, 256, torch.zeros(8, 256).to(f8), torch.zeros(2, 8))
    fw = svdq.Fp8Weight(256, 136, torch.zeros(136, 256).to(f8), torch.zeros(2, 2))
    _raises("CUDA", svdq.fp8_linear, qa, fw)                               # well formed
    _raises("bias: shape", svdq.fp8_linear, qa, fw, _bf(128))
    _raises("out_dtype", svdq.fp8_linear, qa, fw, out_dtype="bf16_gelu")
    _raises("qa.scales: shape", svdq.fp8_linear, svdq.Fp8Act(8, 256, qa.codes, torch.zeros(8, 2)), fw)
    _raises("qa.codes: dtype", svdq.fp8_linear, svdq.Fp8Act(8, 256, torch.zeros(8, 256), qa.scales), fw)
    _raises("w.scales: shape", svdq.fp8_linear, qa, svdq.Fp8Weight(256, 136, fw.codes, torch.zeros(1, 2)))
    _raises("W: expected", svdq.fp8_pack_weight, torch.zeros(256, 64, dtype=torch.float64))


def test_binding_checks_rope(lib):
    fr = svdq.rope_freqs(128, device="cpu")
    pos = torch.arange(8)
    x = _bf(8, 512)
    _raises("CUDA", svdq.rope_apply, x, 4, 128, pos, fr)                   # well formed
    _raises("5 heads", svdq.rope_apply, x, 5, 128, pos, fr)
    _raises("layout", svdq.rope_apply, x, 4, 128, pos, fr, layout="split")
    _raises("x: expected", svdq.rope_apply, x.float(), 4, 128, pos, fr)
    _raises("CUDA", svdq.rope_tables, pos, fr)


def test_rope_frequencies():
    """The formulas: base^(-2i/d); linear; ntk's slowest pair at 1/factor and
    its fastest unchanged; yarn's ends and its factor on cos and sin."""
    d, base = 128, 10000.0
    f = svdq.rope_freqs(d, base, device="cpu")
    assert f.factor == 1.0 and f.axis is None and f.freq.dtype == torch.float64
    for i in range(d // 2):
        assert math.isclose(f.freq[i], base ** (-2 * i / d), rel_tol=1e-14)
    lin = svdq.rope_freqs(d, base, "linear", 8.0, device="cpu")
    assert torch.allclose(lin.freq * 8.0, f.freq, rtol=1e-14)
    ntk = svdq.rope_freqs(d, base, "ntk", 8.0, device="cpu")
    assert ntk.freq[0] == 1.0
    assert math.isclose(ntk.freq[-1] * 8.0, f.freq[-1], rel_tol=1e-12)
    yarn = svdq.rope_freqs(d, base, "yarn", 8.0, 4096, device="cpu")
    turns = f.freq * 4096 / (2 * math.pi)
    ratio = f.freq / yarn.freq
    assert torch.allclose(ratio[turns > 40], torch.ones((), dtype=torch.float64))
    assert torch.allclose(ratio[turns < 0.9], torch.full((), 8.0, dtype=torch.float64))
    assert (ratio[1:] >= ratio[:-1] - 1e-12).all()
    assert math.isclose(yarn.factor, 0.1 * math.log(8.0) + 1.0)
    ax = svdq.rope_freqs((16, 56, 56), device="cpu")
    assert ax.axis.tolist() == [0] * 8 + [1] * 28 + [2] * 28 and ax.axis.dtype == torch.int32
    assert ax.freq[0] == 1.0 and ax.freq[8] == 1.0 and ax.freq[36] == 1.0
    for bad in (127, 0, (16, 7), []):
        _raises("rot_dim", svdq.rope_freqs, bad, device="cpu")
    _raises("scaling", svdq.rope_freqs, 64, scaling="dynamic", device="cpu")
    _raises("original_len", svdq.rope_freqs, 64, scaling="yarn", factor=2.0, device="cpu")
    _raises("factor", svdq.rope_freqs, 64, scaling="linear", factor=0.5, device="cpu")
