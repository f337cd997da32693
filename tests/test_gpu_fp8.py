"""The 8-bit linear layer on the GPU against its definition in 64 bits:
norm + residual + quantisation, weight pack, and the GEMM at few and many
rows. Bounds count the kernels' roundings (tests/_plain.py)."""

import math

import pytest
import torch

import bit_w4a4_quantized_nvfp4_b200 as svdq
from tests import _plain as plain

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
# a norm's value: a sum of squares over up to 32768 columns (chains of at most
# 128 + 20 additions), its mean, square root (two steps) and two products:
# under 2^8 roundings of 2^-24
NORM_DELTA = 2.0 ** -16
QUANT_DELTA = 2.0 ** -22


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_w4a4_quantized_nvfp4_b200 import build

    build.build()
    svdq.load()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _acts(M, K, seed, spread=20.0):
    g = _gen(seed)
    wide = torch.where(torch.rand(K, generator=g, device="cuda") < 0.02, spread, 1.0)
    return (torch.randn(M, K, generator=g, device="cuda") * wide).to(torch.bfloat16)


def _codes(rows, K, seed):
    return torch.randn(rows, K, generator=_gen(seed), device="cuda").mul(60.0).clamp(-448, 448).to(F8)


def _positive(*shape, seed):
    return torch.rand(*shape, generator=_gen(seed), device="cuda") * 0.02 + 1e-3


def _ok():
    torch.cuda.synchronize()
    assert svdq.device_error() == 0


# ------------------------------------------------------------------ activations
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (2, 4096), (77, 1040), (129, 2064), (5, 12288), (4, 16384),
                                 (3, 32768), (2, 40000), (700, 256), (1500, 512)])
def test_quantize_act(M, K):
    x = _acts(M, K, M + K)
    qa = svdq.fp8_quantize_act(x)
    _ok()
    plain.check_codes(qa.codes, qa.scales, x.double(), QUANT_DELTA)


@pytest.mark.parametrize("M,K,residual", [(1, 16, True), (1, 128, False), (1, 4096, True), (3, 144, True), (9, 1040, False),
                                          (129, 2064, True), (5, 12288, True), (4, 16400, True), (3, 32768, True),
                                          (2, 32768, False), (700, 256, True), (33, 8192, False), (600, 5120, True),
                                          (3700, 1040, True), (3700, 2064, False), (4000, 128, True)])
def test_norm_quantize(M, K, residual):
    x = _acts(M, K, M + K)
    w = (1 + 0.2 * torch.randn(K, generator=_gen(1), device="cuda")).to(torch.bfloat16)
    res = _acts(M, K, M + K + 1) if residual else None
    qa, r = svdq.fp8_norm_quantize(x, w, 1e-6, residual=res)
    _ok()
    v, r64 = plain.norm64(x, w, 1e-6, res)
    if residual:
        assert torch.equal(r.view(torch.int16), r64.view(torch.int16))
    else:
        assert r is None
    plain.check_codes(qa.codes, qa.scales, v, NORM_DELTA)


@pytest.mark.parametrize("M", [9, 3700])
def test_norm_quantize_extremes(M):
    """Rows of zeros (with eps and without values), tiny and huge rows, a NaN,
    an infinity, products with the weight past fp32's range, blocks of zeros:
    each row as its definition gives, the rows beside it as ever. Few rows are
    spread over several warps, many have one each."""
    K = 400
    x = _acts(M, K, 3)
    x[1] = 0.0
    x[2] *= 1e-30
    x[3] = 3.0e18
    x[4, 130] = float("nan")
    x[5, 7] = float("inf")
    x[6] = torch.finfo(torch.bfloat16).tiny
    x[7, 128:256] = 0.0
    w = torch.ones(K, device="cuda", dtype=torch.bfloat16)
    qa, _ = svdq.fp8_norm_quantize(x, w, 1e-6)
    _ok()
    fine = [m for m in range(M) if m not in (4, 5)]
    v, _ = plain.norm64(x, w, 1e-6)
    plain.check_codes(qa.codes[fine], qa.scales[:, fine], v[fine], NORM_DELTA)
    got = qa.codes.float() * plain.spread(qa.scales, K)
    assert got[4].isnan().all()          # the NaN is in the row's mean square
    assert got[5, 7].isnan()             # inf / inf; the other values of the row go to 0
    assert (qa.codes[1].float() == 0).all() and (qa.scales[:, 1] == plain.MIN_SCALE).all()
    assert (qa.codes[7, 128:256].float() == 0).all()
    x[8] = 1e30
    w[:] = 1e20
    w[5] = 1e-30
    qa, _ = svdq.fp8_norm_quantize(x, w, 0.0, residual=torch.zeros_like(x))
    _ok()
    v, _ = plain.norm64(x, w, 0.0)
    fine = [m for m in range(M) if m not in (1, 4, 5)]
    plain.check_codes(qa.codes[fine], qa.scales[:, fine], v[fine], NORM_DELTA)
    assert (qa.codes[1].float() * plain.spread(qa.scales, K)[1]).isnan().all()   # 0 / 0


@pytest.mark.parametrize("M,K,residual", [(3700, 7184, False), (3700, 2320, True), (40, 30736, False), (1300, 4112, True),
                                          (9000, 1040, False), (300, 12304, True)])
def test_norm_quantize_ragged(M, K, residual):
    """Rows whose last step is short, in each number of loads in flight, with
    rows that are summed again and blocks that are done again in between."""
    x = _acts(M, K, M + K)
    w = (1 + 0.2 * torch.randn(K, generator=_gen(2), device="cuda")).to(torch.bfloat16)
    x[1] *= 1e-30
    x[2] = 3.0e18
    x[3, -144:] = 0.0
    x[M - 1, :-16] *= 1e-3
    w[K - 130] = 1e-38
    w[-16:] = 1e30
    res = torch.zeros_like(x) if residual else None
    if residual:
        res[5] = x[5]
    qa, r = svdq.fp8_norm_quantize(x, w, 0.0, residual=res)
    _ok()
    v, r64 = plain.norm64(x, w, 0.0, res)
    if residual:
        assert torch.equal(r.view(torch.int16), r64.view(torch.int16))
    plain.check_codes(qa.codes, qa.scales, v, NORM_DELTA)


def test_quantize_extremes():
    """Without the norm a NaN or an infinity spoils its block of 128 alone."""
    x = _acts(4, 400, 4)
    x[1, 130] = float("nan")
    x[2, 7] = float("-inf")
    x[3, :128] = 0.0
    x[3, 128:256] = 1e-39                # subnormal
    x[3, 256:] = 3.0e38
    qa = svdq.fp8_quantize_act(x)
    _ok()
    got = qa.codes.float() * plain.spread(qa.scales, 400)
    assert got[1, 128:256].isnan().all() and not got[1, :128].isnan().any() and not got[1, 256:].isnan().any()
    assert got[2, :128].isnan().all() and not got[2, 128:].isnan().any()
    plain.check_codes(qa.codes[[0, 3]], qa.scales[:, [0, 3]], x[[0, 3]].double(), QUANT_DELTA)


def test_strided_rows_in_place_and_sentinels():
    """Column ranges of wider tensors as inputs and as the residual's output;
    in place on x and on the residual; nothing written beside the outputs."""
    M, K = 37, 272
    wide = _acts(M, 1024, 5)
    res = _acts(M, 512, 6)
    w = _acts(1, K, 7).view(-1)
    x, r = wide[:, 256:256 + K], res[:, 16:16 + K]
    v, r64 = plain.norm64(x, w, 1e-5, r)
    codes = torch.full((M * K + 4096,), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((3 * M + 64,), -7.0, device="cuda")
    big = torch.full((M, 640), -3.0, dtype=torch.bfloat16, device="cuda")
    out = svdq.Fp8Act(M, K, codes[:M * K].view(F8).view(M, K), scales[:3 * M].view(3, M))
    qa, ro = svdq.fp8_norm_quantize(x, w, 1e-5, residual=r, out=out, residual_out=big[:, 320:320 + K])
    _ok()
    assert qa is out
    plain.check_codes(qa.codes, qa.scales, v, NORM_DELTA)
    assert torch.equal(ro, r64)
    assert (codes[M * K:] == 0x55).all() and (scales[3 * M:] == -7.0).all()
    assert (big[:, :320] == -3.0).all() and (big[:, 320 + K:] == -3.0).all()
    q2 = svdq.fp8_quantize_act(x)
    plain.check_codes(q2.codes, q2.scales, x.double(), QUANT_DELTA)
    for into in ("x", "residual"):
        xs, rs = wide.clone()[:, 256:256 + K], res.clone()[:, 16:16 + K]
        q3, ro = svdq.fp8_norm_quantize(xs, w, 1e-5, residual=rs, residual_out=xs if into == "x" else rs)
        _ok()
        assert torch.equal(ro, r64) and ro.data_ptr() == (xs if into == "x" else rs).data_ptr()
        assert torch.equal(q3.codes.view(torch.uint8), qa.codes.view(torch.uint8))
        assert torch.equal(q3.scales, qa.scales)


def test_empty_rows():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    qa = svdq.fp8_quantize_act(x)
    assert qa.codes.shape == (0, 256) and qa.scales.shape == (2, 0)
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    qa, r = svdq.fp8_norm_quantize(x, w, 1e-6, residual=x)
    assert r.shape == (0, 256)
    fw = svdq.fp8_pack_weight(torch.ones(256, 64, device="cuda"))
    assert svdq.fp8_linear(qa, fw).shape == (0, 64)
    _ok()


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows as their definition gives."""
    M, K = 132000, 16384
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = _acts(3, K, 8)
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    qa, r = svdq.fp8_norm_quantize(x, w, 1e-6, residual=x)
    _ok()
    v, r64 = plain.norm64(x[-3:], w, 1e-6, x[-3:])
    assert torch.equal(r[-3:], r64)
    plain.check_codes(qa.codes[-3:], qa.scales[:, -3:], v, NORM_DELTA)
    assert (qa.codes[:64].float() == 0).all()


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("K,N", [(16, 8), (128, 128), (144, 200), (2064, 1000), (512, 1032)])
def test_pack_weight(K, N):
    W = 0.02 * torch.randn(K, N, generator=_gen(K + N), device="cuda")
    W[:min(K, 128), :min(N, 128)] *= 30.0
    if K > 128:
        W[128:, :8] = 0.0
    fw = svdq.fp8_pack_weight(W)
    _ok()
    T = W.t().double()
    nb, kb = math.ceil(N / 128), math.ceil(K / 128)
    full = torch.zeros(nb * 128, kb * 128, dtype=torch.float64, device="cuda")
    full[:N, :K] = T
    s = (full.view(nb, 128, kb, 128).abs().amax((1, 3)) / 448.0).clamp_min(plain.MIN_SCALE)
    assert ((fw.scales.double() - s).abs() <= 2.0 ** -23 * s).all()
    q = T / s.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    err = (fw.codes.double() - q).abs()
    assert (err <= 0.5 * plain.e4m3_step(q * (1 + 2.0 ** -20)) + 2.0 ** -21 * q.abs()).all()


# ------------------------------------------------------------------ the product
SHAPES = [
    # few rows
    (1, 16, 8), (1, 128, 128), (1, 4096, 9216), (1, 2064, 1000), (2, 12288, 264), (3, 144, 40), (4, 256, 4096),
    (8, 1040, 1032), (13, 512, 136), (16, 12288, 1024), (17, 4096, 512), (31, 272, 3000), (32, 2048, 2056), (33, 640, 128),
    (48, 1024, 384), (63, 400, 200), (64, 4096, 1280),
    # more rows
    (65, 128, 256), (77, 2064, 1000), (96, 4096, 520), (128, 16, 8), (129, 144, 264), (200, 1040, 264), (256, 256, 256),
    (257, 384, 520), (300, 2048, 776), (511, 128, 1000), (1000, 912, 2048), (1025, 4096, 1288), (2048, 1024, 4096),
]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear(M, K, N):
    """bf16 and fp32 outputs, with and without bias, within the bound that
    counts the roundings; the same bits when called again."""
    G, nb = math.ceil(K / 128), math.ceil(N / 128)
    qa = svdq.Fp8Act(M, K, _codes(M, K, M), _positive(G, M, seed=N))
    w = svdq.Fp8Weight(K, N, _codes(N, K, K), _positive(nb, G, seed=M + 1))
    bias = torch.randn(N, generator=_gen(9), device="cuda").to(torch.bfloat16)
    for b in (bias, None):
        y64, mag = plain.linear64(qa.codes, qa.scales, w.codes, w.scales, b)
        f = svdq.fp8_linear(qa, w, b, out_dtype="f32")
        h = svdq.fp8_linear(qa, w, b)
        _ok()
        assert f.dtype == torch.float32 and h.dtype == torch.bfloat16
        ef, eh = (f.double() - y64).abs(), (h.double() - y64).abs()
        assert (ef <= plain.linear_bound(mag, K)).all(), float((ef / mag.clamp_min(1e-30)).max())
        assert (eh <= plain.linear_bound(mag, K, y64)).all()
        # the fp32 output rounds to the bf16 one
        assert torch.equal(f.to(torch.bfloat16), h)
        assert torch.equal(svdq.fp8_linear(qa, w, b, out_dtype="f32"), f)


@pytest.mark.parametrize("M,K,N", [(1, 1024, 264), (16, 272, 512), (64, 1024, 1000), (130, 1024, 264), (300, 400, 520)])
def test_linear_exact_sums(M, K, N):
    """Whole codes up to 8 and scales that are powers of two: every partial
    sum is a whole number below 2^24 times a power of two near the others', so
    the fp32 result is exact, whatever the order."""
    G, nb = math.ceil(K / 128), math.ceil(N / 128)
    g = _gen(M)
    a = torch.randint(-8, 9, (M, K), generator=g, device="cuda").float().to(F8)
    c = torch.randint(-8, 9, (N, K), generator=g, device="cuda").float().to(F8)
    sa = torch.exp2(torch.randint(-1, 2, (G, M), generator=g, device="cuda").float())
    sw = torch.exp2(torch.randint(-1, 2, (nb, G), generator=g, device="cuda").float())
    y64, _ = plain.linear64(a, sa, c, sw)
    f = svdq.fp8_linear(svdq.Fp8Act(M, K, a, sa), svdq.Fp8Weight(K, N, c, sw), out_dtype="f32")
    _ok()
    assert torch.equal(f.double(), y64)


@pytest.mark.parametrize("M,K,N", [(1, 3600, 9216), (16, 3600, 4480), (7, 3600, 6400), (5, 2064, 5120), (3, 3600, 5120), (2, 640, 1024),
                                   (32, 3600, 9216), (20, 3600, 4480), (31, 3600, 6400), (17, 2064, 5120), (18, 656, 8200),
                                   (64, 4112, 5120), (77, 2064, 1000), (33, 4096, 2048), (100, 1552, 2560), (45, 1680, 3200),
                                   (64, 1936, 1920), (130, 2064, 1000)])
def test_linear_every_split(M, K, N):
    """K in two to eight parts, whose sizes differ and whose tokens do not
    divide evenly among those that add them."""
    test_linear(M, K, N)
    test_linear_exact_sums(M, K, N)


@pytest.mark.parametrize("M", [1, 16, 40, 200])
def test_linear_each_block_has_its_scale(M):
    """One block of K at a time carries a scale, the others 0: a scale taken
    from a neighbouring block, row or column block shows at once."""
    K, N = 656, 392
    G, nb = 6, 4
    a, c = _codes(M, K, 1), _codes(N, K, 2)
    for g in range(G):
        sa, sw = torch.zeros(G, M, device="cuda"), torch.zeros(nb, G, device="cuda")
        sa[g] = torch.arange(1, M + 1, device="cuda") / M
        sw[:, g] = torch.arange(1, nb + 1, device="cuda").float()
        y64, mag = plain.linear64(a, sa, c, sw)
        f = svdq.fp8_linear(svdq.Fp8Act(M, K, a, sa), svdq.Fp8Weight(K, N, c, sw), out_dtype="f32")
        _ok()
        assert ((f.double() - y64).abs() <= plain.linear_bound(mag, K)).all()


@pytest.mark.parametrize("M", [5, 40, 600])
def test_linear_bias_at_any_four_bytes(M):
    """A bias that starts 4, 8 and 12 bytes past a 16-byte boundary, both outputs."""
    K, N = 272, 392
    qa = svdq.Fp8Act(M, K, _codes(M, K, 1), _positive(3, M, seed=2))
    w = svdq.Fp8Weight(K, N, _codes(N, K, 3), _positive(4, 3, seed=4))
    many = torch.randn(N + 8, generator=_gen(5), device="cuda").to(torch.bfloat16)
    for at in (0, 2, 4, 6):
        b = many[at:at + N]
        y64, mag = plain.linear64(qa.codes, qa.scales, w.codes, w.scales, b)
        f, h = svdq.fp8_linear(qa, w, b, out_dtype="f32"), svdq.fp8_linear(qa, w, b)
        _ok()
        assert ((f.double() - y64).abs() <= plain.linear_bound(mag, K)).all()
        assert torch.equal(f.to(torch.bfloat16), h)


def test_two_streams_at_once():
    """Calls of every kernel on two streams, in each other's way: the bits of
    the same calls one after another."""
    K, N = 2064, 1032
    w = svdq.Fp8Weight(K, N, _codes(N, K, 3), _positive(9, 17, seed=4))
    acts = [svdq.Fp8Act(M, K, _codes(M, K, M), _positive(17, M, seed=M + 1)) for M in (1, 20, 70, 300, 3000)]
    x, g = _acts(500, K, 9), torch.ones(K, dtype=torch.bfloat16, device="cuda")
    want = [svdq.fp8_linear(a, w) for a in acts]
    qa, _ = svdq.fp8_norm_quantize(x, g, 1e-6)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for rep in range(20):
        for i, s in enumerate(streams):
            for a in acts[::1 if i else -1]:
                got[i].append(svdq.fp8_linear(a, w, stream=s))
            got[i].append(svdq.fp8_norm_quantize(x, g, 1e-6, stream=s)[0].codes)
    _ok()
    for i in range(2):
        for k, y in enumerate(got[i]):
            k %= 6
            ref = qa.codes if k == 5 else want[k if i else 4 - k]
            assert torch.equal(y.view(torch.uint8), ref.view(torch.uint8))


@pytest.mark.parametrize("M", [1, 20, 64, 130])
def test_linear_nan_stays_in_its_row(M):
    K, N = 400, 264
    a, c = _codes(M, K, 3), _codes(N, K, 4)
    sa, sw = _positive(4, M, seed=5), _positive(3, 4, seed=6)
    bad = M // 2
    sa[2, bad] = float("nan")
    f = svdq.fp8_linear(svdq.Fp8Act(M, K, a, sa), svdq.Fp8Weight(K, N, c, sw))
    _ok()
    assert f[bad].isnan().all()
    rows = [m for m in range(M) if m != bad]
    assert not f[rows].isnan().any()
    a2 = a.clone().view(torch.uint8)
    a2[bad, 399] = 0x7F                  # a NaN code in the short last block
    f = svdq.fp8_linear(svdq.Fp8Act(M, K, a2.view(F8), _positive(4, M, seed=5)), svdq.Fp8Weight(K, N, c, sw))
    _ok()
    assert f[bad].isnan().all() and not f[rows].isnan().any()


@pytest.mark.parametrize("M,N", [(1, 40), (33, 264), (77, 520), (300, 264)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_writes_nothing_past_y(M, N, out):
    K = 272
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    qa = svdq.Fp8Act(M, K, _codes(M, K, 1), _positive(3, M, seed=2))
    w = svdq.Fp8Weight(K, N, _codes(N, K, 3), _positive(math.ceil(N / 128), 3, seed=4))
    want = svdq.fp8_linear(qa, w, out_dtype=out)
    buf = torch.full((M * N + 70000,), -555.0, dtype=dt, device="cuda")
    svdq.fp8_linear(qa, w, out_dtype=out, out=buf[:M * N].view(M, N))
    _ok()
    assert torch.equal(buf[:M * N].view(M, N), want)
    assert (buf[M * N:] == -555.0).all()


def test_linear_offsets_past_32_bits():
    """An output of more than 2^31 elements: its last rows."""
    M, K, N = 70000, 128, 32768
    qa = svdq.Fp8Act(M, K, _codes(M, K, 1), _positive(1, M, seed=2))
    w = svdq.Fp8Weight(K, N, _codes(N, K, 3), _positive(256, 1, seed=4))
    y = svdq.fp8_linear(qa, w)
    _ok()
    for rows in (slice(0, 5), slice(M - 5, M)):
        y64, mag = plain.linear64(qa.codes[rows], qa.scales[:, rows], w.codes, w.scales)
        assert ((y[rows].double() - y64).abs() <= plain.linear_bound(mag, K, y64)).all()


# ------------------------------------------------------------------ streams, graphs, the layer as a whole
def test_streams_and_graph_replay():
    """A call on another stream, two graphs captured apart and replayed in
    turn on new inputs, each with the eager call's bits."""
    K, N = 1040, 520
    fw = svdq.fp8_pack_weight(0.02 * torch.randn(K, N, generator=_gen(1), device="cuda"))
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    for M in (1, 24, 150):
        x, res = _acts(M, K, M), _acts(M, K, M + 1)

        def layer(a, b, stream=None):
            qa, r = svdq.fp8_norm_quantize(a, w, 1e-6, residual=b, stream=stream)
            return svdq.fp8_linear(qa, fw, stream=stream), r

        want, r = layer(x, res)
        torch.cuda.synchronize()
        got, r2 = layer(x, res, stream=side)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(r, r2)
        graphs = []
        for k in range(2):
            sx, sr = torch.zeros_like(x), torch.zeros_like(x)
            layer(sx, sr)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                y = layer(sx, sr)[0]
            graphs.append((g, sx, sr, y))
        for k, (g, sx, sr, y) in enumerate(graphs + graphs[::-1]):
            a, b = _acts(M, K, 50 + k), _acts(M, K, 60 + k)
            sx.copy_(a)
            sr.copy_(b)
            g.replay()
            _ok()
            assert torch.equal(y, layer(a, b)[0])


@pytest.mark.parametrize("M", [1, 7, 64, 200])
def test_block_of_a_transformer(M):
    """The operators as they are used together: residual + norm + 8-bit Q/K/V
    projection + rotary on Q and K (in place in the projection's rows), then
    the 8-bit output projection of the values, residual + norm + 8-bit MLP.
    Each step against 64 bits on the step's own inputs."""
    H, heads, D = 512, 4, 128
    x, res = _acts(M, H, 1), _acts(M, H, 2)
    w1 = _acts(1, H, 3, spread=1.0).view(-1)
    wq = svdq.fp8_pack_weight(0.02 * torch.randn(H, 3 * H, generator=_gen(4), device="cuda"))
    wo = svdq.fp8_pack_weight(0.02 * torch.randn(H, H, generator=_gen(5), device="cuda"))
    wu = svdq.fp8_pack_weight(0.02 * torch.randn(H, 4 * H, generator=_gen(6), device="cuda"))
    bias = _acts(1, 3 * H, 7, spread=1.0).view(-1)
    fr = svdq.rope_freqs(D, scaling="yarn", factor=4.0, original_len=4096)
    pos = torch.arange(M, device="cuda") + 9000

    qa, r = svdq.fp8_norm_quantize(x, w1, 1e-6, residual=res)
    qkv = svdq.fp8_linear(qa, wq, bias)
    before = qkv.clone()
    svdq.rope_apply(qkv, 2 * heads, D, pos, fr, layout="half")
    va = svdq.fp8_quantize_act(qkv[:, 2 * H:])
    o = svdq.fp8_linear(va, wo)
    qb, r2 = svdq.fp8_norm_quantize(o, w1, 1e-6, residual=r, residual_out=r.clone())
    u = svdq.fp8_linear(qb, wu, out_dtype="f32")
    _ok()

    v, r64 = plain.norm64(x, w1, 1e-6, res)
    assert torch.equal(r, r64)
    plain.check_codes(qa.codes, qa.scales, v, NORM_DELTA)
    y64, mag = plain.linear64(qa.codes, qa.scales, wq.codes, wq.scales, bias)
    assert ((before.double() - y64).abs() <= plain.linear_bound(mag, H, y64)).all()
    t = plain.angles64(pos, fr.freq)
    z64, zmag = plain.rope64(before, 2 * heads, D, t, fr.factor, "half")
    assert ((qkv[:, :2 * H].double() - z64).abs()
            <= (plain.TABLE_TOL + 2.0 ** -23) * fr.factor * zmag + 2.0 ** -8 * z64.abs()).all()
    assert torch.equal(qkv[:, 2 * H:], before[:, 2 * H:])
    plain.check_codes(va.codes, va.scales, before[:, 2 * H:].double(), QUANT_DELTA)
    y64, mag = plain.linear64(va.codes, va.scales, wo.codes, wo.scales)
    assert ((o.double() - y64).abs() <= plain.linear_bound(mag, H, y64)).all()
    v, r64 = plain.norm64(o, w1, 1e-6, r)
    assert torch.equal(r2, r64)
    plain.check_codes(qb.codes, qb.scales, v, NORM_DELTA)
    y64, mag = plain.linear64(qb.codes, qb.scales, wu.codes, wu.scales)
    assert ((u.double() - y64).abs() <= plain.linear_bound(mag, H)).all()


@pytest.mark.parametrize("M", [1, 16, 64, 700])
def test_captured_layers_give_the_bits_of_single_calls(M):
    """Norm, linear, rotary in place, quantise, linear, three times over, each
    on the previous one's output: a replayed graph, whose kernels start before
    their predecessors end, against calls with a wait after each."""
    D, F = 1024, 2560
    pk = []
    for i in range(3):
        g = _gen(20 + i)
        pk.append((svdq.fp8_pack_weight(torch.randn(D, F, generator=g, device="cuda") / 32),
                   svdq.fp8_pack_weight(torch.randn(F, D, generator=g, device="cuda") / 50)))
    w = torch.ones(D, device="cuda", dtype=torch.bfloat16)
    fr, pos = svdq.rope_freqs(128), torch.arange(M, device="cuda") + 5

    def layers(h, r, wait):
        for a, b in pk:
            qa, r = svdq.fp8_norm_quantize(h, w, 1e-6, residual=r, residual_out=r)
            wait()
            u = svdq.fp8_linear(qa, a)
            wait()
            svdq.rope_apply(u, F // 128, 128, pos, fr, layout="half")
            wait()
            qu = svdq.fp8_quantize_act(u)
            wait()
            h = svdq.fp8_linear(qu, b)
            wait()
        return h, r

    sh, sr = _acts(M, D, 1), _acts(M, D, 2)
    layers(sh, sr, lambda: None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oh, orr = layers(sh, sr, lambda: None)
    for it in range(20):
        h, r = _acts(M, D, 100 + it), _acts(M, D, 200 + it)
        sh.copy_(h)
        sr.copy_(r)
        graph.replay()
        eh, er = layers(h, r, torch.cuda.synchronize)
        _ok()
        assert torch.equal(eh, oh) and torch.equal(er, orr)
