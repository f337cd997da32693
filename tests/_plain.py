"""The 8-bit layer and the rotary positions in 64 bits, as the tests' plain
implementation, and error bounds that follow from the kernels' roundings.
Nothing here is shared with the package."""

from __future__ import annotations

import math

import torch

BLOCK = 128
MIN_SCALE = 2.0 ** -126


def norm64(x, weight, eps, residual=None):
    """(v, r): r = bf16(x + residual) and its RMS norm in 64 bits."""
    r = x
    if residual is not None:
        r = (x.double() + residual.double()).to(torch.bfloat16)
    d = r.double()
    return d / (d.square().mean(1, keepdim=True) + eps).sqrt() * weight.double(), r


def scales64(v):
    """[G, M] of v [M, K]: max(max|v| / 448, 2^-126) per 128 columns (NaN where a group holds one)."""
    out = []
    for k in range(0, v.shape[1], BLOCK):
        out.append((v[:, k:k + BLOCK].abs().amax(1) / 448.0).clamp_min(MIN_SCALE))
    return torch.stack(out)


def spread(scales, K):
    """scales [G, M] -> [M, K]"""
    return scales.t().repeat_interleave(BLOCK, 1)[:, :K]


def e4m3_step(q):
    """Spacing of the E4M3 values around q: 2^(e-3), 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6)))
    return torch.exp2(e - 3)


def check_codes(codes, scales, v, delta):
    """codes/scales of v (64 bits): the scale within delta of the definition's,
    the code within half a step of v / scale (delta more for v's own error).
    At a binade's border the step above is taken, since v's error may cross it."""
    K = v.shape[1]
    s = scales64(v)
    assert scales.shape == s.shape
    assert ((scales.double() - s).abs() <= delta * s).all()
    q = v / spread(s, K)
    c = codes.double()
    err = (c - q).abs()
    bound = 0.5 * e4m3_step(q * (1 + 4 * delta)) + 4 * delta * q.abs()
    assert (err <= bound).all(), float((err - bound).max())


def linear64(qa_codes, qa_scales, w_codes, w_scales, bias=None):
    """(y, mag): the 8-bit product in 64 bits and the sum of its terms' magnitudes."""
    a, w = qa_codes.double(), w_codes.double()
    M, K = a.shape
    N = w.shape[0]
    y = torch.zeros(M, N, dtype=torch.float64, device=a.device)
    mag = torch.zeros_like(y)
    for g in range(math.ceil(K / BLOCK)):
        c = slice(g * BLOCK, min(K, (g + 1) * BLOCK))
        s = qa_scales[g].double()[:, None] * w_scales[:, g].double().repeat_interleave(BLOCK)[:N][None, :]
        y += s * (a[:, c] @ w[:, c].t())
        mag += s.abs() * (a[:, c].abs() @ w[:, c].abs().t())
    if bias is not None:
        y += bias.double()
        mag += bias.double().abs()
    return y, mag


def linear_bound(mag, K, y=None):
    """Products of E4M3 codes are exact in fp32. A block's sum has up to 128
    additions in the tensor core (each off by at most 2^-23 of the sum of
    magnitudes, truncation included); scaling and adding the blocks, split
    over up to 8 partial sums, takes three roundings of 2^-24 per block and 8
    more. bf16 outputs add half a step, 2^-8 |y|."""
    G = math.ceil(K / BLOCK)
    b = (128 * 2.0 ** -23 + (3 * G + 16) * 2.0 ** -24) * mag
    return b if y is None else b + 2.0 ** -8 * (y.abs() + b)


def angles64(pos, freq, axis=None):
    pos = pos[:, None] if pos.dim() == 1 else pos
    cols = torch.zeros(freq.shape[0], dtype=torch.long, device=pos.device) if axis is None else axis.long()
    return pos.double()[:, cols] * freq[None, :]


def rope64(x, heads, head_dim, t, factor, layout):
    """Heads of x [M, >= heads * head_dim] rotated by angles t [M, pairs], in 64 bits."""
    P = t.shape[1]
    y = x[:, :heads * head_dim].double().reshape(x.shape[0], heads, head_dim).clone()
    i = torch.arange(P, device=x.device)
    p, q = (i, i + P) if layout == "half" else (2 * i, 2 * i + 1)
    a, b = y[:, :, p].clone(), y[:, :, q].clone()
    c, s = torch.cos(t)[:, None, :] * factor, torch.sin(t)[:, None, :] * factor
    y[:, :, p] = a * c - b * s
    y[:, :, q] = a * s + b * c
    mag = torch.zeros_like(y)
    mag[:, :, p] = a.abs() + b.abs()
    mag[:, :, q] = a.abs() + b.abs()
    return y.reshape(x.shape[0], -1), mag.reshape(x.shape[0], -1)


# cos and sin: the reduced angle rounded to fp32 (half a step of at most pi:
# 2^-23), the fp32 function (2 steps of at most 1: 2^-23), the factor (2^-24)
TABLE_TOL = 2.0 ** -23 + 2.0 ** -23 + 2.0 ** -24
