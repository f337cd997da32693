"""The 8-bit linear path and the rotary positions, as calls to be measured.

Three operators, each in its plain form (elementary torch operations in 32
bits) and, where ``own`` is set, through the package's entry points:

- "norm" / "quantize": root-mean-square norm with the residual's addition and
  an E4M3 output with one fp32 scale per 128 columns of a row; the same output
  without the norm for inputs that are not normed.
- "linear": the product of two E4M3 operands whose scales cover 1 x 128
  (activations) and 128 x 128 (weights) blocks, with bias.
- "rope" / "tables": rotary positions applied to the heads of a projection's
  output, and the cos/sin tables alone (the fused Q/K/V epilogue takes them).
"""

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126


def listed():
    return [
        # one token of a decoding step: residual added, normed, quantised for the next projection
        dict(name="norm 1x4096 residual", op="norm", M=1, H=4096, residual=True),
        # the tokens of a 1024 x 1024 image and its prompt, between two blocks
        dict(name="norm 4608x4096 residual", op="norm", M=4608, H=4096, residual=True),
        # a text encoder's ragged prompt; the last group has 16 columns
        dict(name="quantize 77x1040", op="quantize", M=77, H=1040),
        # the hidden activations of an MLP ahead of its down-projection
        dict(name="quantize 4608x12288", op="quantize", M=4608, H=12288),
        # one token through the grouped Q/K/V projection
        dict(name="linear 1x4096x9216", op="linear", M=1, K=4096, N=9216, bias=True, out="bf16"),
        # a decoding batch through an MLP's down-projection
        dict(name="linear 16x12288x4096", op="linear", M=16, K=12288, N=4096, bias=False, out="bf16"),
        # a ragged prompt, odd output width, a tail of K, unrounded output
        dict(name="linear 77x2064x1000 f32", op="linear", M=77, K=2064, N=1000, bias=True, out="f32"),
        # an image's tokens through an MLP's up-projection
        dict(name="linear 4608x4096x12288", op="linear", M=4608, K=4096, N=12288, bias=True, out="bf16"),
        # a long prompt through a wide square projection
        dict(name="linear 8192x8192x8192", op="linear", M=8192, K=8192, N=8192, bias=False, out="bf16"),
        # one token far into a long context, 40 query and 8 key heads
        dict(name="rope 1x48x128 half", op="rope", M=1, heads=48, head_dim=128, rot=128, layout="half",
             scaling="yarn", span=1 << 20, row=7168),
        # the Q and K sections of a long prompt's Q/K/V rows; half of the head is rotated
        dict(name="rope 16384x64x128 part", op="rope", M=16384, heads=64, head_dim=128, rot=64,
             layout="interleaved", scaling="linear", span=1 << 17, row=12288),
        # the tables of an image's tokens: three position axes (frame, row, column) and a prompt
        dict(name="tables 4608x64 3 axes", op="tables", M=4608, rot=128, axes=3, span=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "linear", "linear", "rope", "rope", "tables"])
    if op in ("norm", "quantize"):
        H = 16 * _log(rng, 8, 1024)
        M = min(_log(rng, 1, 16384), (4608 * 12288) // H)
        return dict(op="norm", M=M, H=H, residual=rng.random() < 0.6) if op == "norm" else dict(op=op, M=M, H=H)
    if op == "linear":
        K, N = 16 * _log(rng, 8, 1024), 8 * _log(rng, 8, 2048)
        M = min(_log(rng, 1, 9000), 8192 * 8192 * 8192 // (K * N))
        return dict(op=op, M=M, K=K, N=N, bias=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "rope":
        D = rng.choice([32, 64, 80, 96, 128, 192, 256])
        rot = rng.choice([D, D, D // 2])
        heads = _log(rng, 1, 96)
        row = heads * D + rng.choice([0, 8, D, heads * D // 2 // 8 * 8])
        M = min(_log(rng, 1, 16384), 16384 * 12288 // row)
        return dict(op=op, M=M, heads=heads, head_dim=D, rot=rot, layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), span=1 << rng.randint(10, 21), row=row)
    return dict(op=op, M=_log(rng, 1, 65536), rot=rng.choice([32, 64, 96, 128]), axes=rng.choice([1, 2, 3]),
                span=1 << rng.randint(8, 20))


def _inverse_frequencies(rot, base, scaling, factor, original):
    """Turns per position of the rot / 2 pairs, in 64 bits, and the factor on
    cos and sin. linear: positions shrink by the factor; ntk: the base grows so
    that the slowest pair shrinks by it; yarn: pairs with fewer than 1 turn in
    the original length shrink, those with more than 32 stay, a ramp between."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        def at(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        keep = 1.0 - ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f / factor * (1.0 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _groups(v):
    """[M, H] in groups of 128 columns, the last one filled with zeros: [M, G, 128]."""
    H = v.shape[1]
    pad = -H % BLOCK
    return torch.nn.functional.pad(v, (0, pad)).view(v.shape[0], (H + pad) // BLOCK, BLOCK)


def _quantised(v):
    """E4M3 codes [M, H] and scales [G, M] of v."""
    g = _groups(v)
    s = (g.abs().amax(2) / E4M3_MAX).clamp_min(MIN_SCALE)
    q = (g / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(v.shape[0], -1)[:, :v.shape[1]]
    return q.contiguous().to(torch.float8_e4m3fn), s.t().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def activations(M, K):
        # one channel in a hundred is an outlier, as in a transformer's residual stream
        wide = torch.rand(K, generator=gen, device=dev) < 0.01
        return (normal(M, K) * torch.where(wide, 20.0, 1.0)).to(torch.bfloat16)

    op, s = case["op"], dict(op=case["op"])
    if op in ("norm", "quantize"):
        s["x"] = activations(case["M"], case["H"])
        if op == "norm":
            s["w"] = (1.0 + 0.2 * normal(case["H"])).to(torch.bfloat16)
            s["eps"] = 1e-6
            s["residual"] = activations(case["M"], case["H"]) if case["residual"] else None
    elif op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        s["a"], s["sa"] = _quantised(activations(M, K).float())
        W = 0.02 * normal(N, K)
        nb, kb = -(-N // BLOCK), -(-K // BLOCK)
        W = torch.nn.functional.pad(W, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(nb, BLOCK, kb, BLOCK)
        s["sw"] = (W.abs().amax((1, 3)) / E4M3_MAX).clamp_min(MIN_SCALE)
        W = (W / s["sw"][:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(nb * BLOCK, kb * BLOCK)
        s["w"] = W[:N, :K].contiguous().to(torch.float8_e4m3fn)
        s["bias"] = (0.1 * normal(N)).to(torch.bfloat16) if case["bias"] else None
        s["out"] = case["out"]
    elif op == "rope":
        s["x"] = normal(case["M"], case["row"]).to(torch.bfloat16)
        first = int(torch.randint(0, case["span"], (1,), generator=gen, device=dev))
        s["pos"] = torch.arange(case["M"], device=dev) + first
        f, s["factor"] = _inverse_frequencies(case["rot"], 10000.0, case["scaling"], 8.0, 8192)
        s["freq"] = f.to(dev)
        s.update(heads=case["heads"], head_dim=case["head_dim"], rot=case["rot"], layout=case["layout"])
        s["y"] = torch.empty(case["M"], case["heads"] * case["head_dim"], dtype=torch.bfloat16, device=dev)
    else:
        s["pos"] = torch.randint(0, case["span"], (case["M"], case["axes"]), generator=gen, device=dev)
        pairs = case["rot"] // 2
        # each axis has its own share of the pairs, and its own run of frequencies
        share = [pairs // case["axes"]] * (case["axes"] - 1)
        share.append(pairs - sum(share))
        s["axis"] = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(share)).to(dev, torch.int32)
        s["freq"] = torch.cat([_inverse_frequencies(2 * n, 10000.0, "none", 1.0, 8192)[0] for n in share]).to(dev)
        s["factor"] = 1.0
    return s


def _angles(s):
    pos = s["pos"].double()
    pos = pos[:, None] if pos.dim() == 1 else pos[:, s["axis"].long()]
    return pos * s["freq"][None, :]


def _dequantised(s):
    """Both operands of a linear layer as fp32 values."""
    M, K = s["a"].shape
    N = s["w"].shape[0]
    sa = s["sa"].t().repeat_interleave(BLOCK, 1)[:, :K]
    sw = s["sw"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return s["a"].float() * sa, s["w"].float() * sw


def _rotated(x, c, n, s):
    """The heads of x [M, row] with the first rot columns of each rotated by cos c, sin n [M, rot / 2]."""
    M, H, D, R = x.shape[0], s["heads"], s["head_dim"], s["rot"]
    h = x[:, :H * D].view(M, H, D)
    c, n = c[:, None, :], n[:, None, :]
    if s["layout"] == "half":
        a, b = h[:, :, :R // 2], h[:, :, R // 2:R]
        turned = torch.cat([a * c - b * n, a * n + b * c], 2)
    else:
        a, b = h[:, :, 0:R:2], h[:, :, 1:R:2]
        turned = torch.stack([a * c - b * n, a * n + b * c], 3).flatten(2)
    return torch.cat([turned, h[:, :, R:]], 2).reshape(M, H * D)


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _quantised(s["x"].float())
    if op == "norm":
        r = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
        f = r.float()
        v = f * torch.rsqrt((f * f).mean(1, keepdim=True) + s["eps"]) * s["w"].float()
        q, sc = _quantised(v)
        return (q, sc) if s["residual"] is None else (q, sc, r)
    if op == "linear":
        a, w = _dequantised(s)
        y = a @ w.t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return y if s["out"] == "f32" else y.to(torch.bfloat16)
    # angles of far positions: 64 bits
    t = _angles(s)
    c, n = (t.cos() * s["factor"]).float(), (t.sin() * s["factor"]).float()
    if op == "tables":
        return c, n
    return _rotated(s["x"].float(), c, n, s).to(torch.bfloat16)


def _own(s):
    import bit_w4a4_quantized_nvfp4_b200 as svdq

    op = s["op"]
    if op == "quantize":
        qa = svdq.fp8_quantize_act(s["x"])
        return qa.codes, qa.scales
    if op == "norm":
        qa, r = svdq.fp8_norm_quantize(s["x"], s["w"], s["eps"], residual=s["residual"])
        return (qa.codes, qa.scales) if r is None else (qa.codes, qa.scales, r)
    if op == "linear":
        qa = svdq.Fp8Act(s["a"].shape[0], s["a"].shape[1], s["a"], s["sa"])
        w = svdq.Fp8Weight(s["w"].shape[1], s["w"].shape[0], s["w"], s["sw"])
        return svdq.fp8_linear(qa, w, s["bias"], out_dtype=s["out"])
    if op == "tables":
        return svdq.rope_tables(s["pos"], svdq.RopeFreqs(s["freq"], s["factor"], s["axis"]))
    return svdq.rope_apply(s["x"], s["heads"], s["head_dim"], s["pos"], svdq.RopeFreqs(s["freq"], s["factor"]),
                           layout=s["layout"], out=s["y"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, M = case["op"], case["M"]
    if op in ("norm", "quantize"):
        H = case["H"]
        b = M * H * 3 + 4 * M * -(-H // BLOCK)
        if op == "norm":
            b += 2 * H + (4 * M * H if case["residual"] else 0)
        return {"bytes": b, "flops": 8 * M * H}
    if op == "linear":
        K, N = case["K"], case["N"]
        kb = -(-K // BLOCK)
        b = M * K + N * K + 4 * M * kb + 4 * kb * -(-N // BLOCK) + M * N * (4 if case["out"] == "f32" else 2)
        return {"bytes": b + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if op == "rope":
        b = 4 * M * case["heads"] * case["head_dim"] + 8 * M + 4 * case["rot"]
        return {"bytes": b, "flops": 3 * M * case["heads"] * case["rot"]}
    return {"bytes": 4 * M * case["rot"] + 8 * M * case["axes"] + 6 * case["rot"], "flops": 10 * M * case["rot"]}


def exact(case, seed):
    """The definitions in 64 bits: what is rounded to 8 or 16 bits at the end
    is given before that rounding; the residual's sum is rounded to bf16 where
    the norm reads it, since that is the value the operator stores and norms."""
    s = prepare(case, seed)
    op = s["op"]
    if op in ("norm", "quantize"):
        v, r = s["x"].double(), None
        if op == "norm":
            if s["residual"] is not None:
                r = v + s["residual"].double()
                v = r.to(torch.bfloat16).double()
            v = v / ((v ** 2).sum(1, keepdim=True) / v.shape[1] + s["eps"]).sqrt() * s["w"].double()
        M, H = v.shape
        q, scales = torch.empty_like(v), []
        for k in range(0, H, BLOCK):
            part = v[:, k:k + BLOCK]
            scale = torch.clamp(part.abs().max(1).values / E4M3_MAX, min=MIN_SCALE)
            q[:, k:k + BLOCK] = part / scale[:, None]
            scales.append(scale)
        return (q, torch.stack(scales)) if r is None else (q, torch.stack(scales), r)
    if op == "linear":
        M, K = s["a"].shape
        N = s["w"].shape[0]
        y = torch.zeros(M, N, dtype=torch.float64, device=s["a"].device)
        for g in range(-(-K // BLOCK)):
            cols = slice(g * BLOCK, min(K, (g + 1) * BLOCK))
            part = s["a"][:, cols].double() @ s["w"][:, cols].double().t()
            rows = s["sw"][:, g].double().repeat_interleave(BLOCK)[:N]
            y += part * s["sa"][g].double()[:, None] * rows[None, :]
        return y if s["bias"] is None else y + s["bias"].double()
    pos = s["pos"].double()
    if op == "tables":
        t = torch.stack([pos[:, int(a)] for a in s["axis"]], 1) * s["freq"]
        return torch.cos(t) * s["factor"], torch.sin(t) * s["factor"]
    t = torch.outer(pos, s["freq"])
    c, n = torch.cos(t) * s["factor"], torch.sin(t) * s["factor"]
    H, D, R = s["heads"], s["head_dim"], s["rot"]
    y = s["x"][:, :H * D].double().reshape(-1, H, D).clone()
    half = s["layout"] == "half"
    for i in range(R // 2):
        p, q = (i, i + R // 2) if half else (2 * i, 2 * i + 1)
        a, b = y[:, :, p].clone(), y[:, :, q].clone()
        y[:, :, p] = a * c[:, i, None] - b * n[:, i, None]
        y[:, :, q] = a * n[:, i, None] + b * c[:, i, None]
    return y.reshape(-1, H * D)
