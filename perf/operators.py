"""The microscaled (MX) operators of the layer, as cases to measure.

Four operators that a program serving a Mixture-of-Experts layer with 4-bit expert
weights calls one after the other:

  norm   residual addition and root-mean-square norm, with the normalised rows also in
         E4M3 with one E8M0 scale per 32 columns (the layer's input)
  quant  microscaled quantisation of a matrix, to E2M1 (expert weights) or E4M3 (tokens)
  mm     products grouped by expert: E4M3 rows in expert order times E2M1 weights
  ffn    the grouped expert FFN on such operands: w13, SwiGLU, E4M3 again, w2

An MX block is 32 consecutive elements of a row with the scale 2^(code - 127).  The
scale of a block with largest magnitude m is 2^(floor(log2 m) - e), clamped to
2^-127 .. 2^127, with e = 2 for E2M1 and e = 8 for E4M3; elements are rounded to the nearest
value (ties to even) and saturate.  E2M1 codes lie two to a byte, the lower column in
the low nibble.

`own` false: the operators written with elementary torch operations.  `own` true: the
library's entry points.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
_MX4_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decoding step of 8 sequences: the smallest call, where latency counts
        {"name": "norm_decode", "op": "norm", "T": 8, "H": 2048, "residual": True, "mx": True},
        # a step of 64 sequences of a wide layer
        {"name": "norm_wide", "op": "norm", "T": 64, "H": 7168, "residual": True, "mx": True},
        # a prompt of 8192 tokens
        {"name": "norm_prefill", "op": "norm", "T": 8192, "H": 4096, "residual": True, "mx": True},
        # the down projections of one layer's experts, once at load time
        {"name": "quant_weights", "op": "quant", "rows": 128 * 2048, "cols": 768,
         "dtype": "bfloat16", "fmt": "e2m1"},
        # token rows of a layer whose norm is not fused, an odd number of them
        {"name": "quant_tokens", "op": "quant", "rows": 1237, "cols": 4128,
         "dtype": "bfloat16", "fmt": "e4m3"},
        # one product over a decoding step's 64 routed rows
        {"name": "mm_decode", "op": "mm", "R": 64, "E": 128, "N": 2048, "K": 768, "zipf": 0.0},
        # ragged groups, some of them empty, with a hot expert; N no multiple of a tile
        {"name": "mm_ragged", "op": "mm", "R": 1999, "E": 37, "N": 1160, "K": 640, "zipf": 1.2},
        # one product over a prompt's routed rows
        {"name": "mm_prefill", "op": "mm", "R": 65536, "E": 128, "N": 4096, "K": 1536, "zipf": 0.0},
        # a single token
        {"name": "ffn_token", "op": "ffn", "T": 1, "E": 128, "k": 8, "H": 2048, "I": 768,
         "zipf": 0.0},
        # a decoding step of 8 sequences
        {"name": "ffn_decode", "op": "ffn", "T": 8, "E": 128, "k": 8, "H": 2048, "I": 768,
         "zipf": 0.0},
        # 64 sequences, skewed routing, a wide layer of 256 experts
        {"name": "ffn_skewed", "op": "ffn", "T": 64, "E": 256, "k": 8, "H": 7168, "I": 2048,
         "zipf": 1.2},
        # a prompt of 8192 tokens
        {"name": "ffn_prefill", "op": "ffn", "T": 8192, "E": 128, "k": 8, "H": 4096, "I": 1536,
         "zipf": 0.0},
    ]


def _log(rng, lo, hi):
    """An integer of lo .. hi, uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "mm", "ffn"])
    if op == "norm":
        H = 32 * _log(rng, 4, 256)
        return {"op": op, "T": _log(rng, 1, 33_000_000 // H), "H": H,
                "residual": rng.random() < 0.75, "mx": rng.random() < 0.75}
    if op == "quant":
        cols = 32 * _log(rng, 1, 256)
        return {"op": op, "rows": _log(rng, 1, 100_000_000 // cols), "cols": cols,
                "dtype": rng.choice(["bfloat16", "float32"]), "fmt": rng.choice(["e2m1", "e4m3"])}
    if op == "mm":
        K, N = 128 * _log(rng, 1, 32), 8 * _log(rng, 1, 640)
        E, zipf = _log(rng, 1, min(256, 800_000_000 // (N * K))), rng.choice([0.0, 0.6, 1.2])
        R = _log(rng, 1, 4096 if zipf else 16384)
        return {"op": op, "R": R, "E": E, "N": N, "K": K, "zipf": zipf}
    H, I = 128 * _log(rng, 1, 40), 128 * _log(rng, 1, 16)
    E = _log(rng, 1, min(256, 800_000_000 // (H * I)))
    k = rng.randint(1, min(E, 8))
    return {"op": op, "T": _log(rng, 1, 2048), "E": E, "k": k, "H": H, "I": I,
            "zipf": rng.choice([0.0, 0.0, 1.2])}


# ------------------------------------------------------------------ inputs


def _generator(seed, device=None):
    return torch.Generator(device=device or DEVICE).manual_seed(int(seed) * 1009 + 17)


def _zipf(E, s):
    p = torch.arange(1, E + 1, dtype=torch.float64).pow(-s)
    return p / p.sum()


def _routing(case, seed, device=None):
    """(expert_offsets [E + 1], permuted_rows [T k]) int32 of T tokens that each pick the k
    experts with the largest N(0, 1) logits (plus the logarithm of a Zipf weight)."""
    g = _generator(seed, device)
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, generator=g, device=g.device)
    if case["zipf"]:
        logits += 2 * torch.log(_zipf(E, case["zipf"])).to(g.device, torch.float32)
    ids = torch.topk(logits, k, dim=1).indices.flatten()
    rows = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E)
    return _offsets(counts), rows.to(torch.int32)


def _groups(case, seed, device=None):
    """expert_offsets int32 [E + 1] of R rows, each of an expert drawn by its Zipf weight."""
    g = _generator(seed, device)
    p = _zipf(case["E"], case["zipf"]).to(g.device, torch.float32)
    ids = torch.multinomial(p, case["R"], replacement=True, generator=g)
    return _offsets(torch.bincount(ids, minlength=case["E"]))


def _offsets(counts):
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def _draw_mx(g, fmt, shape, std):
    """MX codes and scales of an N(0, std^2) matrix, drawn a part at a time."""
    lead, cols = shape[:-1], shape[-1]
    parts = lead[0] if len(lead) > 1 else 1
    codes = torch.empty(*lead, cols // 2 if fmt == "e2m1" else cols, dtype=torch.uint8, device=DEVICE)
    scales = torch.empty(*lead, cols // 32, dtype=torch.uint8, device=DEVICE)
    for i in range(parts):
        part = lead[1:] if len(lead) > 1 else lead
        v = torch.randn(*part, cols, generator=g, device=DEVICE) * std
        c, s = _quantize(v.to(torch.bfloat16).float(), fmt)
        at = (i,) if len(lead) > 1 else ()
        codes[at + (...,)] = c
        scales[at + (...,)] = s
    return codes, scales


def prepare(case, seed):
    g = _generator(seed + 7_000_003)
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        x = torch.randn(T, H, generator=g, device=DEVICE).to(torch.bfloat16)
        res = (4 * torch.randn(T, H, generator=g, device=DEVICE)).to(torch.bfloat16)
        w = (1 + 0.2 * torch.randn(H, generator=g, device=DEVICE)).to(torch.bfloat16)
        return {"op": op, "x": x, "residual": res if case["residual"] else None, "weight": w,
                "mx": case["mx"]}
    if op == "quant":
        src = torch.randn(case["rows"], case["cols"], generator=g, device=DEVICE)
        # rows of different sizes, as weights and activations have
        src *= torch.exp(torch.randn(case["rows"], 1, generator=g, device=DEVICE))
        return {"op": op, "src": src.to(getattr(torch, case["dtype"])), "fmt": case["fmt"]}
    if op == "mm":
        R, E, N, K = case["R"], case["E"], case["N"], case["K"]
        a, sa = _draw_mx(g, "e4m3", (R, K), 1.0)
        w, sw = _draw_mx(g, "e2m1", (E, N, K), 1 / math.sqrt(K))
        return {"op": op, "a": a, "a_scale": sa, "w": w, "w_scale": sw,
                "offsets": _groups(case, seed), "pairs": _pairs()}
    T, E, H, I = case["T"], case["E"], case["H"], case["I"]
    x, sx = _draw_mx(g, "e4m3", (T, H), 1.0)
    w13, s13 = _draw_mx(g, "e2m1", (E, 2 * I, H), 1 / math.sqrt(H))
    w2, s2 = _draw_mx(g, "e2m1", (E, H, I), 1 / math.sqrt(I))
    offsets, rows = _routing(case, seed)
    return {"op": op, "x": x, "x_scale": sx, "w13": w13, "w13_scale": s13, "w2": w2,
            "w2_scale": s2, "offsets": offsets, "rows": rows, "k": case["k"], "pairs": _pairs()}


# ------------------------------------------------------------------ plain forms


def _largest(v, emax):
    """E8M0 scale codes of fp32 blocks [..., 32]: floor(log2 of the largest magnitude) - emax."""
    m = v.abs().amax(dim=-1)
    e = torch.frexp(m).exponent - 1 - emax
    e = torch.where(m > 0, e, torch.full_like(e, -127))
    return (e.clamp(-127, 127) + 127).to(torch.uint8)


def _power(codes):
    """2^(code - 127) in fp32 of E8M0 codes; 255 is NaN."""
    bits = codes.int() << 23
    bits = torch.where(codes == 0, 1 << 22, bits)  # 2^-127 is subnormal in fp32
    return torch.where(codes == 255, 0x7FC00000, bits).view(torch.float32)


def _pairs():
    """fp32 [256, 2]: the two E2M1 values of each byte."""
    one = list(_MX4_LEVELS) + [-x for x in _MX4_LEVELS]
    return torch.tensor([[one[c & 15], one[c >> 4]] for c in range(256)], device=DEVICE)


def _quantize(v, fmt):
    """(codes, scale codes) of an fp32 matrix, MX blocks along the last dimension."""
    b = v.unflatten(-1, (-1, 32))
    scales = _largest(b, 2 if fmt == "e2m1" else 8)
    u = b / _power(scales).unsqueeze(-1)
    if fmt == "e4m3":
        codes = u.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return codes.flatten(-2), scales
    a = u.abs()
    # ties go to the even code: up at 0.75, 1.75 and 3.5, down at the other midpoints
    n = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
         + (a >= 3.5) + (a > 5)).to(torch.uint8)
    n += torch.signbit(u).to(torch.uint8) * 8
    n = n.flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), scales


def _values8(codes, scales):
    """fp32 values of E4M3 codes [..., cols] with their scales."""
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return (v * _power(scales).unsqueeze(-1)).flatten(-2)


def _values4(pairs, codes, scales):
    """fp32 values of E2M1 codes [..., cols / 2] with their scales."""
    v = pairs[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    return v.mul_(_power(scales).unsqueeze(-1)).flatten(-2)


def _grouped(pairs, a, w, w_scale, offsets):
    """fp32 [R, N]: the rows offsets[e] .. offsets[e + 1] of a times w[e] transposed, as one
    batched product over the experts that have rows, padded to the longest group."""
    counts = offsets[1:] - offsets[:-1]
    used = torch.nonzero(counts).flatten()
    n = counts[used]
    slot = torch.arange(int(n.max()), device=a.device, dtype=torch.int32)
    live = slot < n[:, None]
    at = offsets[:-1][used][:, None] + slot
    rows = a[torch.where(live, at, torch.zeros_like(at))]
    y = torch.bmm(rows, _values4(pairs, w[used], w_scale[used]).transpose(1, 2))
    out = torch.empty(a.shape[0], w.shape[1], device=a.device)
    out[at[live]] = y[live]
    return out


def _plain_norm(s):
    x = s["x"].float()
    h = None
    if s["residual"] is not None:
        h = (x + s["residual"].float()).to(torch.bfloat16)
        x = h.float()
    n = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * s["weight"].float()
    codes, scales = _quantize(n, "e4m3") if s["mx"] else (None, None)
    return h, n.to(torch.bfloat16), codes, scales


def _plain_ffn(s):
    H, I = s["x"].shape[1], s["w2"].shape[2] * 2
    rows = s["rows"].long()
    x = _values8(s["x"], s["x_scale"])[rows // s["k"]]
    h = _grouped(s["pairs"], x, s["w13"], s["w13_scale"], s["offsets"])
    gate, up = h[:, :I], h[:, I:]
    act = gate / (1 + torch.exp(-gate)) * up
    act = _values8(*_quantize(act, "e4m3"))
    y = torch.empty(rows.numel(), H, dtype=torch.bfloat16, device=x.device)
    y[rows] = _grouped(s["pairs"], act, s["w2"], s["w2_scale"], s["offsets"]).to(torch.bfloat16)
    return y


# ------------------------------------------------------------------ one pass


def _mx8(codes, scales):
    """E4M3 codes and E8M0 scales as the values that they hold."""
    if codes is None:
        return None, None
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def run(s):
    op = s["op"]
    if own:
        import mixture_experts_layer_logits_b200 as moe

        if op == "norm":
            h, n, codes, scales = moe.moe_add_rmsnorm(s["x"], s["weight"], EPS,
                                                      residual=s["residual"], quantize=s["mx"])
        elif op == "quant":
            codes, scales = moe.moe_quantize_mx(s["src"], s["fmt"])
        elif op == "mm":
            return moe.moe_grouped_mm_mx4(s["a"], s["a_scale"], s["w"], s["w_scale"], s["offsets"])
        else:
            return moe.moe_grouped_ffn_mx4(s["x"], s["x_scale"], s["w13"], s["w13_scale"], s["w2"],
                                           s["w2_scale"], s["offsets"], s["rows"], s["k"])
    elif op == "norm":
        h, n, codes, scales = _plain_norm(s)
    elif op == "quant":
        codes, scales = _quantize(s["src"].float(), s["fmt"])
    elif op == "mm":
        return _grouped(s["pairs"], _values8(s["a"], s["a_scale"]), s["w"],
                        s["w_scale"], s["offsets"]).to(torch.bfloat16)
    else:
        return _plain_ffn(s)
    if op == "quant" and s["fmt"] == "e2m1":
        # two values to a byte, which no type of torch can be read as: the bytes themselves
        return {"codes": codes, "scales": scales.view(torch.float8_e8m0fnu)}
    codes, scales = _mx8(codes, scales)
    return {"codes": codes, "scales": scales} | ({"h": h, "out": n} if op == "norm" else {})


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["H"]
        res, mx = case["residual"], case["mx"]
        per = 2 + (4 if res else 0) + 2 + (1 + 1 / 32 if mx else 0)
        return {"bytes": int(n * per) + 2 * case["H"], "flops": n * (4 + res + 3 * mx)}
    if op == "quant":
        n = case["rows"] * case["cols"]
        out = (0.5 if case["fmt"] == "e2m1" else 1) + 1 / 32
        return {"bytes": int(n * ((2 if case["dtype"] == "bfloat16" else 4) + out)), "flops": 2 * n}
    w, t = 0.5 + 1 / 32, 1 + 1 / 32  # bytes of a weight and of a token element
    if op == "mm":
        used = int((_groups(case, 0, "cpu").diff() > 0).sum())
        R, N, K = case["R"], case["N"], case["K"]
        return {"bytes": int(used * N * K * w + R * K * t + R * N * 2), "flops": 2 * R * N * K}
    used = int((_routing(case, 0, "cpu")[0].diff() > 0).sum())
    T, R, H, I = case["T"], case["T"] * case["k"], case["H"], case["I"]
    return {"bytes": int(used * 3 * I * H * w + T * H * t + R * H * 2 + R * 4),
            "flops": 6 * R * I * H}


# ------------------------------------------------------------------ from the definition, in 64 bits


def _exact_blocks(v, emax, levels):
    """fp64 MX values of a matrix: the element nearest to v / scale in `levels` (the format's
    values that are not negative, ascending; a tie takes the one at an even place)."""
    shape = v.shape
    b = v.reshape(-1, 32)
    m = b.abs().amax(dim=1, keepdim=True)
    scale = torch.exp2((torch.floor(torch.log2(m)) - emax).clamp(-127, 127))
    # log2 may be rounded across a whole number next to a power of two
    scale = torch.where(scale * 2.0 ** emax > m, (scale / 2).clamp(min=2.0 ** -127), scale)
    scale = torch.where(scale * 2.0 ** (emax + 1) <= m, scale * 2, scale)
    u = (b / scale).abs().clamp(max=levels[-1])
    hi = torch.searchsorted(levels, u).clamp(1, len(levels) - 1)
    lo = hi - 1
    below, above = u - levels[lo], levels[hi] - u
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    place = torch.where(up, hi, lo)
    return (levels[place] * torch.sign(b)), place, scale, shape


def _levels8():
    v = [m / 8 * 2.0 ** -6 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:-1], dtype=torch.float64, device=DEVICE)  # the last code is NaN


def _exact_mx8(v):
    q, _, scale, shape = _exact_blocks(v, 8, _levels8())
    return q.reshape(shape), scale.reshape(*shape[:-1], shape[-1] // 32)


def _exact_decode(codes, scales, fmt):
    s = torch.ldexp(torch.ones_like(scales, dtype=torch.float64), scales.int() - 127)
    if fmt == "e4m3":
        sign = 1.0 - 2.0 * (codes >> 7).double()
        v = sign * torch.cat([_levels8(), _levels8().new_tensor([math.nan])])[(codes & 127).long()]
    else:
        lv = torch.tensor(_MX4_LEVELS, dtype=torch.float64, device=DEVICE)
        both = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
        v = (1.0 - 2.0 * (both >> 3).double()) * lv[(both & 7).long()]
    return v * s.repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x, h = s["x"].double(), None
        if s["residual"] is not None:
            h = x + s["residual"].double()
            x = h.to(torch.bfloat16).double()
        n = x / torch.sqrt((x * x).sum(dim=1, keepdim=True) / x.shape[1] + EPS) * s["weight"].double()
        codes, scales = _exact_mx8(n) if s["mx"] else (None, None)
        return {"codes": codes, "scales": scales, "h": h, "out": n}
    if op == "quant":
        if case["rows"] * case["cols"] > 40_000_000:
            return None
        v = s["src"].double()
        if case["fmt"] == "e4m3":
            codes, scales = _exact_mx8(v)
            return {"codes": codes, "scales": scales}
        lv = torch.tensor(_MX4_LEVELS, dtype=torch.float64, device=DEVICE)
        _, place, scale, shape = _exact_blocks(v, 2, lv)
        code = (place.reshape(shape) + 8 * torch.signbit(v)).to(torch.uint8)
        return {"codes": code[:, 0::2] + 16 * code[:, 1::2],
                "scales": scale.reshape(*shape[:-1], shape[-1] // 32)}
    off = s["offsets"].tolist()
    if op == "mm":
        y = torch.zeros(case["R"], case["N"], dtype=torch.float64, device=DEVICE)
        for e in range(case["E"]):
            i, j = off[e], off[e + 1]
            if j > i:
                y[i:j] = (_exact_decode(s["a"][i:j], s["a_scale"][i:j], "e4m3")
                          @ _exact_decode(s["w"][e], s["w_scale"][e], "e2m1").T)
        return y
    I, rows = case["I"], s["rows"].long()
    y = torch.zeros(rows.numel(), case["H"], dtype=torch.float64, device=DEVICE)
    for e in range(case["E"]):
        r = rows[off[e]:off[e + 1]]
        if r.numel():
            tok = torch.div(r, case["k"], rounding_mode="floor")
            h = (_exact_decode(s["x"][tok], s["x_scale"][tok], "e4m3")
                 @ _exact_decode(s["w13"][e], s["w13_scale"][e], "e2m1").T)
            act = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
            q, scale = _exact_mx8(act)
            y[r] = ((q * scale.repeat_interleave(32, dim=1))
                    @ _exact_decode(s["w2"][e], s["w2_scale"][e], "e2m1").T)
    return y
