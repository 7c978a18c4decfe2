"""The 4-bit block-scaled operators and the few-token expert layer on their real workloads.

Operators: quantization of 16-bit rows to E2M1 codes (one E4M3 scale for each 16
values along K, one FP32 scale for each row) and reading them back, the matrix
product of two such operands, its form for a mixture of experts (one product per
expert over rows sorted by expert), and the whole expert layer of a few tokens
on 8-bit or 4-bit weights.

listed() and draw() give cases, prepare() a user's inputs, run() one pass
(through the library where `own` is set, else in plain torch operations),
exact() the same in 64 bits, work() the bytes and operations of a pass.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
GROUP = 16                      # values that share an E4M3 scale
TOP = 448.0 * 6.0               # largest scale times the largest code's value


def _lib():
    import precision_matmul_dg_gb300 as dg
    return dg


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # activations of a decoding batch of 16 tokens in front of a linear layer, written in
        # 4 bits and read back (what a calibration run does to measure the error)
        dict(name="quant_decode", kind="quant", rows=16, k=4096, type="f16"),
        # a long prompt's activations, an odd number of rows
        dict(name="quant_prefill", kind="quant", rows=8191, k=4096, type="bf16"),
        # one token through an up-projection with bias and GELU
        dict(name="gemm_decode", kind="gemm", m=1, n=8960, k=1536, type="f16",
             epilogue="bias_gelu"),
        # a batch of short prompts, odd sizes, FP32 out
        dict(name="gemm_odd", kind="gemm", m=500, n=2900, k=2902, type="f32", epilogue="none"),
        # a long prompt through a large square layer
        dict(name="gemm_prefill", kind="gemm", m=8192, n=8192, k=8192, type="bf16",
             epilogue="none"),
        # a short prompt, 2 of 8 experts for each token, in 128-row segments
        dict(name="experts_short", kind="experts", tokens=300, top_k=2, count=8, n=2048, k=1536,
             type="f16", epilogue="none"),
        # a long prompt, 8 of 64 experts for each token
        dict(name="experts_prefill", kind="experts", tokens=4096, top_k=8, count=64, n=4096,
             k=2048, type="bf16", epilogue="gelu"),
        # one decoded token through an expert layer, 8 of 64 experts, 8-bit weights
        dict(name="layer_one_fp8", kind="layer", format="fp8", tokens=1, top_k=8, count=64,
             width=2048, hidden=4096, type="bf16", activation="gelu", bias=False),
        # the same with 4-bit weights
        dict(name="layer_one_nvf4", kind="layer", format="nvf4", tokens=1, top_k=8, count=64,
             width=2048, hidden=4096, type="bf16", activation="gelu", bias=False),
        # a decoding batch of 8 tokens, gated experts in 8 bits
        dict(name="layer_batch_fp8", kind="layer", format="fp8", tokens=8, top_k=8, count=64,
             width=2048, hidden=2048, type="f16", activation="swiglu", bias=False),
        # a decoding batch of 16 tokens, gated experts in 4 bits
        dict(name="layer_batch_nvf4", kind="layer", format="nvf4", tokens=16, top_k=8, count=64,
             width=2048, hidden=2048, type="bf16", activation="swiglu", bias=False),
        # two tokens of a small model: few and small experts, with biases
        dict(name="layer_small_nvf4", kind="layer", format="nvf4", tokens=2, top_k=2, count=8,
             width=1536, hidden=1000, type="f16", activation="gelu", bias=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["quant", "gemm", "gemm", "experts", "experts", "layer", "layer", "layer"])
    if kind == "quant":
        return dict(kind=kind, rows=_log(rng, 1, 8192), k=_log(rng, 32, 8192),
                    type=rng.choice(["f16", "bf16"]))
    if kind == "gemm":
        return dict(kind=kind, m=_log(rng, 1, 8192), n=_log(rng, 256, 8192),
                    k=_log(rng, 256, 8192), type=rng.choice(["f16", "bf16", "f32"]),
                    epilogue=rng.choice(["none", "none", "bias", "bias_gelu"]))
    if kind == "experts":
        return dict(kind=kind, tokens=_log(rng, 1, 4096), top_k=rng.choice([1, 2, 4, 8]),
                    count=rng.choice([8, 16, 64]), n=_log(rng, 512, 4096),
                    k=_log(rng, 512, 2048), type=rng.choice(["f16", "bf16"]),
                    epilogue=rng.choice(["none", "gelu"]))
    activation = rng.choice(["gelu", "swiglu"])
    hidden = _log(rng, 256, 2048)
    return dict(kind=kind, format=rng.choice(["fp8", "nvf4"]), tokens=_log(rng, 1, 16),
                top_k=rng.choice([1, 2, 4, 8]), count=rng.choice([8, 16, 64]),
                width=8 * _log(rng, 32, 256),
                hidden=hidden if activation == "gelu" else _ceil(hidden, 128) * 128,
                type=rng.choice(["f16", "bf16"]), activation=activation,
                bias=rng.choice([False, False, True]))


# ------------------------------------------------------------ block scaling

def _tiled(s):
    """Scales [..., rows, groups] in tiles of 128 rows x 4 groups: line l of a tile holds those of
    its rows l, 32 + l, 64 + l and 96 + l, four bytes each; zeros where there is none."""
    rows, groups = s.shape[-2:]
    rb, gb = _ceil(rows, 128), _ceil(groups, 4)
    t = torch.nn.functional.pad(s.view(torch.uint8), (0, gb * 4 - groups, 0, rb * 128 - rows))
    t = t.reshape(s.shape[:-2] + (rb, 4, 32, gb, 4)).transpose(-4, -2)
    return t.reshape(s.shape[:-2] + (rb, gb, 32, 16)).contiguous().view(F8)


def _untiled(t, rows, groups):
    """The scales [..., rows, groups] that such tiles hold."""
    lead, (rb, gb) = t.shape[:-4], t.shape[-4:-2]
    s = t.view(torch.uint8).reshape(lead + (rb, gb, 32, 4, 4)).transpose(-4, -2)
    return s.reshape(lead + (rb * 128, gb * 4))[..., :rows, :groups].contiguous().view(F8)


def _packed(codes):
    """Codes [..., k] two to a byte, the even one in the low half, in rows that start on 16-byte
    boundaries; an odd last one gets a zero beside it."""
    k = codes.shape[-1]
    room = torch.zeros(codes.shape[:-1] + (_ceil(k, 32) * 32,), dtype=torch.uint8,
                       device=codes.device)
    room[..., :k] = codes
    return (room[..., 0::2] | (room[..., 1::2] << 4))[..., :_ceil(k, 2)]


def _quantized_fp32(x):
    """FP32 [rows, k] -> codes (one to a byte), scales [rows, groups] and the rows' scales.  Every
    quotient and product is rounded to FP32."""
    rows, k = x.shape
    groups = _ceil(k, GROUP)
    v = torch.nn.functional.pad(x, (0, groups * GROUP - k)).reshape(rows, groups, GROUP)
    amax = v.abs().amax(2)
    # the smallest power of two whose TOP multiple reaches the row's largest value
    m, e = torch.frexp(amax.amax(1).double() / TOP)
    e = torch.where(m == 0.5, e - 1, e).clamp(-100, 126)
    row = torch.ldexp(torch.ones_like(m), e).float()
    scale = (amax / (6.0 * row[:, None])).to(F8).float().clamp_min(2.0 ** -9)
    q = v / (scale * row[:, None])[..., None]
    a = q.abs()
    code = sum((a > b).to(torch.uint8) for b in (0.25, 1.25, 2.5, 5.0))
    code = code + sum((a >= b).to(torch.uint8) for b in (0.75, 1.75, 3.5))
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    return code.reshape(rows, groups * GROUP)[:, :k], scale.to(F8), row


def _values_fp32(codes, scales, row_scales, k):
    """FP32 values [..., rows, k] of packed codes."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack([table[byte & 15], table[byte >> 4]], 1)
    v = pair[codes.int()].reshape(codes.shape[:-1] + (-1,))[..., :k]
    s = _untiled(scales, codes.shape[-2], _ceil(k, GROUP)).float() * row_scales[..., None]
    return v * s.repeat_interleave(GROUP, -1)[..., :k]


def _values_fp8(codes, scales):
    """FP32 values [..., rows, k] of E4M3 codes with a scale for each 128 x 128 block."""
    rows, k = codes.shape[-2:]
    s = scales.repeat_interleave(128, -2)[..., :rows, :].repeat_interleave(128, -1)[..., :k]
    return codes.float() * s


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols):
    """Rows of their own size, and a few columns that stand out, as hidden states have."""
    x = _normal(g, rows, cols) * torch.exp(0.5 * _normal(g, rows, 1))
    return x * torch.where(torch.rand(1, cols, generator=g, device="cuda") < 0.01, 12.0, 1.0)


def _operand(x):
    """An operand's packed codes, tiled scales and row scales."""
    codes, scales, row = _quantized_fp32(x)
    return _packed(codes), _tiled(scales), row


def _weights_nvf4(g, k, *shape):
    """Weights in stored form: uniform codes, scales of a few binades; products of k of them with
    unit values come out near one."""
    rows = shape[-1]
    lead = shape[:-1]
    room = torch.randint(0, 256, shape + (_ceil(k, 32) * 16,), generator=g, device="cuda",
                         dtype=torch.uint8)[..., :_ceil(k, 2)]
    if k % 2:
        room[..., -1] &= 15
    scales = torch.randint(0x40, 0x50, shape + (_ceil(k, GROUP),), generator=g, device="cuda",
                           dtype=torch.uint8).view(F8)
    row = torch.exp(0.1 * _normal(g, *shape)) / (2.93 * 4.3 * math.sqrt(k))
    return room, _tiled(scales), row


def _weights_fp8(g, k, *shape):
    room = torch.zeros(shape + (_ceil(k, 16) * 16,), dtype=torch.uint8, device="cuda").view(F8)
    room[..., :k] = (40.0 * torch.randn(shape + (k,), generator=g, device="cuda",
                                        dtype=torch.float16)).to(F8)
    blocks = shape[:-1] + (_ceil(shape[-1], 128), _ceil(k, 128))
    return room[..., :k], torch.exp(0.2 * _normal(g, *blocks)) / (40.0 * math.sqrt(k))


def _choices(g, tokens, top_k, count):
    """Each token's experts: distinct, some experts chosen more often."""
    score = _normal(g, tokens, count) + 0.5 * _normal(g, 1, count)
    return score.topk(top_k, dim=1).indices.to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    s = {"case": dict(case)}
    t = TYPES[case["type"]]
    if kind == "quant":
        rows, k = case["rows"], case["k"]
        s["x"] = _activations(g, rows, _ceil(k, 8) * 8).to(t)[:, :k]
        room = torch.zeros(rows, _ceil(k, 32) * 16, dtype=torch.uint8, device="cuda")
        s["out"] = (room[:, :_ceil(k, 2)],
                    torch.zeros(_ceil(rows, 128), _ceil(k, 64), 32, 16, dtype=torch.uint8,
                                device="cuda").view(F8),
                    torch.zeros(rows, device="cuda"))
        s["d"] = torch.zeros(rows, _ceil(k, 8) * 8, dtype=t, device="cuda")[:, :k]
    elif kind == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = _operand(_activations(g, m, k))
        s["b"] = _operand(_normal(g, n, k) / math.sqrt(k))
        s["bias"] = (0.1 * _normal(g, n)).to(t) if "bias" in case["epilogue"] else None
        s["d"] = torch.zeros(m, n, dtype=t, device="cuda")
    elif kind == "experts":
        n, k, count, top_k = case["n"], case["k"], case["count"], case["top_k"]
        ids = _choices(g, case["tokens"], top_k, count)
        flat = ids.reshape(-1).long()
        sizes = torch.zeros(count, dtype=torch.long, device="cuda").index_add_(
            0, flat, torch.ones_like(flat))
        ends = (_ceil(sizes, 128) * 128).cumsum(0)
        s["offsets"] = torch.cat([ends.new_zeros(1), ends]).int()
        order = torch.sort(flat, stable=True).indices
        row = s["offsets"].long()[flat[order]] + torch.arange(flat.numel(), device="cuda") - (
            sizes.cumsum(0) - sizes)[flat[order]]
        rows = _rows_of(case)
        x = torch.zeros(rows, k, device="cuda")
        x[row] = _activations(g, case["tokens"], k)[order // top_k]
        s["a"] = _operand(x)
        s["b"] = _weights_nvf4(g, k, count, n)
        s["d"] = torch.zeros(rows, n, dtype=t, device="cuda")
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    else:
        width, hidden, count = case["width"], case["hidden"], case["count"]
        first = hidden * (2 if case["activation"] == "swiglu" else 1)
        make = _weights_fp8 if case["format"] == "fp8" else _weights_nvf4
        s["x"] = _activations(g, case["tokens"], width).to(t)
        s["ids"] = _choices(g, case["tokens"], case["top_k"], count)
        s["w"] = torch.softmax(_normal(g, case["tokens"], case["top_k"]), 1).contiguous()
        s["up"] = make(g, width, count, first)
        s["down"] = make(g, hidden, count, width)
        s["bias"] = (None, None)
        if case["bias"]:
            s["bias"] = ((0.1 * _normal(g, count, first)).to(t),
                         (0.1 * _normal(g, count, width)).to(t))
        s["d"] = torch.zeros(case["tokens"], width, dtype=t, device="cuda")
    return s


def _rows_of(case):
    """Rows that the sort of an experts case needs room for, segments of 128."""
    slots = case["tokens"] * case["top_k"]
    return _ceil(slots + min(case["count"], slots) * 127, 128) * 128


# -------------------------------------------------------------------- run

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    dg = _lib()
    case = s["case"]
    kind = case["kind"]
    if kind == "quant":
        codes, scales, row = dg.quantize_nvf4(s["x"], out=s["out"])
        return dg.dequantize_nvf4(codes, scales, row, s["d"]), scales, row
    if kind == "gemm":
        return dg.gemm_nvf4(*s["a"], *s["b"], s["d"], bias=s["bias"], epilogue=case["epilogue"])
    if kind == "experts":
        return dg.gemm_nvf4_grouped(*s["a"], *s["b"], s["offsets"], s["d"],
                                    epilogue=case["epilogue"])
    return dg.moe_layer(s["x"], s["ids"], s["w"], s["up"], s["down"], s["d"],
                        activation=case["activation"], bias_up=s["bias"][0],
                        bias_down=s["bias"][1])


def _gelu_fp32(v):
    return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))


def _run_plain(s):
    case = s["case"]
    kind = case["kind"]
    t = TYPES[case["type"]]
    if kind == "quant":
        codes, scales, row = _quantized_fp32(s["x"].float())
        codes, scales = _packed(codes), _tiled(scales)
        return _values_fp32(codes, scales, row, case["k"]).to(t), scales, row
    if kind == "gemm":
        v = _values_fp32(*s["a"], case["k"]) @ _values_fp32(*s["b"], case["k"]).t()
        if s["bias"] is not None:
            v = v + s["bias"].float()
        return (_gelu_fp32(v) if "gelu" in case["epilogue"] else v).to(t)
    if kind == "experts":
        at = s["offsets"][:-1, None].long() + torch.arange(s["most"], device="cuda")
        inside = at < s["offsets"][1:, None]
        a = _values_fp32(*s["a"], case["k"])
        a = a[at.clamp_max(a.shape[0] - 1)]
        v = torch.bmm(a, _values_fp32(*s["b"], case["k"]).transpose(1, 2))
        v = (_gelu_fp32(v) if "gelu" in case["epilogue"] else v).to(t)
        d = torch.zeros(s["d"].shape[0] + 1, case["n"], dtype=t, device=v.device)
        d[torch.where(inside, at, s["d"].shape[0])] = v
        return d[:-1]
    flat = s["ids"].reshape(-1).long()
    if case["format"] == "fp8":
        up, down = _values_fp8(*s["up"]), _values_fp8(*s["down"])
    else:
        up = _values_fp32(*s["up"], case["width"])
        down = _values_fp32(*s["down"], case["hidden"])
    x = s["x"].float().repeat_interleave(case["top_k"], 0)
    h = torch.bmm(up[flat], x[..., None])[..., 0]
    if case["bias"]:
        h = h + s["bias"][0][flat].float()
    if case["activation"] == "swiglu":
        gate, value = h[:, :case["hidden"]], h[:, case["hidden"]:]
        h = gate / (1.0 + torch.exp(-gate)) * value
    else:
        h = _gelu_fp32(h)
    y = torch.bmm(down[flat], h[..., None])[..., 0]
    if case["bias"]:
        y = y + s["bias"][1][flat].float()
    return (y.reshape(s["w"].shape + (-1,)) * s["w"][..., None]).sum(1).to(t)


# ------------------------------------------------------------------ exact

def _nvf4_exactly(codes, scales, row, k):
    """Values [rows, k] of one operand in 64 bits, nibble by nibble."""
    rows = codes.shape[0]
    v = torch.zeros(rows, 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        n = (codes >> (4 * half)) & 15
        e, m = (n >> 1) & 3, (n & 1).double()
        mag = torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1.0) * (1.0 + 0.5 * m))
        v[:, half::2] = torch.where(n > 7, -mag, mag)
    v = v[:, :k]
    line = torch.arange(rows, device=codes.device)
    tile, part, line = line // 128, line // 32 % 4, line % 32
    s = scales.double()
    for j in range(_ceil(k, GROUP)):
        of = s[tile, j // 4, line, 4 * part + j % 4]
        v[:, GROUP * j:GROUP * (j + 1)] *= (of * row.double())[:, None]
    return v


def _gelu_exactly(v):
    return v * torch.special.ndtr(v)


def _quantized_exactly(x):
    """The values that the definition gives x in 64 bits, the scales and the rows' scales."""
    rows, k = x.shape
    top = x.abs().amax(1)
    row = torch.exp2(torch.ceil(torch.log2(top / TOP)).clamp(-100, 126))
    row = torch.where(top / TOP <= row / 2, row / 2, torch.where(top / TOP > row, row * 2, row))
    out = torch.zeros_like(x)
    scales = x.new_zeros(rows, _ceil(k, GROUP))
    for j in range(scales.shape[1]):
        part = x[:, GROUP * j:GROUP * (j + 1)]
        t = part.abs().amax(1) / (6.0 * row)
        step = torch.exp2((torch.frexp(t)[1].double() - 1).clamp_min(-6) - 3)
        sc = (torch.round(t / step) * step).clamp_min(2.0 ** -9)
        q = part / (sc * row)[:, None]
        step = torch.exp2((torch.frexp(q)[1].double() - 1).clamp(0, 2) - 1)
        out[:, GROUP * j:GROUP * (j + 1)] = (torch.round(q / step) * step).clamp(-6, 6) * (
            sc * row)[:, None]
        scales[:, j] = sc
    return out, scales, row


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quant":
        values, scales, row = _quantized_exactly(s["x"].double())
        tiles = torch.zeros(s["out"][1].shape, dtype=torch.float64, device="cuda")
        line = torch.arange(case["rows"], device="cuda")
        for j in range(scales.shape[1]):
            tiles[line // 128, j // 4, line % 32, 4 * (line // 32 % 4) + j % 4] = scales[:, j]
        return values, tiles, row
    if kind == "gemm":
        v = _nvf4_exactly(*s["a"], case["k"]) @ _nvf4_exactly(*s["b"], case["k"]).t()
        if s["bias"] is not None:
            v = v + s["bias"].double()
        return _gelu_exactly(v) if "gelu" in case["epilogue"] else v
    if kind == "experts":
        ends = s["offsets"].tolist()
        d = s["d"].double()
        a = _nvf4_exactly(*s["a"], case["k"])
        for e in range(case["count"]):
            if ends[e + 1] > ends[e]:
                at = slice(ends[e], ends[e + 1])
                v = a[at] @ _nvf4_exactly(*(p[e] for p in s["b"]), case["k"]).t()
                d[at] = _gelu_exactly(v) if "gelu" in case["epilogue"] else v
        return d
    ids = s["ids"].tolist()
    y = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")

    def weights(of, e, k):
        if case["format"] == "nvf4":
            return _nvf4_exactly(*(p[e] for p in of), k)
        v, sc = of[0][e].double(), of[1][e].double()
        for i in range(sc.shape[0]):
            for j in range(sc.shape[1]):
                v[128 * i:128 * (i + 1), 128 * j:128 * (j + 1)] *= sc[i, j]
        return v
    for e in sorted({e for row in ids for e in row}):
        at = [(t, j) for t, row in enumerate(ids) for j, v in enumerate(row) if v == e]
        tokens = torch.tensor([t for t, _ in at], device="cuda")
        h = s["x"].double()[tokens] @ weights(s["up"], e, case["width"]).t()
        if case["bias"]:
            h = h + s["bias"][0][e].double()
        if case["activation"] == "swiglu":
            h = h[:, :case["hidden"]] * torch.sigmoid(h[:, :case["hidden"]]) * h[:, case["hidden"]:]
        else:
            h = _gelu_exactly(h)
        rows = h @ weights(s["down"], e, case["hidden"]).t()
        if case["bias"]:
            rows = rows + s["bias"][1][e].double()
        for i, (t, j) in enumerate(at):
            y[t] += s["w"][t, j].double() * rows[i]
    return y


# ------------------------------------------------------------------- work

def work(case):
    kind = case["kind"]
    z = BYTES[case["type"]]
    code = 0.5 + 1.0 / GROUP    # bytes of a 4-bit value with its share of a scale
    if kind == "quant":
        rows, k = case["rows"], case["k"]
        return {"bytes": rows * k * (2 * z + 2 * code) + 8 * rows, "flops": 4 * rows * k}
    if kind == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (k * code + 4) + m * n * z, "flops": 2 * m * n * k}
    slots = case["tokens"] * case["top_k"]
    count = case["count"]
    # experts that get a row: of `count`, when each token's choices are a fair draw
    used = count * (1.0 - (1.0 - case["top_k"] / count) ** case["tokens"])
    if kind == "experts":
        n, k = case["n"], case["k"]
        return {"bytes": used * n * (k * code + 4) + slots * (k * code + 4 + n * z),
                "flops": 2 * slots * n * k}
    width, hidden = case["width"], case["hidden"]
    first = hidden * (2 if case["activation"] == "swiglu" else 1)
    of = 1.0 + 4.0 / 128 ** 2 if case["format"] == "fp8" else code
    return {"bytes": used * of * width * (first + hidden) + 2 * case["tokens"] * width * z +
            8 * slots, "flops": 2 * slots * width * (first + hidden)}
