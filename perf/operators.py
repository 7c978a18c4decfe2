"""The 8-bit floating-point operators on their real workloads.

Operators: block quantization to E4M3 (one FP32 scale per 1 x 128 or 128 x 128
block), the matrix product of two such operands, its form for a mixture of
experts (one product per expert over rows sorted by expert, and the weight
gradients), the sort of tokens by expert with the move of their rows into that
order, and the way back with the routing weights and its gradient.

listed() and draw() give cases, prepare() a user's inputs, run() one pass
(through the library where `own` is set, else in plain torch operations),
exact() the same in 64 bits, work() the bytes and operations of a pass.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
TOP = 448.0                     # largest finite E4M3 value
FLOOR = TOP * 2.0 ** -126       # a block's amax is taken as at least this
BLOCK = 128
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}


def _lib():
    import precision_matmul_dg_gb300 as dg
    return dg


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # activations of a decoding batch of 16 tokens in front of a linear layer
        dict(name="quant_decode", kind="quant", rows=16, k=4096, type="f16", form="rows",
             block_rows=1),
        # a training step's activations: codes for the forward product and, transposed, for
        # the weight gradient
        dict(name="quant_train", kind="quant", rows=8191, k=4096, type="bf16", form="both",
             block_rows=1),
        # one token through an up-projection with bias and GELU
        dict(name="gemm_decode", kind="gemm", m=1, n=8960, k=1536, block_rows=128, type="f16",
             epilogue="bias_gelu"),
        # a long prompt through a large square layer
        dict(name="gemm_prefill", kind="gemm", m=8192, n=8192, k=8192, block_rows=128,
             type="bf16", epilogue="none"),
        # a weight gradient of that kind: both operands scaled by 1 x 128 blocks along an odd
        # number of tokens, FP32 out
        dict(name="gemm_wgrad", kind="gemm", m=1536, n=8960, k=4093, block_rows=1, type="f32",
             epilogue="none"),
        # 8 decoded tokens through 64 experts, 8 each: about one row per expert
        dict(name="experts_decode", kind="experts", tokens=8, top_k=8, count=64, n=4096, k=2048,
             type="f16", epilogue="gelu"),
        # a prompt through the same experts
        dict(name="experts_prefill", kind="experts", tokens=4096, top_k=8, count=64, n=4096,
             k=2048, type="bf16", epilogue="gelu"),
        # the experts' weight gradients of a training step
        dict(name="experts_wgrad", kind="experts_wgrad", tokens=2048, top_k=8, count=64, n=4096,
             k=2048, type="f32"),
        # 8 decoded tokens sorted by expert and quantized in that order
        dict(name="route_decode", kind="route", tokens=8, top_k=8, count=64, width=2048,
             type="f16", align=1, form="fp8", dropped=False),
        # a training batch, some of whose choices were dropped, in 128-row segments
        dict(name="route_train", kind="route", tokens=16384, top_k=8, count=64, width=2048,
             type="bf16", align=128, form="fp8", dropped=True),
        # 8 decoded tokens' expert rows back, weighted
        dict(name="combine_decode", kind="combine", tokens=8, top_k=8, count=64, width=4096,
             type="f16", align=1, train=False, dropped=False),
        # a training batch's way back, its gradient, and the gradient of the way there
        dict(name="combine_train", kind="combine", tokens=8192, top_k=8, count=64, width=4096,
             type="bf16", align=128, train=True, dropped=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["quant", "gemm", "gemm", "experts", "experts", "experts_wgrad", "route",
                       "combine"])
    if kind == "quant":
        return dict(kind=kind, rows=_log(rng, 1, 16384), k=_log(rng, 64, 8192),
                    type=rng.choice(["f16", "bf16"]), form=rng.choice(["rows", "both"]),
                    block_rows=rng.choice([1, 1, 128]))
    if kind == "gemm":
        return dict(kind=kind, m=_log(rng, 1, 8192), n=_log(rng, 256, 8192),
                    k=_log(rng, 256, 8192), block_rows=rng.choice([1, 128, 128]),
                    type=rng.choice(["f16", "bf16", "f32"]),
                    epilogue=rng.choice(["none", "none", "bias", "bias_gelu"]))
    count = rng.choice([8, 16, 64, 128])
    top_k = rng.choice([1, 2, 4, 8])
    if kind == "experts":
        return dict(kind=kind, tokens=_log(rng, 1, 4096), top_k=top_k, count=count,
                    n=_log(rng, 512, 4096), k=_log(rng, 512, 2048),
                    type=rng.choice(["f16", "bf16"]), epilogue=rng.choice(["none", "gelu"]))
    if kind == "experts_wgrad":
        return dict(kind=kind, tokens=_log(rng, 16, 2048), top_k=top_k, count=min(count, 64),
                    n=_log(rng, 512, 4096), k=_log(rng, 512, 2048),
                    type=rng.choice(["f32", "bf16"]))
    if kind == "route":
        return dict(kind=kind, tokens=_log(rng, 1, 16384), top_k=top_k, count=count,
                    width=8 * _log(rng, 32, 256), type=rng.choice(["f16", "bf16"]),
                    align=rng.choice([1, 128]), form=rng.choice(["fp8", "copy"]),
                    dropped=rng.choice([False, True]))
    return dict(kind=kind, tokens=_log(rng, 1, 8192), top_k=top_k, count=count,
                width=8 * _log(rng, 32, 512), type=rng.choice(["f16", "bf16"]),
                align=rng.choice([1, 128]), train=rng.choice([False, True]),
                dropped=rng.choice([False, True]))


# ------------------------------------------------------------ block scaling

def _blocks_fp32(x, block_rows):
    """FP32 [..., R, C] -> E4M3 codes of the same shape and their FP32 scales, one for each
    block of block_rows x 128; a block with a NaN or an infinity: codes 0, scale NaN."""
    rows, cols = x.shape[-2:]
    lead = x.shape[:-2]
    br, bc = _ceil(rows, block_rows), _ceil(cols, BLOCK)
    full = torch.nn.functional.pad(x, (0, bc * BLOCK - cols, 0, br * block_rows - rows))
    full = full.reshape(lead + (br, block_rows, bc, BLOCK))
    amax = full.abs().amax(dim=(-3, -1), keepdim=True)
    bad = ~torch.isfinite(amax)
    amax = amax.clamp_min(FLOOR)
    codes = torch.where(bad, torch.zeros_like(full), full * (TOP / amax)).to(F8)
    scales = torch.where(bad, torch.full_like(amax, math.nan), amax / TOP)
    codes = codes.reshape(lead + (br * block_rows, bc * BLOCK))[..., :rows, :cols]
    return codes.contiguous(), scales.reshape(lead + (br, bc)).contiguous()


def _values_fp32(codes, scales, block_rows):
    rows, cols = codes.shape[-2:]
    s = scales.repeat_interleave(BLOCK, -1)[..., :cols]
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, -2)[..., :rows, :]
    return codes.float() * s


def _padded(codes):
    """The same codes in rows that start on 16-byte boundaries."""
    cols = codes.shape[-1]
    room = torch.zeros(codes.shape[:-1] + (_ceil(cols, 16) * 16,), dtype=torch.uint8,
                       device=codes.device)
    room[..., :cols] = codes.view(torch.uint8)
    return room.view(F8)[..., :cols]


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


def _choices(g, tokens, top_k, count, dropped):
    """Each token's experts: distinct, some experts chosen more often; -1 where dropped."""
    score = _normal(g, tokens, count) + 0.5 * _normal(g, 1, count)
    ids = score.topk(top_k, dim=1).indices.to(torch.int32)
    if dropped:
        ids = torch.where(torch.rand(tokens, top_k, generator=g, device="cuda") < 0.05, -1, ids)
        ids = torch.where(torch.rand(tokens, 1, generator=g, device="cuda") < 0.02, -1, ids)
    return ids.contiguous()


def _capacity(tokens, top_k, count, align):
    slots = tokens * top_k
    return _ceil(slots + min(count, slots) * (align - 1), align) * align


def _sorted_by_expert(ids, count, align):
    """offsets [count + 1], row -> slot (-1: none) and slot -> row (-1: dropped)."""
    slots, top_k = ids.numel(), ids.shape[1]
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < count), flat, count)
    sizes = (key[:, None] == torch.arange(count, device=ids.device)).sum(0) if slots < 4096 else \
        torch.zeros(count + 1, dtype=torch.long, device=ids.device).index_add_(
            0, key, torch.ones_like(key))[:count]
    ends = ((sizes + align - 1) // align * align).cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    order = torch.sort(key, stable=True).indices
    first = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)])
    kept = key[order]
    row = offsets[kept] + torch.arange(slots, device=ids.device) - first[kept]
    row = torch.where(kept < count, row, -1)
    cap = _capacity(ids.shape[0], top_k, count, align)
    row_slot = torch.full((cap + 1,), -1, dtype=torch.long, device=ids.device)
    row_slot[torch.where(row >= 0, row, cap)] = order
    slot_row = torch.full((slots,), -1, dtype=torch.long, device=ids.device)
    slot_row[order] = row
    return (offsets.int(), row_slot[:cap].int().contiguous(),
            slot_row.int().reshape(ids.shape).contiguous())


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    s = {"case": dict(case)}
    t = TYPES[case["type"]]
    if kind == "quant":
        s["x"] = _activations(g, case["rows"], _ceil(case["k"], 8) * 8).to(t)[:, :case["k"]]
        rows, k, br = case["rows"], case["k"], case["block_rows"]
        out = []
        for r, c in ((rows, k), (k, rows))[:1 if case["form"] == "rows" else 2]:
            room = torch.zeros(r, _ceil(c, 16) * 16, dtype=torch.uint8, device="cuda")
            out += [room.view(F8)[:, :c],
                    torch.zeros(_ceil(r, br), _ceil(c, BLOCK), device="cuda")]
        s["out"] = tuple(out)
    elif kind == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        a, s["sa"] = _blocks_fp32(_activations(g, m, k), 1)
        b, s["sb"] = _blocks_fp32(_normal(g, n, k) / math.sqrt(k), case["block_rows"])
        s["a"], s["b"] = _padded(a), _padded(b)
        s["bias"] = (0.1 * _normal(g, n)).to(t) if "bias" in case["epilogue"] else None
        s["d"] = torch.zeros(m, n, dtype=t, device="cuda")
    elif kind == "experts":
        n, k, count = case["n"], case["k"], case["count"]
        ids = _choices(g, case["tokens"], case["top_k"], count, False)
        s["offsets"], row_slot, _ = _sorted_by_expert(ids, count, 1)
        x = _activations(g, case["tokens"], k)
        a, s["sa"] = _blocks_fp32(x[row_slot.long() // case["top_k"]], 1)
        b, s["sb"] = _blocks_fp32(_normal(g, count, n, k) / math.sqrt(k), BLOCK)
        s["a"], s["b"] = _padded(a), _padded(b)
        s["d"] = torch.zeros(a.shape[0], n, dtype=t, device="cuda")
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    elif kind == "experts_wgrad":
        n, k, count = case["n"], case["k"], case["count"]
        ids = _choices(g, case["tokens"], case["top_k"], count, False)
        s["offsets"], row_slot, _ = _sorted_by_expert(ids, count, BLOCK)
        there = (row_slot >= 0).float()
        src = row_slot.long().clamp_min(0) // case["top_k"]
        x = _activations(g, case["tokens"], k)[src] * there[:, None]
        dy = 1e-3 * _normal(g, row_slot.numel(), n) * there[:, None]
        s["a"], s["sa"] = _blocks_fp32(dy.t(), 1)
        s["b"], s["sb"] = _blocks_fp32(x.t(), 1)
        s["d"] = torch.zeros(count, n, k, dtype=t, device="cuda")
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    else:
        tokens, top_k, count, width = (case[v] for v in ("tokens", "top_k", "count", "width"))
        s["ids"] = _choices(g, tokens, top_k, count, case["dropped"])
        cap = _capacity(tokens, top_k, count, case["align"])
        if kind == "route":
            s["x"] = _activations(g, tokens, width).to(t)
            s["sorted"] = (torch.zeros(count + 1, dtype=torch.int32, device="cuda"),
                           torch.zeros(cap, dtype=torch.int32, device="cuda"),
                           torch.zeros(tokens, top_k, dtype=torch.int32, device="cuda"))
            if case["form"] == "fp8":
                room = torch.zeros(cap, _ceil(width, 16) * 16, dtype=torch.uint8, device="cuda")
                s["out"] = (room.view(F8)[:, :width],
                            torch.zeros(cap, _ceil(width, BLOCK), device="cuda"))
            else:
                s["out"] = (torch.zeros(cap, width, dtype=t, device="cuda"),)
        else:
            _, s["row_slot"], s["slot_row"] = _sorted_by_expert(s["ids"], count, case["align"])
            there = (s["row_slot"] >= 0).float()[:, None]
            s["y"] = (_normal(g, cap, width) * there).to(t)
            s["w"] = torch.softmax(_normal(g, tokens, top_k), 1).contiguous()
            s["d"] = torch.zeros(tokens, width, dtype=t, device="cuda")
            if case["train"]:
                s["dd"] = (1e-3 * _normal(g, tokens, width)).to(t)
                s["dxs"] = (1e-3 * _normal(g, cap, width) * there).to(t)
                s["dy"] = torch.zeros(cap, width, dtype=t, device="cuda")
                s["dw"] = torch.zeros(tokens, top_k, device="cuda")
                s["dx"] = torch.zeros(tokens, width, dtype=t, device="cuda")
    return s


# -------------------------------------------------------------------- run

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    dg = _lib()
    case = s["case"]
    kind = case["kind"]
    if kind == "quant":
        return dg.quantize_fp8(s["x"], form=case["form"], block_rows=case["block_rows"],
                               out=s["out"])
    if kind == "gemm":
        return dg.gemm_fp8(s["a"], s["sa"], s["b"], s["sb"], s["d"], bias=s["bias"],
                           epilogue=case["epilogue"])
    if kind == "experts":
        return dg.gemm_fp8_grouped(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], s["d"],
                                   epilogue=case["epilogue"])
    if kind == "experts_wgrad":
        return dg.gemm_fp8_grouped_wgrad(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], s["d"])
    if kind == "route":
        offsets, row_slot, slot_row = dg.moe_sort(s["ids"], case["count"], align=case["align"],
                                                  out=s["sorted"])
        if case["form"] == "fp8":
            dg.moe_dispatch_fp8(s["x"], row_slot, case["top_k"], *s["out"])
        else:
            dg.moe_dispatch(s["x"], row_slot, case["top_k"], *s["out"])
        return (offsets, row_slot, slot_row) + s["out"]
    dg.moe_combine(s["y"], s["slot_row"], s["d"], weights=s["w"])
    if not case["train"]:
        return s["d"]
    dg.moe_combine_backward(s["dd"], s["y"], s["slot_row"], s["row_slot"], s["w"], s["dy"],
                            s["dw"])
    dg.moe_combine(s["dxs"], s["slot_row"], s["dx"])
    return s["d"], s["dy"], s["dw"], s["dx"]


def _activate_fp32(v, bias, epilogue):
    if "bias" in epilogue:
        v = v + bias.float()
    if "gelu" in epilogue:
        v = 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v


def _segments(offsets, most):
    """[count, most] row numbers and whether each lies in its expert's segment."""
    at = offsets[:-1, None].long() + torch.arange(most, device=offsets.device)
    return at, at < offsets[1:, None]


def _gather_sum_fp32(rows, slot_row, weights):
    """sum over j of weights[t, j] * rows[slot_row[t, j]], dropped slots left out."""
    got = rows[slot_row.long().clamp_min(0)].float()
    got = torch.where((slot_row >= 0)[..., None], got, torch.zeros_like(got))
    return (got if weights is None else got * weights[..., None]).sum(1)


def _run_plain(s):
    case = s["case"]
    kind = case["kind"]
    t = TYPES[case["type"]]
    if kind == "quant":
        x = s["x"].float()
        out = _blocks_fp32(x, case["block_rows"])
        if case["form"] == "both":
            out += _blocks_fp32(x.t(), case["block_rows"])
        return out
    if kind == "gemm":
        v = _values_fp32(s["a"], s["sa"], 1) @ _values_fp32(s["b"], s["sb"],
                                                            case["block_rows"]).t()
        return _activate_fp32(v, s["bias"], case["epilogue"]).to(t)
    if kind == "experts":
        at, inside = _segments(s["offsets"], s["most"])
        a = _values_fp32(s["a"], s["sa"], 1)
        a = a[at.clamp_max(a.shape[0] - 1)]
        v = torch.bmm(a, _values_fp32(s["b"], s["sb"], BLOCK).transpose(1, 2))
        v = _activate_fp32(v, None, case["epilogue"]).to(t)
        d = torch.zeros(s["d"].shape[0] + 1, case["n"], dtype=t, device=v.device)
        d[torch.where(inside, at, s["d"].shape[0])] = v
        return d[:-1]
    if kind == "experts_wgrad":
        at, inside = _segments(s["offsets"], s["most"])
        last = s["a"].shape[1] - 1
        a = _values_fp32(s["a"], s["sa"], 1).t()[at.clamp_max(last)] * inside[..., None]
        b = _values_fp32(s["b"], s["sb"], 1).t()[at.clamp_max(last)]
        return torch.bmm(a.transpose(1, 2), b).to(t)
    if kind == "route":
        offsets, row_slot, slot_row = _sorted_by_expert(s["ids"], case["count"], case["align"])
        x = s["x"].float()[row_slot.long().clamp_min(0) // case["top_k"]]
        x = torch.where((row_slot >= 0)[:, None], x, torch.zeros_like(x))
        return (offsets, row_slot, slot_row) + (_blocks_fp32(x, 1) if case["form"] == "fp8"
                                                else (x.to(t),))
    d = _gather_sum_fp32(s["y"], s["slot_row"], s["w"]).to(t)
    if not case["train"]:
        return d
    kept = s["slot_row"] >= 0
    dd = s["dd"].float()
    y = s["y"][s["slot_row"].long().clamp_min(0)].float()
    dw = torch.where(kept, (y * dd[:, None, :]).sum(-1), torch.zeros_like(s["w"]))
    src = s["row_slot"].long().clamp_min(0)
    dy = dd[src // case["top_k"]] * s["w"].reshape(-1)[src][:, None]
    dy = torch.where((s["row_slot"] >= 0)[:, None], dy, torch.zeros_like(dy)).to(t)
    return d, dy, dw, _gather_sum_fp32(s["dxs"], s["slot_row"], None).to(t)


# ------------------------------------------------------------------ exact

def _quantized_exactly(x, block_rows):
    """Codes' values and scales by the definition, in 64 bits."""
    rows, cols = x.shape
    values = torch.zeros_like(x)
    scales = x.new_zeros(_ceil(rows, block_rows), _ceil(cols, BLOCK))
    for j in range(scales.shape[1]):
        part = x[:, j * BLOCK:(j + 1) * BLOCK]
        top = part.abs().amax(1)
        if block_rows > 1:
            top = torch.stack([p.amax() for p in top.split(block_rows)])
        scale = top.clamp_min(FLOOR) / TOP
        scales[:, j] = scale
        v = part / scale.repeat_interleave(block_rows)[:rows, None]
        step = torch.exp2((torch.frexp(v)[1].double() - 1).clamp_min(-6) - 3)
        values[:, j * BLOCK:(j + 1) * BLOCK] = torch.round(v / step) * step
    return values, scales


def _product_exactly(a, sa, b, sb):
    """sum over 128-wide blocks of (a . b^T) times both blocks' scales; sb has one row for each
    row of b, or one for each 128."""
    a, sa = a.double(), sa.double()
    b, sb = b.double(), sb.double()
    if sb.shape[0] != b.shape[0]:
        sb = sb.repeat_interleave(BLOCK, 0)[:b.shape[0]]
    total = a.new_zeros(a.shape[0], b.shape[0])
    for j in range(sa.shape[1]):
        at = slice(j * BLOCK, (j + 1) * BLOCK)
        total += (a[:, at] * sa[:, j:j + 1]) @ (b[:, at] * sb[:, j:j + 1]).t()
    return total


def _activated_exactly(v, bias, epilogue):
    if bias is not None:
        v = v + bias.double()
    if "gelu" in epilogue:
        v = v * torch.special.ndtr(v)
    return v


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quant":
        x = s["x"].double()
        out = _quantized_exactly(x, case["block_rows"])
        return out + _quantized_exactly(x.t().contiguous(), case["block_rows"]) \
            if case["form"] == "both" else out
    if kind == "gemm":
        return _activated_exactly(_product_exactly(s["a"], s["sa"], s["b"], s["sb"]), s["bias"],
                                  case["epilogue"])
    if kind == "experts":
        ends = s["offsets"].tolist()
        d = s["d"].double()
        for e in range(case["count"]):
            at = slice(ends[e], ends[e + 1])
            d[at] = _activated_exactly(_product_exactly(s["a"][at], s["sa"][at], s["b"][e],
                                                        s["sb"][e]), None, case["epilogue"])
        return d
    if kind == "experts_wgrad":
        ends = s["offsets"].tolist()
        d = s["d"].double()
        for e in range(case["count"]):
            at = slice(ends[e], ends[e + 1])
            of = slice(ends[e] // BLOCK, ends[e + 1] // BLOCK)
            d[e] = _product_exactly(s["a"][:, at], s["sa"][:, of], s["b"][:, at], s["sb"][:, of])
        return d
    top_k = case["top_k"]
    if kind == "route":
        ids = s["ids"].tolist()
        filled = [[] for _ in range(case["count"])]
        for t, row in enumerate(ids):
            for j, e in enumerate(row):
                if e >= 0:
                    filled[e].append(t * top_k + j)
        src, at = [], 0
        for slots in filled:
            src += slots + [-1] * (-len(slots) % case["align"])
        src += [-1] * (s["sorted"][1].numel() - len(src))
        src = torch.tensor(src, device="cuda")
        x = s["x"].double()[src.clamp_min(0) // top_k] * (src >= 0)[:, None]
        return (None, None, None) + (_quantized_exactly(x, 1) if case["form"] == "fp8" else (x,))
    slot_row = s["slot_row"].long()
    width = case["width"]

    def back(rows, weights):
        total = torch.zeros(case["tokens"], width, dtype=torch.float64, device="cuda")
        for j in range(top_k):
            w = (slot_row[:, j] >= 0).double() * (1.0 if weights is None
                                                  else weights[:, j].double())
            total += w[:, None] * rows[slot_row[:, j].clamp_min(0)].double()
        return total

    d = back(s["y"], s["w"])
    if not case["train"]:
        return d
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
    dd = s["dd"].double()
    for j in range(top_k):
        t = torch.nonzero(slot_row[:, j] >= 0)[:, 0]
        r = slot_row[t, j]
        dy[r] = s["w"][t, j].double()[:, None] * dd[t]
        dw[t, j] = (s["y"][r].double() * dd[t]).sum(1)
    return d, dy, dw, back(s["dxs"], None)


# ------------------------------------------------------------------- work

def work(case):
    kind = case["kind"]
    z = BYTES[case["type"]]
    if kind == "quant":
        rows, k, br = case["rows"], case["k"], case["block_rows"]
        forms = 1 if case["form"] == "rows" else 2
        scales = _ceil(rows, br) * _ceil(k, BLOCK) + (forms - 1) * _ceil(k, br) * _ceil(rows, BLOCK)
        return {"bytes": rows * k * (z + forms) + 4 * scales, "flops": 2 * rows * k * forms}
    if kind == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = _ceil(k, BLOCK)
        return {"bytes": (m + n) * k + m * n * z + 4 * kb * (m + _ceil(n, case["block_rows"])),
                "flops": 2 * m * n * k}
    slots = case["tokens"] * case["top_k"]
    count = case["count"]
    if kind == "experts":
        n, k = case["n"], case["k"]
        # experts that get a row: of `count`, when each slot's expert is a fair draw
        used = count * (1.0 - (1.0 - case["top_k"] / count) ** case["tokens"])
        return {"bytes": used * n * k * (1 + 4 / BLOCK ** 2) + slots * (k * (1 + 4 / BLOCK) + n * z),
                "flops": 2 * slots * n * k}
    if kind == "experts_wgrad":
        n, k = case["n"], case["k"]
        return {"bytes": slots * (n + k) * (1 + 4 / BLOCK) + count * n * k * z,
                "flops": 2 * slots * n * k}
    width, tokens = case["width"], case["tokens"]
    cap = _capacity(tokens, case["top_k"], count, case["align"])
    if kind == "route":
        out = width * (1 + 4 / BLOCK) if case["form"] == "fp8" else width * z
        return {"bytes": 4 * (2 * slots + cap + count) + tokens * width * z + cap * out,
                "flops": 2 * slots * width if case["form"] == "fp8" else 0}
    if not case["train"]:
        return {"bytes": slots * (8 + width * z) + tokens * width * z, "flops": 2 * slots * width}
    # forward: rows in, tokens out; backward: rows and tokens in, rows out; the way there's
    # gradient: rows in, tokens out
    return {"bytes": 3 * slots * width * z + cap * width * z + 3 * tokens * width * z + 20 * slots,
            "flops": 7 * slots * width}
