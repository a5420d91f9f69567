"""The 4-bit floating-point operators, case by case: quantisation, product, product grouped by expert.

A matrix is held as 4-bit E2M1 codes (two a byte, the even column in the low
half, rows padded to 32 columns) with one scale a block of columns:

  mxfp4  blocks of 32 columns, scale 2^e (one byte, e + 127),
         e = floor(log2 of the block's largest magnitude) - 2
  nvfp4  blocks of 16 columns, scale s in E4M3, and one fp32 scale t for the
         matrix (each expert's rows): t = largest magnitude / 2688 rounded to
         fp32, s = E4M3 nearest to (block's largest magnitude) / (6 t)

A value is code * s * t with the code nearest to x / (s t), ties to the even
code.  Scale bytes are stored in tiles of 128 rows x 4 blocks (512 bytes, row r
at 16 (r % 32) + 4 (r / 32)), each expert's rows starting a new tile.
"""
import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16}


def listed():
    return [
        # One token's activations on their way into a 4-bit layer: the shortest call there is.
        {"name": "quantize_token", "op": "quantize", "format": "nvfp4", "dtype": "bf16", "tokens": 1, "n": 4096, "experts": 0, "top": 0},
        # A prompt's activations (8192 tokens) before a projection, with outlier channels.
        {"name": "quantize_prompt", "op": "quantize", "format": "nvfp4", "dtype": "bf16", "tokens": 8192, "n": 4096, "experts": 0, "top": 0},
        # A layer's fp32 weights turned into mxfp4 once, with the values that they now stand for.
        {"name": "quantize_weight", "op": "quantize", "format": "mxfp4", "dtype": "f32", "tokens": 11008, "n": 4096, "experts": 0, "top": 0},
        # Dispatch to experts: each token's row gathered to its four experts, a scale for each expert, a width that ends inside a tile.
        {"name": "quantize_dispatch", "op": "quantize", "format": "nvfp4", "dtype": "bf16", "tokens": 1500, "n": 2056, "experts": 24, "top": 4},
        # A layer on one token: quantise and multiply, fp32 out as the packed matvec has it.
        {"name": "linear_token", "op": "matmul", "format": "nvfp4", "dtype": "f32", "tokens": 1, "n": 4096, "rows": 4096, "raw": True, "experts": 0, "top": 0},
        # A layer on a batch of 48 sequences that decode together.
        {"name": "linear_decode", "op": "matmul", "format": "mxfp4", "dtype": "bf16", "tokens": 48, "n": 4096, "rows": 11008, "raw": True, "experts": 0, "top": 0},
        # Odd sizes everywhere: tokens, width and rows that fill no tile.
        {"name": "product_odd", "op": "matmul", "format": "mxfp4", "dtype": "bf16", "tokens": 777, "n": 2000, "rows": 1111, "raw": False, "experts": 0, "top": 0},
        # A prompt through a wide projection whose input another projection has quantised already.
        {"name": "product_prompt", "op": "matmul", "format": "nvfp4", "dtype": "bf16", "tokens": 8192, "n": 4096, "rows": 11008, "raw": False, "experts": 0, "top": 0},
        # One token through its four experts of 32: four short products in one call.
        {"name": "experts_token", "op": "grouped", "format": "nvfp4", "dtype": "bf16", "tokens": 1, "n": 4096, "rows": 2048, "raw": True, "experts": 32, "top": 4},
        # 64 decoding sequences through 32 experts: a few rows each, every expert's weights read.
        {"name": "experts_decode", "op": "grouped", "format": "mxfp4", "dtype": "bf16", "tokens": 64, "n": 4096, "rows": 2048, "raw": True, "experts": 32, "top": 4},
        # Few experts of odd sizes, ragged and unevenly loaded.
        {"name": "experts_odd", "op": "grouped", "format": "mxfp4", "dtype": "bf16", "tokens": 333, "n": 1000, "rows": 700, "raw": True, "experts": 7, "top": 2},
        # A prompt's 16384 dispatched rows through 32 experts, quantised before.
        {"name": "experts_prompt", "op": "grouped", "format": "nvfp4", "dtype": "bf16", "tokens": 4096, "n": 2048, "rows": 4096, "raw": False, "experts": 32, "top": 4},
    ]


def _spread(rng, low, high):
    """A whole number, spread over its logarithm."""
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "grouped"])
    form = rng.choice(["mxfp4", "nvfp4"])
    if op == "quantize":
        experts = rng.choice([0, 0, _spread(rng, 2, 64)])
        top = rng.randint(1, min(8, experts)) if experts else 0
        n = _spread(rng, 48, 11008)
        most = 8192 * 4096 // (n * max(1, top))
        return {"op": op, "format": form, "dtype": rng.choice(["bf16", "f32"]), "tokens": _spread(rng, 1, min(8192, most)), "n": n,
                "experts": experts, "top": top}
    n, rows = _spread(rng, 96, 11008), _spread(rng, 64, 11008)
    if op == "matmul":
        tokens = _spread(rng, 1, min(8192, 8192 * 4096 * 11008 // (n * rows)))
        return {"op": op, "format": form, "dtype": rng.choice(["bf16", "f32"]) if tokens <= 64 else "bf16", "tokens": tokens, "n": n, "rows": rows,
                "raw": rng.random() < 0.5, "experts": 0, "top": 0}
    experts = _spread(rng, 2, max(2, min(64, 32 * 4096 * 2048 // (n * rows))))
    top = rng.randint(1, min(8, experts))
    tokens = _spread(rng, 1, max(1, min(4096, 8192 * 2048 * 4096 // (n * rows * top))))
    return {"op": op, "format": form, "dtype": "bf16", "tokens": tokens, "n": n, "rows": rows, "raw": rng.random() < 0.5, "experts": experts, "top": top}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _activations(tokens, n, gen):
    """N(0, 1) with one channel in a hundred scaled up twenty times, as layer inputs have them."""
    x = torch.randn((tokens, n), generator=gen, device="cuda")
    outlier = torch.rand(n, generator=gen, device="cuda") < 0.01
    return x * torch.where(outlier, 20.0, 1.0)


def _route(tokens, experts, top, gen):
    """Each token's `top` experts of an uneven router, as rows sorted by expert:
    the token of each row, where each expert's rows begin, and the most that one has."""
    logits = torch.randn((tokens, experts), generator=gen, device="cuda") + 0.5 * torch.randn(experts, generator=gen, device="cuda")
    expert = torch.topk(logits, top, dim=1).indices.reshape(-1)
    order = torch.argsort(expert, stable=True)
    counts = torch.bincount(expert, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return (order // top).to(torch.int32), offsets, int(counts.max())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    form, tokens, n, experts = case["format"], case["tokens"], case["n"], case["experts"]
    state = {"case": case, "index": None, "offsets": None, "most": tokens}
    if experts:
        state["index"], state["offsets"], state["most"] = _route(tokens, experts, case["top"], gen)
    if case["op"] == "quantize":
        x = _activations(tokens, n, gen)
        state["x"] = x if case["dtype"] == "f32" else x.to(torch.bfloat16)
        return state
    x = _activations(tokens, n, gen).to(torch.bfloat16)
    if case["raw"]:
        state["x"] = x
    else:
        state["x"] = _packed(x if not experts else x[state["index"].long()], form, state["offsets"])
    groups = max(1, experts)
    w = 0.02 * torch.randn((groups * case["rows"], n), generator=gen, device="cuda")
    at = torch.arange(groups + 1, dtype=torch.int32, device="cuda") * case["rows"]
    state["w"] = _packed(w.to(torch.bfloat16), form, at)
    return state


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------


def _group_of(rows, offsets):
    """The group (expert) of each of `rows` rows."""
    at = torch.arange(rows, device=offsets.device, dtype=torch.int32)
    return torch.searchsorted(offsets, at, right=True) - 1


def _quantized(x, form, offsets):
    """Codes' values, block scales and tensor scales of x [rows, n], rows in groups at `offsets`;
    in 64 bits, as values next to a rounding border decide the code."""
    rows, n = x.shape
    block = BLOCK[form]
    pad = -n % block
    x = torch.nn.functional.pad(x.double(), (0, pad)).reshape(rows, -1, block)
    most = x.abs().amax(-1)
    t = torch.ones(offsets.numel() - 1, device=x.device)
    if form == "mxfp4":
        scale = torch.ldexp(torch.ones_like(most), torch.where(most > 0, torch.frexp(most).exponent - 3, -127).clamp(-127, 127))
        unit = scale
    else:
        group = _group_of(rows, offsets)
        tensor_most = torch.zeros(t.numel(), dtype=torch.float64, device=x.device).scatter_reduce(0, group, most.amax(-1), "amax")
        t = (tensor_most / torch.full_like(tensor_most, 2688.0)).float().clamp_min(2.0 ** -126)  # a true quotient: by a number torch takes the reciprocal
        share = most / (6.0 * t.double()[group])[:, None]
        step = torch.ldexp(torch.ones_like(share), (torch.frexp(share).exponent - 1).clamp_min(-6) - 3)
        scale = (torch.round(share / step) * step).clamp_max(448.0)
        unit = scale * t.double()[group][:, None]
    q = torch.where(unit[..., None] > 0, x / unit[..., None], 0.0)
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp_max(6.0) * torch.sign(q), scale, t


def _tile_rows(rows, offsets):
    """The row of the scale tiles that holds each row's scales, and how many tiles there may be."""
    group = _group_of(rows, offsets)
    counts = (offsets[1:] - offsets[:-1]).long()
    tiles = (counts + 127) // 128
    first = torch.cumsum(tiles, 0) - tiles
    at = torch.arange(rows, device=offsets.device)
    return first[group] * 128 + at - offsets[group].long(), rows // 128 + counts.numel()


def _whole(rows):
    return torch.tensor([0, rows], dtype=torch.int32, device="cuda")


def _packed(x, form, offsets):
    """A quantised matrix as a program keeps it between calls."""
    rows, n = x.shape
    groups = 1 if offsets is None else offsets.numel() - 1
    offsets = _whole(rows) if offsets is None else offsets
    value, scale, t = _quantized(x, form, offsets)
    code = torch.bucketize(value.abs().float(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")).to(torch.uint8)
    code = (code + 8 * (value < 0).to(torch.uint8)).reshape(rows, -1)
    code = torch.nn.functional.pad(code, (0, -n % 32 - (-n % BLOCK[form])))
    packed = code[:, 0::2] + 16 * code[:, 1::2]
    exponent = torch.frexp(scale).exponent
    if form == "mxfp4":
        byte = exponent + 126
    else:
        e = (exponent - 1).clamp_min(-6)
        byte = torch.where(scale > 0, torch.round(torch.ldexp(scale, 3 - e)).to(torch.int32) + (e + 6) * 8, 0)
    row, tiles = _tile_rows(rows, offsets)
    quads = (byte.shape[1] + 3) // 4
    table = torch.zeros((tiles * 128, quads * 4), dtype=torch.uint8, device="cuda")
    table[row, : byte.shape[1]] = byte.to(torch.uint8)
    tiled = table.reshape(tiles, 4, 32, quads, 4).permute(0, 3, 2, 1, 4).reshape(tiles, quads, 512)
    return {"packed": packed.contiguous(), "scales": tiled.contiguous(), "tensor_scale": t if form == "nvfp4" else None, "rows": rows, "n": n,
            "format": form, "groups": groups}


def _values(q, offsets):
    """code * s of a packed matrix, exact in 32 bits."""
    rows, form = q["rows"], q["format"]
    byte = q["packed"].long()
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device="cuda")
    code = table[torch.stack((byte & 15, byte >> 4), -1).reshape(rows, -1)]
    tiles, quads = q["scales"].shape[:2]
    flat = q["scales"].reshape(tiles, quads, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tiles * 128, quads * 4)
    b = flat[_tile_rows(rows, offsets)[0]].int()
    if form == "mxfp4":
        scale = torch.ldexp(torch.ones_like(b, dtype=torch.float32), b - 127)
    else:
        scale = torch.ldexp(((b & 7) + 8 * (b >= 8)).float(), (b >> 3).clamp_min(1) - 10)
    n = q["n"]
    return code[:, :n] * torch.repeat_interleave(scale, BLOCK[form], dim=1)[:, :n]


def _plain_quantize(x, form, index, offsets):
    x = x if index is None else x[index.long()]
    at = _whole(x.shape[0]) if offsets is None else offsets
    value, scale, t = _quantized(x, form, at)
    values = (value * scale[..., None]).float().reshape(x.shape[0], -1)[:, : x.shape[1]]
    return values, t, at


def _plain_product(w, x, tx, offsets, most, dtype):
    """y = tw tx X W^T, each row of x with its group's weights (padded to the longest group)."""
    groups = w["groups"]
    rows = w["rows"] // groups
    at = torch.arange(groups + 1, dtype=torch.int32, device="cuda") * rows
    weights = _values(w, at).reshape(groups, rows, -1)
    tw = torch.ones(groups, device="cuda") if w["tensor_scale"] is None else w["tensor_scale"]
    if groups == 1:
        y = x @ weights[0].T * tw * tx
    else:
        group = _group_of(x.shape[0], offsets)
        place = torch.arange(x.shape[0], device="cuda") - offsets[group].long()
        padded = torch.zeros((groups, most, x.shape[1]), device="cuda")
        padded[group, place] = x
        y = torch.bmm(padded, weights.transpose(1, 2))[group, place] * (tw * tx)[group][:, None]
    return y.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def run(state):
    case, index, offsets = state["case"], state["index"], state["offsets"]
    form = case["format"]
    if own:
        import post_weight_quantization_accum_b200 as gq

        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case["op"] == "quantize":
            q = gq.gptq_fp4_quantize(state["x"], form, row_index=index, offsets=offsets, want_deq=True)
            return {"values": q["deq"], "tensor_scale": q["tensor_scale"]}
        if case["raw"]:
            return {"y": gq.fp4_linear(state["w"], state["x"], dtype=dtype, row_index=index, offsets=offsets)}
        if case["op"] == "matmul":
            return {"y": gq.gptq_fp4_matmul(state["w"], state["x"], dtype=dtype)}
        return {"y": gq.gptq_fp4_grouped_matmul(state["w"], state["x"], offsets, dtype=dtype)}
    if case["op"] == "quantize":
        values, t, at = _plain_quantize(state["x"], form, index, offsets)
        return {"values": values * t[_group_of(values.shape[0], at)][:, None], "tensor_scale": t if form == "nvfp4" else None}
    if case["raw"]:
        x, tx, at = _plain_quantize(state["x"], form, index, offsets)
    else:
        at = _whole(state["x"]["rows"]) if offsets is None else offsets
        x, tx = _values(state["x"], at), state["x"]["tensor_scale"]
    return {"y": _plain_product(state["w"], x, 1.0 if tx is None else tx, at, state["most"], case["dtype"])}


def work(case):
    form, n, experts = case["format"], case["n"], case["experts"]
    held = 0.5 + 1.0 / BLOCK[form]  # bytes a quantised value takes
    rows = case["tokens"] * max(1, case["top"])
    if case["op"] == "quantize":
        read = case["tokens"] * n * (4 if case["dtype"] == "f32" else 2) + 4 * rows * (case["top"] > 0)
        return {"bytes": read + rows * n * (held + 4), "flops": 4.0 * rows * n}
    x = case["tokens"] * n * 2 if case["raw"] else rows * n * held
    weights = min(max(1, experts), rows) * case["rows"] * n * held
    return {"bytes": x + weights + rows * case["rows"] * (4 if case["dtype"] == "f32" else 2), "flops": 2.0 * rows * n * case["rows"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits, by tables of the formats' values
# ---------------------------------------------------------------------------


def _nearest(a, table):
    """Index of the entry of `table` (rising) nearest to each a >= 0, ties to the even index, the last one where a is over it."""
    middle = (table[1:] + table[:-1]) / 2
    at = torch.searchsorted(middle, a.contiguous())
    tie = (at < middle.numel()) & (middle[at.clamp_max(middle.numel() - 1)] == a)
    return at + (tie & (at % 2 == 1)).long()


def _tables():
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    e4m3 = torch.tensor([(i & 7) * 2.0 ** -9 if i < 8 else (8 + (i & 7)) * 2.0 ** ((i >> 3) - 10) for i in range(127)], dtype=torch.float64, device="cuda")
    e8m0 = torch.tensor([2.0 ** (i - 127) for i in range(255)], dtype=torch.float64, device="cuda")
    return e2m1, e4m3, e8m0


def _exact_values(x, form, offsets):
    """What the quantised rows of one group after another stand for."""
    e2m1, e4m3, e8m0 = _tables()
    block = BLOCK[form]
    bounds = [0, x.shape[0]] if offsets is None else offsets.tolist()
    parts, ts = [], []
    for first, last in zip(bounds[:-1], bounds[1:]):
        v = x[first:last].double()
        v = torch.cat((v, v.new_zeros((last - first, -x.shape[1] % block))), 1).reshape(last - first, (x.shape[1] + block - 1) // block, block)
        m = v.abs().max(-1).values if last > first else v.new_zeros(v.shape[:2])
        if form == "mxfp4":
            bits = (m.view(torch.int64) >> 52) & 2047  # the exponent of a double, 1023 more than floor(log2)
            unit = e8m0[torch.where(m > 0, bits - 1023 - 2, torch.full_like(bits, -127)).clamp(-127, 127) + 127]
            ts.append(1.0)
        else:
            top = float(m.max()) if m.numel() else 0.0
            t = max(float(torch.tensor(top / 2688.0, dtype=torch.float64).to(torch.float32)), 2.0 ** -126)
            unit = e4m3[_nearest(m / (6 * t), e4m3)] * t
            ts.append(t)
        u = unit[..., None]
        q = torch.where(u > 0, v.abs() / u, torch.zeros_like(v))
        parts.append((torch.copysign(e2m1[_nearest(q, e2m1)], v) * u).flatten(1)[:, : x.shape[1]])
    return torch.cat(parts), torch.tensor(ts, dtype=torch.float64, device="cuda")


def _exact_unpacked(q, bounds):
    """What a packed matrix stands for, group by group, without the tensor scales' product."""
    e2m1, e4m3, e8m0 = _tables()
    code = torch.empty((q["rows"], 2 * q["packed"].shape[1]), dtype=torch.long, device="cuda")
    code[:, 0::2], code[:, 1::2] = (q["packed"] % 16).long(), (q["packed"] // 16).long()
    value = e2m1[code % 8] * (1 - 2 * (code // 8))
    block, tile, parts = BLOCK[q["format"]], 0, []
    j = torch.arange(q["n"], device="cuda") // block
    for g, (first, last) in enumerate(zip(bounds[:-1], bounds[1:])):
        r = torch.arange(last - first, device="cuda")[:, None]
        byte = q["scales"][tile + r // 128, j[None] // 4, r % 32 * 16 + r % 128 // 32 * 4 + j[None] % 4].long()
        s = (e8m0 if q["format"] == "mxfp4" else e4m3)[byte]
        if q["tensor_scale"] is not None:
            s = s * q["tensor_scale"][g].double()
        parts.append(value[first:last, : q["n"]] * s)
        tile += (last - first + 127) // 128
    return parts


def exact(case, seed):
    state = prepare(case, seed)
    form, offsets = case["format"], state["offsets"]
    if case["op"] == "quantize" or case["raw"]:
        x = state["x"] if state["index"] is None else state["x"].index_select(0, state["index"])
        values, ts = _exact_values(x, form, offsets)
        if case["op"] == "quantize":
            return {"values": values, "tensor_scale": ts if form == "nvfp4" else None}
    bounds = [0, case["tokens"]] if offsets is None else offsets.tolist()
    if not case["raw"]:
        values = torch.cat(_exact_unpacked(state["x"], bounds))
    groups = max(1, case["experts"])
    weights = _exact_unpacked(state["w"], [g * case["rows"] for g in range(groups + 1)])
    return {"y": torch.cat([values[a:b] @ w.T for a, b, w in zip(bounds[:-1], bounds[1:], weights)])}
