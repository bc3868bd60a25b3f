"""Cases and plain forms of the operators around a block's quantized linears.

Grouped products by expert (a router's tokens through low-bit expert weights):
  plan      expert ids -> where each (token, choice) row stands in expert order
  quantize  tokens -> low-bit rows in expert order, one copy per choice
  product   rows in expert order x their expert's low-bit weight
  combine   each token's rows weighted and added
and the step behind the q/k/v projection:
  heads     norm of every q and k head with the position rotation, written in
            16 or 32 bits or quantized to MXFP8 for a low-bit cache

`run` is the plain form in elementary torch operations; with `own` set it
makes the calls a user makes of the library.
"""
import math

import numpy as np
import torch

own = False

# format ids of the library (mxq_fmt)
MXFP8, MXFP4, NVFP4, INT8_ROW, FP8_TENSOR = 0, 1, 2, 5, 6
FMT = {"mxfp8": MXFP8, "mxfp4": MXFP4, "nvfp4": NVFP4, "int8": INT8_ROW, "fp8": FP8_TENSOR}
BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16, "int8": 0, "fp8": 0}
MMA = 1
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a served batch: 48 tokens, 8 of 128 experts
        {"name": "plan_decode", "op": "plan", "tokens": 48, "topk": 8, "experts": 128, "pad": 0.0, "bits": 32},
        # a long prefill over many experts, ids as a top-k returns them (64 bits), padded tokens at -1
        {"name": "plan_prefill", "op": "plan", "tokens": 32768, "topk": 8, "experts": 256, "pad": 0.03, "bits": 64},
        # a decode step's activations, width of the 4096-wide linears
        {"name": "quantize_decode", "op": "quantize", "tokens": 32, "topk": 8, "experts": 64, "pad": 0.0,
         "cols": 4096, "fmt": "mxfp8", "dtype": "bf16"},
        # a prefill's activations
        {"name": "quantize_prefill", "op": "quantize", "tokens": 8192, "topk": 4, "experts": 32, "pad": 0.02,
         "cols": 4096, "fmt": "mxfp8", "dtype": "bf16"},
        # one token through 8 of 64 experts: reading the chosen weights is all there is
        {"name": "product_token_nvfp4", "op": "product", "tokens": 1, "topk": 8, "experts": 64, "pad": 0.0,
         "n": 2048, "cols": 4096, "fmt": "nvfp4", "out": "bf16"},
        # a served batch through the MLP up-projection of the DiT blocks as experts
        {"name": "product_batch_mxfp8", "op": "product", "tokens": 64, "topk": 4, "experts": 32, "pad": 0.05,
         "n": 4608, "cols": 1152, "fmt": "mxfp8", "out": "bf16"},
        # a ragged chunk through few experts, 8-bit integers, widths that end inside a tile
        {"name": "product_chunk_int8", "op": "product", "tokens": 1000, "topk": 2, "experts": 8, "pad": 0.0,
         "n": 1160, "cols": 4608, "fmt": "int8", "out": "bf16"},
        # a prefill through many experts: the tensor cores' share
        {"name": "product_prefill_nvfp4", "op": "product", "tokens": 8192, "topk": 4, "experts": 32, "pad": 0.0,
         "n": 4096, "cols": 4096, "fmt": "nvfp4", "out": "bf16"},
        {"name": "combine_decode", "op": "combine", "tokens": 32, "topk": 8, "experts": 64, "pad": 0.0,
         "n": 4096, "dtype": "bf16"},
        {"name": "combine_prefill", "op": "combine", "tokens": 16384, "topk": 4, "experts": 32, "pad": 0.02,
         "n": 4096, "dtype": "bf16"},
        # a decode step behind a grouped-query q/k/v projection, far positions, halves rotated
        {"name": "heads_decode", "op": "heads", "tokens": 64, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "norm": "rms", "dtype": "bf16", "fmt": "none", "hadamard": 0, "positions": 131072},
        # a prefill whose q and k go to MXFP8 behind a Hadamard rotation of each head
        {"name": "heads_prefill_mxfp8", "op": "heads", "tokens": 8192, "q_heads": 32, "k_heads": 8, "dim": 128,
         "rot": 128, "interleaved": True, "norm": "rms", "dtype": "bf16", "fmt": "mxfp8", "hadamard": 128,
         "positions": 8192},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "quantize", "product", "product", "combine", "heads"])
    if op == "heads":
        tokens = _log(rng, 1, 8192)
        dim = rng.choice([64, 72, 80, 96, 128, 256])
        fmt = rng.choice(["none", "none", "mxfp8"]) if dim % 32 == 0 else "none"
        had = rng.choice([0, dim]) if fmt != "none" and dim & (dim - 1) == 0 else 0
        k_heads = rng.randint(1, 8)
        return {"op": op, "tokens": tokens, "q_heads": k_heads * rng.randint(1, 4), "k_heads": k_heads, "dim": dim,
                "rot": rng.choice([dim, dim // 16 * 8]), "interleaved": rng.random() < 0.5,
                "norm": rng.choice(["rms", "layer"]), "dtype": rng.choice(["bf16", "bf16", "f32"]), "fmt": fmt,
                "hadamard": had, "positions": _log(rng, 64, 131072)}
    experts = _log(rng, 2, 256 if op == "plan" else 64)
    case = {"op": op, "tokens": _log(rng, 1, 32768 if op == "plan" else 8192), "topk": rng.randint(1, min(8, experts)),
            "experts": experts, "pad": rng.choice([0.0, 0.0, 0.05, 0.3])}
    if op == "plan":
        case["bits"] = rng.choice([32, 64])
        return case
    if op == "product":
        case["fmt"] = rng.choice(["nvfp4", "mxfp4", "mxfp8", "int8", "fp8"])
        case["n"] = 8 * rng.randint(16, 256) if rng.random() < 0.8 else rng.randint(100, 2000)
        case["cols"] = 64 * rng.randint(4, 64)
        case["out"] = "bf16"
        while 2.0 * case["tokens"] * case["topk"] * case["n"] * case["cols"] > 8e11:
            case["tokens"] = case["tokens"] // 2
        return case
    if op == "quantize":
        case["cols"] = 64 * rng.randint(4, 64)
        case["topk"] = min(case["topk"], 4)
        case["fmt"] = rng.choice(["mxfp8", "int8", "fp8"])
        case["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        return case
    case["n"] = 8 * rng.randint(16, 512) if rng.random() < 0.8 else rng.randint(100, 4000)
    case["dtype"] = rng.choice(["bf16", "bf16", "f32"])
    return case


# ------------------------------------------------------------------ inputs

def _route(case, g):
    """Distinct expert ids per token from skewed router logits, padded tokens at -1: int64 [tokens, topk]."""
    t, e, k = case["tokens"], case["experts"], case["topk"]
    logits = torch.randn(t, e, generator=g, device="cuda") + 0.7 * torch.randn(e, generator=g, device="cuda")
    top = torch.topk(logits, k, dim=1)
    ids = top.indices
    ids[torch.rand(t, generator=g, device="cuda") < case["pad"]] = -1
    return ids, torch.softmax(top.values, dim=1)


def _place(ids, experts):
    """offsets [experts + 1] and slot [tokens, topk] (int32) of ids, choices of an expert in token order."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel(), device=flat.device)
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = torch.cumsum(counts, 0)
    slot = torch.where(key < experts, place, torch.full_like(place, -1)).to(torch.int32)
    return offsets, slot.reshape(ids.shape)


def _up(a, b):
    return (a + b - 1) // b * b


def _scale_at(row, col, padded_cols):
    """Byte of (row, scale column) in the MMA scale layout."""
    return ((row // 128) * (padded_cols // 4) + col // 4) * 512 + (row % 32) * 16 + ((row % 128) // 32) * 4 + col % 4


def _scale_rows(offsets, rows):
    """Row in the grouped scale layout of every row in expert order: each group begins at a multiple of 128 rows."""
    counts = (offsets[1:] - offsets[:-1]).long()
    tiles = (counts + 127) // 128
    first = torch.cumsum(tiles, 0) - tiles
    j = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:].long().contiguous(), j, right=True).clamp(max=counts.numel() - 1)
    return first[e] * 128 + j - offsets[:-1].long()[e], e


def _scale_bytes(rows, experts, cols, block):
    """Size of the grouped scale layout: no group can need more than one ragged 128-row tile."""
    return (rows // 128 + min(rows, experts)) * 128 * _up(cols // block, 16)


def _e2m1(u):
    """E2M1 codes (sign in bit 3) of u: nearest, ties to the even code."""
    a = u.abs()
    c = sum(((a > m) | ((a == m) if odd else torch.zeros_like(a, dtype=torch.bool))).to(torch.uint8)
            for m, odd in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)))
    return c | ((u < 0).to(torch.uint8) << 3)


def _quantize(x, fmt):
    """(codes uint8 [rows, bytes], byte scales [rows, blocks] or fp32 row scales or None, tensor scale or None) of fp32 x."""
    rows, cols = x.shape
    if fmt == "int8":
        s = x.abs().amax(1) / 127.0
        q = torch.round(x / torch.where(s == 0, torch.ones_like(s), s)[:, None]).clamp(-127, 127)
        return q.to(torch.int8).view(torch.uint8), s, None
    if fmt == "fp8":
        s = (x.abs().amax() if rows else x.new_zeros(())) / 448.0
        s = torch.where(s == 0, torch.ones_like(s), s)
        return (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), None, s.reshape(1)
    b = x.reshape(rows, cols // BLOCK[fmt], BLOCK[fmt])
    amax = b.abs().amax(2)
    if fmt == "nvfp4":
        ts = x.abs().amax() / 2688.0
        ts = torch.where(ts == 0, torch.ones_like(ts), ts)
        e4 = ((amax / 6.0) / ts).clamp(max=448).to(torch.float8_e4m3fn)
        d = e4.float() * ts
        u = torch.where(d[..., None] > 0, b / torch.where(d > 0, d, torch.ones_like(d))[..., None], torch.zeros_like(b))
        scales = e4.view(torch.uint8)
    else:
        ts = None
        e = torch.frexp(amax).exponent.int() - 1 - (8 if fmt == "mxfp8" else 2)
        e = torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))
        u = torch.ldexp(b, -e[..., None])
        scales = (e + 127).to(torch.uint8)
        if fmt == "mxfp8":
            return u.clamp(-448, 448).reshape(rows, cols).to(torch.float8_e4m3fn).view(torch.uint8), scales, None
    c = _e2m1(u.reshape(rows, cols))
    return c[:, 0::2] | (c[:, 1::2] << 4), scales, None if ts is None else ts.reshape(1)


def _rope_tables(n, rot):
    """cos and sin of every position's angles, from 64 bits: fp32 [n, rot / 2]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, s = case["op"], dict(case)
    if op == "heads":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        qkv = torch.randn(t, (hq + 2 * hk) * d, generator=g, device="cuda")
        qkv = (qkv * torch.exp(0.7 * torch.randn((hq + 2 * hk) * d, generator=g, device="cuda"))).to(DTYPE[case["dtype"]])
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["wq"], s["wk"] = (1 + 0.2 * torch.randn(2, d, generator=g, device="cuda")).unbind(0)
        s["cos"], s["sin"] = _rope_tables(case["positions"], case["rot"])
        s["pos"] = torch.randint(0, case["positions"], (t,), generator=g, device="cuda", dtype=torch.int32)
        if case["fmt"] == "none":
            s["out"] = [torch.zeros_like(x.contiguous()) for x in (s["q"], s["k"])]
        else:
            s["out"] = [(torch.zeros(t * h * d, dtype=torch.uint8, device="cuda"),
                         torch.zeros(t * h * d // 32, dtype=torch.uint8, device="cuda")) for h in (hq, hk)]
        return s
    ids, weights = _route(case, g)
    rows = ids.numel()
    if op == "plan":
        s["ids"] = ids.to(torch.int64 if case["bits"] == 64 else torch.int32)
        return s
    s["offsets"], s["slot"] = _place(ids, case["experts"])
    if op == "combine":
        s["y"] = torch.randn(rows, case["n"], generator=g, device="cuda").to(DTYPE[case["dtype"]])
        s["weights"] = weights.contiguous()
        s["out"] = torch.empty(case["tokens"], case["n"], dtype=DTYPE[case["dtype"]], device="cuda")
        return s
    cols, fmt = case["cols"], case["fmt"]
    block = BLOCK[fmt]
    # activations: a few columns far above the others, as the pages' layers have them
    x = torch.randn(case["tokens"], cols, generator=g, device="cuda")
    x = x * torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    if op == "quantize":
        s["x"] = x.to(DTYPE[case["dtype"]])
        s["codes"] = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda")
        s["scales"] = (torch.zeros(_scale_bytes(rows, case["experts"], cols, block), dtype=torch.uint8, device="cuda") if block
                       else torch.zeros(rows * 4, dtype=torch.uint8, device="cuda") if fmt == "int8" else None)
        s["ts"] = torch.zeros(1, device="cuda") if fmt == "fp8" else None
        return s
    # the rows in expert order, quantized
    flat = s["slot"].reshape(-1).long()
    placed = flat >= 0
    xr = torch.zeros(rows, cols, device="cuda")
    xr[flat[placed]] = x.repeat_interleave(case["topk"], 0)[placed].to(torch.bfloat16).float()
    s["xc"], xs, s["xts"] = _quantize(xr, fmt)
    e, n = case["experts"], case["n"]
    w = torch.randn(e, n, cols, generator=g, device="cuda").mul_(0.02)
    parts = [_quantize(w[i], fmt) for i in range(e)]
    s["wc"] = torch.stack([p[0] for p in parts])
    s["wts"] = torch.cat([p[2] for p in parts]) if parts[0][2] is not None else None
    if block:
        sp, np_ = _up(cols // block, 16), _up(n, 128)
        c = torch.arange(cols // block, device="cuda")
        s["xs"] = torch.zeros(_scale_bytes(rows, e, cols, block), dtype=torch.uint8, device="cuda")
        used = int(s["offsets"][-1])
        at = _scale_rows(s["offsets"], rows)[0][:used]
        s["xs"][_scale_at(at[:, None], c[None], sp)] = xs[:used]
        s["ws"] = torch.zeros(e, np_ * sp, dtype=torch.uint8, device="cuda")
        s["ws"][:, _scale_at(torch.arange(n, device="cuda")[:, None], c[None], sp)] = torch.stack([p[1] for p in parts])
    elif fmt == "int8":
        s["xs"], s["ws"] = xs.contiguous(), torch.stack([p[1] for p in parts])
    else:
        s["xs"] = s["ws"] = None
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    s["y"] = torch.zeros(rows, n, dtype=DTYPE[case["out"]], device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _values(codes, fmt, dtype=torch.float32):
    """Values of the codes, last axis unpacked."""
    if fmt in ("mxfp4", "nvfp4"):
        lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
        return torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).to(dtype)


def _scale_values(b, fmt, dtype=torch.float32):
    if fmt == "nvfp4":
        return b.view(torch.float8_e4m3fn).to(dtype)
    return torch.ldexp(torch.ones((), dtype=dtype, device=b.device), b.int() - 127)


def _plain_plan(s):
    flat = s["ids"].reshape(-1).long()
    e = s["experts"]
    key = torch.where((flat >= 0) & (flat < e), flat, torch.full_like(flat, e))
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel(), device=flat.device)
    bounds = torch.searchsorted(key[order], torch.arange(e + 1, device=flat.device))
    slot = torch.where(key < e, place, torch.full_like(place, -1))
    return bounds.to(torch.int32), slot.to(torch.int32).reshape(s["ids"].shape)


def _plain_quantize(s):
    fmt, cols = s["fmt"], s["cols"]
    flat = s["slot"].reshape(-1).long()
    placed = flat >= 0
    x = s["x"].float()
    rows = flat.numel()
    token = torch.arange(rows, device=x.device) // s["topk"]
    xr = torch.zeros(rows + 1, cols, device=x.device)
    xr[torch.where(placed, flat, torch.full_like(flat, rows))] = x[token]
    xr = xr[:rows]
    used = torch.arange(rows, device=x.device) < s["offsets"][-1]
    xr = torch.where(used[:, None], xr, torch.zeros_like(xr))
    codes, scales, ts = _quantize(xr, fmt)
    if fmt == "int8":
        return codes.view(torch.int8), scales
    codes = codes.view(torch.float8_e4m3fn)
    if fmt == "fp8":
        return codes, ts
    at = _scale_rows(s["offsets"], rows)[0]
    sp = _up(cols // 32, 16)
    size = s["scales"].numel()
    where = _scale_at(at[:, None], torch.arange(cols // 32, device=x.device)[None], sp)
    laid = torch.zeros(size + 1, dtype=torch.uint8, device=x.device)
    laid[torch.where(used[:, None], where, torch.full_like(where, size))] = scales
    return codes, laid[:size].view(torch.float8_e8m0fnu)


def _plain_product(s):
    fmt, cols, e, n = s["fmt"], s["cols"], s["experts"], s["n"]
    rows, block = s["y"].shape[0], BLOCK[s["fmt"]]
    x, w = _values(s["xc"], fmt), _values(s["wc"], fmt)
    scale_row, group = _scale_rows(s["offsets"], rows)
    if block:
        sp = _up(cols // block, 16)
        c = torch.arange(cols // block, device=x.device)
        at = _scale_at(scale_row[:, None], c[None], sp).clamp(max=s["xs"].numel() - 1)
        x = (x.unflatten(1, (-1, block)) * _scale_values(s["xs"][at], fmt)[..., None]).flatten(1)
        at = _scale_at(torch.arange(n, device=x.device)[:, None], c[None], sp)
        w = (w.unflatten(2, (-1, block)) * _scale_values(s["ws"][:, at], fmt)[..., None]).flatten(2)
    elif fmt == "int8":
        x, w = x * s["xs"][:, None], w * s["ws"][..., None]
    if s["xts"] is not None:
        x, w = x * s["xts"], w * s["wts"][:, None, None]
    within = torch.arange(rows, device=x.device) - s["offsets"][:-1].long()[group]
    used = torch.arange(rows, device=x.device) < s["offsets"][-1]
    at = torch.where(used, group * s["most"] + within, torch.full_like(within, e * s["most"]))
    padded = torch.zeros(e * s["most"] + 1, cols, device=x.device)
    padded[at] = x
    y = torch.bmm(padded[:-1].view(e, s["most"], cols), w.transpose(1, 2)).reshape(-1, n)
    y = y[at.clamp(max=e * s["most"] - 1)] if y.shape[0] else torch.zeros(rows, n, device=x.device)
    return torch.where(used[:, None], y, torch.zeros_like(y)).to(DTYPE[s["out"]])


def _plain_combine(s):
    flat = s["slot"].long()
    y = s["y"].float()[flat.clamp(min=0)] * torch.where(flat >= 0, s["weights"], torch.zeros_like(s["weights"]))[..., None]
    return y.sum(1).to(s["y"].dtype)


def _rotate(x, cos, sin, rot, interleaved):
    """The first `rot` elements of every head turned by its position's angles."""
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([r, rest], -1)


def _hadamard(x, b):
    """Every block of b elements times the orthonormal Sylvester matrix."""
    h = torch.ones(1, 1, dtype=x.dtype, device=x.device)
    while h.shape[0] < b:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return (x.unflatten(-1, (-1, b)) @ (h / math.sqrt(b))).flatten(-2)


def _plain_heads(s):
    cos, sin = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        v = x.float()
        if s["norm"] == "layer":
            v = v - v.mean(-1, keepdim=True)
        v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w
        v = _rotate(v, cos, sin, s["rot"], s["interleaved"])
        if s["fmt"] == "none":
            out.append(v.to(x.dtype))
            continue
        if s["hadamard"]:
            v = _hadamard(v, s["hadamard"])
        codes, scales, _ = _quantize(v.flatten(0, 1), "mxfp8")
        out += [codes.view(torch.float8_e4m3fn).flatten(), scales.view(torch.float8_e8m0fnu).flatten()]
    return out


def run(s):
    op = s["op"]
    if own:
        import microscaling_bit_quantization_b200 as mxq
        if op == "plan":
            plan = mxq.expert_plan(s["ids"], s["experts"])
            return plan.offsets, plan.slot
        if op == "quantize":
            rows, cols = s["codes"].shape
            q = mxq.QTensor(FMT[s["fmt"]], MMA, rows, cols, s["codes"], s["scales"], s["ts"])
            mxq.quantize_grouped(s["x"], FMT[s["fmt"]], s["offsets"], s["slot"], out=q)
            if s["fmt"] == "int8":
                return s["codes"].view(torch.int8), s["scales"].view(torch.float32)
            codes = s["codes"].view(torch.float8_e4m3fn)
            return codes, s["ts"] if s["fmt"] == "fp8" else s["scales"].view(torch.float8_e8m0fnu)
        if op == "product":
            xq = mxq.QTensor(FMT[s["fmt"]], MMA, s["y"].shape[0], s["cols"], s["xc"], s["xs"], s["xts"])
            w = mxq.ExpertWeight(FMT[s["fmt"]], s["experts"], s["n"], s["cols"], s["wc"], s["ws"], s["wts"])
            return mxq.qlinear_grouped(xq, w, s["offsets"], out=s["y"])
        if op == "combine":
            return mxq.expert_combine(s["y"], s["slot"], s["weights"], out=s["out"])
        more = dict(eps=1e-6, norm=s["norm"], interleaved=s["interleaved"])
        if s["fmt"] == "none":
            return mxq.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], q_out=s["out"][0],
                                    k_out=s["out"][1], **more)
        t, d = s["tokens"], s["dim"]
        qs = [mxq.QTensor(MXFP8, 0, t * h, d, *s["out"][i], None) for i, h in enumerate((s["q_heads"], s["k_heads"]))]
        mxq.qk_norm_rope_quantize(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], fmt=MXFP8,
                                  hadamard_b=s["hadamard"], q_out=qs[0], k_out=qs[1], **more)
        return [v for c, e in s["out"] for v in (c.view(torch.float8_e4m3fn), e.view(torch.float8_e8m0fnu))]
    return {"plan": _plain_plan, "quantize": _plain_quantize, "product": _plain_product, "combine": _plain_combine,
            "heads": _plain_heads}[op](s)


# ------------------------------------------------------------------ work

def _used_rows(case):
    return case["tokens"] * case["topk"] * (1 - case["pad"])


def _busy_experts(case):
    """Expected experts with a row, were the choices spread evenly."""
    share = case["topk"] / case["experts"]
    return case["experts"] * (1 - (1 - share) ** (case["tokens"] * (1 - case["pad"])))


def work(case):
    op = case["op"]
    if op == "heads":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        esz = 2 if case["dtype"] == "bf16" else 4
        one = t * (hq + hk) * d
        out = one * esz if case["fmt"] == "none" else one + one / 32
        angles = min(t, case["positions"]) * case["rot"] * 4
        had = math.log2(case["hadamard"]) if case["hadamard"] else 0
        return {"bytes": one * esz + out + angles + t * 4 + 8 * d, "flops": one * (8 + had)}
    rows = case["tokens"] * case["topk"]
    if op == "plan":
        return {"bytes": rows * (case["bits"] // 8 + 4) + 4 * (case["experts"] + 1), "flops": rows}
    used = _used_rows(case)
    if op == "combine":
        esz = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": (used + case["tokens"]) * case["n"] * esz + rows * 8, "flops": 2 * used * case["n"]}
    cols, fmt = case["cols"], case["fmt"]
    per = {"mxfp8": 1 + 1 / 32, "mxfp4": 0.5 + 1 / 32, "nvfp4": 0.5 + 1 / 16, "int8": 1.0, "fp8": 1.0}[fmt]
    if op == "quantize":
        esz = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["tokens"] * (1 - case["pad"]) * cols * esz + used * cols * per + rows * 4,
                "flops": 3 * used * cols}
    esz = 2 if case["out"] == "bf16" else 4
    weights = _busy_experts(case) * case["n"] * cols * per
    return {"bytes": weights + used * cols * per + used * case["n"] * esz, "flops": 2 * used * case["n"] * cols}


# ------------------------------------------------------------------ 64 bits

def _round_e4m3(u):
    """Nearest E4M3 value of float64 u, ties to the even code, saturating at 448."""
    m, e = torch.frexp(u)
    step = torch.ldexp(torch.ones_like(u), torch.clamp(e - 1, min=-6).int() - 3)
    return (torch.round(u / step) * step).clamp(-448.0, 448.0)


def _exact_mxfp8(v):
    """(values of the codes, values of the block scales) of float64 rows under the OCP rule."""
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1)
    exp = torch.where(top > 0, (torch.frexp(top).exponent.long() - 9).clamp(-127, 127), torch.zeros_like(top).long())
    scale = torch.ldexp(torch.ones_like(top), exp.int())
    return _round_e4m3(b / scale[..., None]).reshape(v.shape), scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "heads":
        out = []
        half = case["rot"] // 2
        pos = s["pos"].long()
        c, sn = s["cos"].double()[pos], s["sin"].double()[pos]
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            v = x.double()
            if case["norm"] == "layer":
                v = v - v.sum(-1, keepdim=True) / case["dim"]
            v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / case["dim"] + 1e-6) * w.double()
            z = v.clone()
            for i in range(half):
                p, q = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
                z[..., p] = v[..., p] * c[:, None, i] - v[..., q] * sn[:, None, i]
                z[..., q] = v[..., q] * c[:, None, i] + v[..., p] * sn[:, None, i]
            if case["fmt"] == "none":
                out.append(z)
                continue
            if case["hadamard"]:
                bits = np.arange(case["hadamard"])
                signs = np.array([[(-1.0) ** bin(i & j).count("1") for j in bits] for i in bits])
                m = torch.from_numpy(signs / math.sqrt(case["hadamard"])).cuda()
                z = torch.einsum("thbi,ij->thbj", z.unflatten(-1, (-1, case["hadamard"])), m).flatten(-2)
            values, scale = _exact_mxfp8(z.flatten(0, 1))
            out += [values.flatten(), scale.flatten()]
        return out
    off = s["offsets"].tolist()
    slot = s["slot"].cpu().numpy()
    if op == "combine":
        out = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device="cuda")
        y, w = s["y"].double(), s["weights"].double()
        for i in range(case["topk"]):
            at = s["slot"][:, i].long()
            out[at >= 0] += w[at >= 0, i, None] * y[at[at >= 0]]
        return out
    fmt, cols = case["fmt"], case["cols"]
    rows = slot.size
    if op == "quantize":
        token, choice = np.nonzero(slot >= 0)
        xr = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
        xr[torch.from_numpy(slot[token, choice]).long().cuda()] = s["x"].double()[torch.from_numpy(token).cuda()]
        if fmt == "int8":
            return None, xr.abs().amax(1) / 127.0
        if fmt == "fp8":
            ts = float(xr.abs().max()) / 448.0 if rows else 0.0
            ts = float(np.float32(ts)) or 1.0
            return _round_e4m3((xr / ts).float().double()), torch.tensor([ts], dtype=torch.float64)
        values, scale = _exact_mxfp8(xr)
        sp = (cols // 32 + 15) // 16 * 16
        laid = torch.full((s["scales"].numel(),), 2.0 ** -127, dtype=torch.float64, device="cuda")
        tile = 0
        for e in range(case["experts"]):
            count = off[e + 1] - off[e]
            r = 128 * tile + torch.arange(count, device="cuda")[:, None]
            j = torch.arange(cols // 32, device="cuda")[None]
            laid[((r >> 7) * (sp >> 2) + (j >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (j & 3)] = scale[off[e]:off[e + 1]]
            tile += (count + 127) >> 7
        return values, laid
    block, n = BLOCK[fmt], case["n"]
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")

    def matrix(codes, scales, first_row, ts):
        if fmt == "int8":
            return codes.view(torch.int8).double() * scales.double()[:, None]
        if fmt == "fp8":
            return codes.view(torch.float8_e4m3fn).double() * ts.double()
        if fmt == "mxfp8":
            v = codes.view(torch.float8_e4m3fn).double()
        else:
            v = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device="cuda")
            v[:, 0::2], v[:, 1::2] = lut[(codes % 16).long()], lut[(codes // 16).long()]
        sp = (cols // block + 15) // 16 * 16
        r = first_row + torch.arange(codes.shape[0], device="cuda")[:, None]
        j = torch.arange(cols // block, device="cuda")[None]
        b = scales[((r >> 7) * (sp >> 2) + (j >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (j & 3)]
        f = b.view(torch.float8_e4m3fn).double() * ts.double() if fmt == "nvfp4" else torch.exp2(b.double() - 127)
        return v * f.repeat_interleave(block, 1)

    y = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    tile = 0
    for e in range(case["experts"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            xe = matrix(s["xc"][lo:hi], s["xs"][lo:hi] if fmt == "int8" else s["xs"], 128 * tile, s["xts"])
            we = matrix(s["wc"][e], s["ws"][e] if s["ws"] is not None else None, 0, None if s["wts"] is None else s["wts"][e])
            y[lo:hi] = xe @ we.T
        tile += (hi - lo + 127) >> 7
    return y
