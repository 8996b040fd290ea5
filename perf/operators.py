"""The operators around the MoE layer of a decoder block, measured: expert routing with groups, the
norms before and after a block with its gate and residual, writing a quantised paged key-value cache
and reading it back, and the attention of one new token a sequence over that cache.

Every case is a dict of plain values; ``prepare`` makes its inputs on the GPU, ``run`` computes the
operator either in its plain form (elementary torch operations, ``own`` false) or through the
library's entry points (``own`` true), ``exact`` computes it from the definition in 64 bits.

Definitions (H heads of keys and values, G query heads for each, D values a head):

* route: s = softmax(l) over the E experts, or sigmoid(l); c = s + bias, or the logits themselves
  where there is no bias (both scores rise with the logit). A group's score is its largest c, or the
  sum of its two largest s + bias; the best groups are kept, then the k experts of largest c in them,
  equal values to the lower index. The weights are s of the chosen, renormalised if asked, times a
  factor.
* norm: h = residual + alpha * gate * norm_post(z); y = norm_pre(h). RMS: x / sqrt(mean(x^2) + eps)
  * w; layer: (x - mean) / sqrt(var + eps) * w + b.
* cache: blocks of 16 tokens of one head are one record: the K codes, the V codes, the K and V block
  scales (NVFP4), the K and V row exponents (FP8 and NVFP4). FP8: the row scale r is the least power of
  two with amax / r <= 448, the codes are E4M3 of x / r. NVFP4: the least with amax / r <= 6 * 448, an
  E4M3 scale s of amax16 / r / 6 for every 16 values, codes E2M1 of x / r / s. Exponents are kept with
  127 added and from 0 to 254.
* attn: softmax(scale * q . k over the last `window` tokens, or all, and one sink logit a head) . v
"""
import numpy as np
import torch

own = False

FMTS = ("bf16", "fp16", "fp8", "nvfp4")
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a Nemotron-3-Nano-like layer: the latency of the routing step
        {"name": "route_one", "op": "route", "T": 1, "E": 128, "k": 6, "score": "sigmoid", "bias": True,
         "groups": 1, "keep": 1, "gscore": "max", "renorm": True, "factor": 1.0, "logits": "fp32"},
        # a decode batch of a gpt-oss-20b-like layer, router logits straight from a bf16 product
        {"name": "route_batch", "op": "route", "T": 333, "E": 32, "k": 4, "score": "softmax", "bias": False,
         "groups": 1, "keep": 1, "gscore": "max", "renorm": True, "factor": 1.0, "logits": "bf16"},
        # a prefill chunk of a model with 256 experts in 8 groups and a balancing bias
        {"name": "route_prefill", "op": "route", "T": 8192, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "gscore": "top2", "renorm": True, "factor": 2.5, "logits": "fp32"},
        # one token between two blocks of width 2880: pure latency
        {"name": "norm_one", "op": "norm", "T": 1, "H": 2880, "act": "bf16", "res": "bf16", "gate": "none",
         "post": "rms", "pre": "rms", "alpha": 1.0},
        # a decode batch of width 2688 with a 32-bit residual stream, a gate and layer norms
        {"name": "norm_batch", "op": "norm", "T": 100, "H": 2688, "act": "bf16", "res": "fp32", "gate": "full",
         "post": "layer", "pre": "layer", "alpha": 0.5},
        # a prefill chunk of width 2880: memory bandwidth
        {"name": "norm_prefill", "op": "norm", "T": 8192, "H": 2880, "act": "bf16", "res": "bf16", "gate": "row",
         "post": "rms", "pre": "rms", "alpha": 1.0},
        # a decode batch's new tokens into a 4-bit cache
        {"name": "cache_decode", "op": "cache", "T": 64, "H": 8, "D": 64, "fmt": "nvfp4", "page": 16,
         "pages": 2048, "act": "bf16", "prompt": False},
        # a long prompt into an 8-bit cache
        {"name": "cache_prefill", "op": "cache", "T": 12345, "H": 8, "D": 128, "fmt": "fp8", "page": 32,
         "pages": 1024, "act": "bf16", "prompt": True},
        # one user, a short context: latency
        {"name": "attn_one", "op": "attn", "B": 1, "L": 777, "H": 8, "G": 4, "D": 128, "fmt": "fp8", "page": 16,
         "window": 0, "sinks": False, "ragged": False},
        # a decode batch of ragged contexts over a 4-bit cache, 64 query heads on 8, with sinks
        {"name": "attn_batch", "op": "attn", "B": 64, "L": 16384, "H": 8, "G": 8, "D": 64, "fmt": "nvfp4",
         "page": 16, "window": 0, "sinks": True, "ragged": True},
        # the same kind of model's sliding-window layer, an odd number of heads a group
        {"name": "attn_window", "op": "attn", "B": 48, "L": 8192, "H": 4, "G": 5, "D": 64, "fmt": "bf16",
         "page": 64, "window": 128, "sinks": True, "ragged": True},
        # long contexts over a 16-bit cache: memory bandwidth
        {"name": "attn_long", "op": "attn", "B": 16, "L": 65536, "H": 8, "G": 4, "D": 128, "fmt": "bf16",
         "page": 32, "window": 0, "sinks": False, "ragged": False},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("route", "norm", "cache", "attn", "attn"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 5, 8, 16))
        E = groups * rng.randint(max(2, -(-4 // groups)), 256 // groups)
        keep = rng.randint(-(-groups // 2), groups)
        k = rng.randint(1, min(8, keep * (E // groups)))
        return {"op": "route", "T": _log(rng, 1, 8192), "E": E, "k": k,
                "score": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.6, "groups": groups,
                "keep": keep, "gscore": rng.choice(("max", "top2")), "renorm": rng.random() < 0.7,
                "factor": rng.choice((1.0, 2.5)), "logits": rng.choice(("fp32", "bf16", "fp16"))}
    if op == "norm":
        H = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            H -= H % 64
        act = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        case = {"op": "norm", "T": _log(rng, 1, 8192), "H": H, "act": act, "res": rng.choice((act, "fp32")),
                "gate": rng.choice(("none", "full", "row", "col")), "post": rng.choice(("none", "rms", "layer")),
                "pre": rng.choice(("none", "rms", "layer")), "alpha": rng.choice((1.0, 0.25))}
    elif op == "cache":
        T, page = _log(rng, 1, 12345), rng.choice((16, 32, 64, 128))
        case = {"op": "cache", "T": T, "H": rng.randint(1, 16), "D": rng.choice((64, 128, 256)),
                "fmt": rng.choice(FMTS), "page": page, "pages": T // page + 2 + rng.randint(0, 200),
                "act": rng.choice(("bf16", "fp16", "fp32")), "prompt": rng.random() < 0.5}
    else:
        L = _log(rng, 1, 65536)
        case = {"op": "attn", "B": _log(rng, 1, 256), "L": L, "H": rng.randint(1, 16), "G": rng.randint(1, 16),
                "D": rng.choice((64, 128, 256)), "fmt": rng.choice(FMTS), "page": rng.choice((16, 32, 64, 128)),
                "window": rng.choice((0, 0, 0, rng.randint(1, 4096))), "sinks": rng.random() < 0.5,
                "ragged": rng.random() < 0.7}
    # no larger than the largest listed one
    top, size = max(_padded(c) for c in listed()), {"norm": "T", "cache": "T", "attn": "B"}[op]
    while _padded(case) > top and case[size] > 1:
        case[size] = max(1, case[size] * 3 // 4)
    if op == "attn":
        while _padded(case) > top:
            case["L"] = case["L"] * 3 // 4
    return case


def _padded(c):
    """Bytes of a case with every sequence at its full length, 16-bit keys and values."""
    if c["op"] == "attn":
        return 4 * c["B"] * c["L"] * c["H"] * c["D"]
    if c["op"] == "cache":
        return 16 * c["T"] * c["H"] * c["D"]
    return 20 * c["T"] * c["H"] if c["op"] == "norm" else 4 * c["T"] * c["E"]


# ----------------------------------------------------------------------------------------- inputs
def _record(fmt, D):
    """(bytes of one head's row of codes, bytes of a record) of the cache."""
    if fmt in ("bf16", "fp16"):
        return 2 * D, 64 * D
    if fmt == "fp8":
        return D, 32 * D + 32
    return D // 2, 18 * D + 32


def _lens(case, seed):
    """Tokens of every sequence (host list): ragged ones spread over their logarithm, one full, one single."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    g = torch.Generator().manual_seed(seed)
    lens = [max(1, min(L, int(round(L ** u)))) for u in torch.rand(B, generator=g, dtype=torch.float64).tolist()]
    lens[0] = L
    if B > 2:
        lens[1] = 1
    return lens


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    s = {"case": dict(case)}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        s["logits"] = randn(T, E, dtype=DTYPES[case["logits"]], std=1.5)
        s["bias"] = randn(E, std=0.1) if case["bias"] else None
    elif case["op"] == "norm":
        T, H, act = case["T"], case["H"], DTYPES[case["act"]]
        s["z"] = randn(T, H, dtype=act, std=2.0)
        s["res"] = randn(T, H, dtype=DTYPES[case["res"]], std=3.0)
        shape = {"none": None, "full": (T, H), "row": (T, 1), "col": (1, H)}[case["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(randn(*shape)).to(act)
        for n in ("post", "pre"):
            s[n + "_w"] = None if case[n] == "none" else 1.0 + randn(H, std=0.1)
            s[n + "_b"] = randn(H, std=0.1) if case[n] == "layer" else None
    elif case["op"] == "cache":
        T, H, D, page = case["T"], case["H"], case["D"], case["page"]
        rec = _record(case["fmt"], D)[1]
        s["data"] = torch.zeros(case["pages"], H, page // 16, rec, dtype=torch.uint8, device=dev)
        # keys and values as parts of one projection's output; some channels of the keys are large
        qkv = randn(T, 4 * H, D, std=1.0)
        qkv[:, 2 * H:3 * H, ::16] *= 8.0
        qkv = qkv.to(DTYPES[case["act"]])
        s["k"], s["v"] = qkv[:, 2 * H:3 * H], qkv[:, 3 * H:]
        if case["prompt"]:  # whole pages, in a shuffled order of pages
            order = torch.randperm(case["pages"], generator=g, device=dev)
            t = torch.arange(T, device=dev)
            slots = order[t // page] * page + t % page
        else:  # one token of each of many sequences
            slots = torch.randperm(case["pages"] * page, generator=g, device=dev)[:T]
        s["slots"] = slots.to(torch.int32)
        s["k_out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device=dev)
    else:
        B, L, H, G, D, page, fmt = (case[n] for n in ("B", "L", "H", "G", "D", "page", "fmt"))
        lens = _lens(case, seed)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        row, rec = _record(fmt, D)
        n_rec = pages * H * (page // 16)
        data = torch.empty(n_rec, rec, dtype=torch.uint8, device=dev)
        if fmt in ("bf16", "fp16"):
            data.view(DTYPES[fmt])[:] = torch.randn(n_rec, rec // 2, generator=g, device=dev, dtype=DTYPES[fmt])
        else:
            codes = data[:, :32 * row]
            if fmt == "fp8":  # normal values, the largest of a row between 224 and 448
                codes.view(torch.float8_e4m3fn)[:] = torch.randn(n_rec, 32 * row, generator=g, device=dev,
                                                                 dtype=torch.bfloat16).mul_(120).clamp_(-448, 448).to(
                                                                     torch.float8_e4m3fn)
                mid = 120
            else:  # E2M1 codes as normal values give them, block scales in the upper range of E4M3
                share = torch.tensor([0.10, 0.17, 0.14, 0.12, 0.18, 0.12, 0.11, 0.06], device=dev).cumsum(0)
                table = torch.bucketize((torch.arange(256, device=dev) + 0.5) / 256, share).clamp_(max=7)
                at = torch.randint(0, 256, (n_rec, 32 * row, 2), generator=g, device=dev, dtype=torch.uint8)
                mag = table.to(torch.uint8)[at.int()]
                sign = (at & 1) << 3
                codes[:] = (mag[..., 0] | sign[..., 0]) | ((mag[..., 1] | sign[..., 1]) << 4)
                del at, mag, sign
                sc = data[:, 32 * row:32 * row + 2 * D]
                sc.view(torch.float8_e4m3fn)[:] = (torch.rand(n_rec, 2 * D, generator=g, device=dev) * 240 + 120).to(
                    torch.float8_e4m3fn)
                mid = 118
            # most rows of one size, some twice as large or half
            data[:, rec - 32:] = (mid + torch.randn(n_rec, 32, generator=g, device=dev) * 0.5).round().to(torch.uint8)
        s["data"] = data.view(pages, H, page // 16, rec)
        order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32).cpu()
        table = torch.full((B, max(need)), -1, dtype=torch.int32)
        start = 0
        for b, n in enumerate(need):
            table[b, :n] = order[start:start + n]
            start += n
        s["table"] = table.to(dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        qd = torch.float16 if fmt == "fp16" else torch.bfloat16
        s["q"] = randn(B, H * G, D, dtype=qd, std=2.0)
        s["sinks"] = randn(H * G) if case["sinks"] else None
        s["scale"] = D ** -0.5
    return s


# -------------------------------------------------------------------------------------- plain form
def _route(s):
    c = s["case"]
    T, E, k, n = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].double()
    p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    pb = p if s["bias"] is None else p + s["bias"].double()
    rank = l if s["bias"] is None else pb
    if c["gscore"] == "top2":
        group = pb.view(T, n, E // n).topk(2, dim=2).values.sum(2)
    else:
        group = rank.view(T, n, E // n).amax(2)
    best = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
    kept = torch.zeros_like(group, dtype=torch.bool).scatter_(1, best, True)
    kept = kept[:, :, None].expand(T, n, E // n).reshape(T, E)
    rank = torch.where(kept, rank, torch.full_like(rank, -float("inf")))
    ids = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (w * c["factor"]).float()}


def _normed(x, kind, w, b):
    if kind == "none":
        return x
    if kind == "rms":
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w
    x = x - x.mean(1, keepdim=True)
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w + b


def _norm(s):
    c = s["case"]
    u = _normed(s["z"].float(), c["post"], s["post_w"], s["post_b"]) * c["alpha"]
    if s["gate"] is not None:
        u = u * s["gate"].float()
    h = s["res"].float() + u
    out = {"h": h.to(s["res"].dtype)}
    if c["pre"] != "none":
        out["y"] = _normed(h, c["pre"], s["pre_w"], s["pre_b"]).to(s["z"].dtype)
    return out


def _places(slots, page, H, D, fmt, dev):
    """Byte positions in the cache of every slot's K codes [n, H, row], and of its records [n, H].

    The 16-byte pieces of every 128 bytes of codes are stored in another order, so that the lanes of a
    warp find them in different banks of shared memory: piece p of the record's line is at p ^ f."""
    row, rec = _record(fmt, D)
    slots = slots.long()
    i = slots % 16
    record = (slots // page)[:, None] * H + torch.arange(H, device=dev)
    record = (record * (page // 16) + (slots % page // 16)[:, None]) * rec
    f = i & 7 if row >= 128 else i & 6 if row == 64 else (i >> 1) & 2
    at = i[:, None] * row + torch.arange(row, device=dev)
    at = at ^ (f[:, None] * 16)
    return record, record[:, :, None] + at[:, None, :]


def _scale_places(record, slots, fmt, D):
    """Byte positions of the K block scales [n, H, D / 16] of the slots, and of their K row exponents."""
    row, rec = _record(fmt, D)
    i = slots.long()[:, None] % 16
    blocks = record[:, :, None] + 32 * row + torch.arange(D // 16, device=record.device) * 16 + i[:, :, None]
    return blocks, record + rec - 32 + i


def _rows(data, slots, page, fmt, D):
    """Keys and values of the slots, [n, H, D] in 32 bits."""
    H = data.shape[1]
    record, kat = _places(slots, page, H, D, fmt, data.device)
    row = _record(fmt, D)[0]
    flat = data.view(-1)
    k, v = flat[kat], flat[kat + 16 * row]
    if fmt in DTYPES:
        return k.view(DTYPES[fmt]).float(), v.view(DTYPES[fmt]).float()
    blocks, rows = _scale_places(record, slots, fmt, D)
    one = torch.ones((), device=data.device)
    ks = _times_pow2(one, flat[rows].int() - 127)[:, :, None]
    vs = _times_pow2(one, flat[rows + 16].int() - 127)[:, :, None]
    if fmt == "fp8":
        return k.view(torch.float8_e4m3fn).float() * ks, v.view(torch.float8_e4m3fn).float() * vs
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=data.device)
    kc = lut[torch.stack((k & 15, k >> 4), 3).int()].flatten(2)
    vc = lut[torch.stack((v & 15, v >> 4), 3).int()].flatten(2)
    kb = (flat[blocks].view(torch.float8_e4m3fn).float() * ks).repeat_interleave(16, 2)
    vb = (flat[blocks + D].view(torch.float8_e4m3fn).float() * vs).repeat_interleave(16, 2)
    return kc * kb, vc * vb


def _times_pow2(x, e):
    """x 2^e in 32 bits, exact where it is no subnormal: e from -127 to 127, in two steps from the bits of
    powers of two (the device's exp2 and pow of whole numbers are not exact)."""
    half = e >> 1
    return x * ((half + 127) << 23).view(torch.float32) * ((e - half + 127) << 23).view(torch.float32)


def _e2m1(x):
    """E2M1 codes of x, to the nearest, ties to the even code, the sign in bit 3."""
    a = x.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() +
            (a >= 3.5).int() + (a > 5.0).int())
    return code + 8 * torch.signbit(x).int()


def _quantise(x, fmt):
    """Codes [n, H, row], block scales and row exponents of x [n, H, D] (32 bits)."""
    amax = x.abs().amax(2, keepdim=True)
    top = 448.0 if fmt == "fp8" else 2688.0
    m, e = torch.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1
    mt, et = torch.frexp(torch.tensor(top, device=x.device))
    e = torch.where(amax > 0, e - et + (m > mt).int(), torch.full_like(e, -127)).clamp(-127, 127)
    x = _times_pow2(x, -e)
    rows = (e + 127).to(torch.uint8)[:, :, 0]
    if fmt == "fp8":
        return x.to(torch.float8_e4m3fn).view(torch.uint8), None, rows
    b = x.view(x.shape[0], x.shape[1], -1, 16)
    bs = (b.abs().amax(3) / 6.0).to(torch.float8_e4m3fn)
    d = bs.float()[..., None]
    c = _e2m1(torch.where(d > 0, b / d, torch.zeros_like(b))).reshape(x.shape)
    return (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8), bs.view(torch.uint8), rows


def _store(data, slots, page, fmt, D, k, v):
    H = data.shape[1]
    record, kat = _places(slots, page, H, D, fmt, data.device)
    row = _record(fmt, D)[0]
    flat = data.view(-1)
    if fmt in DTYPES:
        flat[kat] = k.to(DTYPES[fmt]).contiguous().view(torch.uint8)
        flat[kat + 16 * row] = v.to(DTYPES[fmt]).contiguous().view(torch.uint8)
        return
    blocks, rows = _scale_places(record, slots, fmt, D)
    kc, kb, kr = _quantise(k.float(), fmt)
    vc, vb, vr = _quantise(v.float(), fmt)
    flat[kat], flat[kat + 16 * row] = kc, vc
    if kb is not None:
        flat[blocks], flat[blocks + D] = kb, vb
    flat[rows], flat[rows + 16] = kr, vr


def _row_exponents(data, fmt):
    """The K and V row exponents of the whole cache, as they lie in its records."""
    return None if fmt in DTYPES else data[..., -32:]


def _cache(s):
    c = s["case"]
    _store(s["data"], s["slots"], c["page"], c["fmt"], c["D"], s["k"], s["v"])
    k, v = _rows(s["data"], s["slots"], c["page"], c["fmt"], c["D"])
    return {"k": k.bfloat16(), "v": v.bfloat16(), "rows": _row_exponents(s["data"], c["fmt"])}


def _attn(s):
    c = s["case"]
    B, H, G, D, page = c["B"], c["H"], c["G"], c["D"], c["page"]
    dev, lens = s["lens"].device, s["lens"].long()
    n = min(c["window"], c["L"]) if c["window"] else c["L"]
    first = (lens - n).clamp(min=0)
    pos = first[:, None] + torch.arange(n, device=dev)  # [B, n]
    seen = pos < lens[:, None]
    pos = torch.where(seen, pos, torch.zeros_like(pos))
    slots = s["table"].long().gather(1, pos // page) * page + pos % page
    k, v = _rows(s["data"], slots.view(-1), page, c["fmt"], D)
    q = s["q"].float().view(B, H, G, D)
    t = torch.einsum("bhgd,bnhd->bhgn", q, k.view(B, n, H, D)) * s["scale"]
    t = torch.where(seen[:, None, None, :], t, torch.full_like(t, -float("inf")))
    m = t.amax(3, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, H, G, 1)
        m = torch.maximum(m, sink)
    p = torch.exp(t - m)
    l = p.sum(3, keepdim=True)
    if s["sinks"] is not None:
        l = l + torch.exp(sink - m)
    out = torch.einsum("bhgn,bnhd->bhgd", p / l, v.view(B, n, H, D))
    return {"out": out.reshape(B, H * G, D).to(s["q"].dtype), "lse": (m + torch.log(l)).view(B, H * G)}


# -------------------------------------------------------------------------------- the library's calls
def _handles(s):
    """What a program keeps beside its inputs: workspace, output buffers, the views of its weights."""
    import bit_block_scaled_gb300 as moe
    c, dev = s["case"], "cuda"
    h = {"moe": moe}
    if c["op"] == "route":
        h["cfg"] = moe.router(c["score"], c["groups"], c["keep"], c["gscore"], c["renorm"], c["factor"])
        h["ids"] = torch.empty(c["T"], c["k"], dtype=torch.int32, device=dev)
        h["w"] = torch.empty(c["T"], c["k"], dtype=torch.float32, device=dev)
        h["ws"] = torch.zeros(moe.STATUS_BYTES, dtype=torch.uint8, device=dev)
    elif c["op"] == "norm":
        for n in ("post", "pre"):
            h[n] = None if c[n] == "none" else moe.norm(c[n], s[n + "_w"], s[n + "_b"], EPS)
        h["h"] = torch.empty_like(s["res"])
        h["y"] = None if c["pre"] == "none" else torch.empty_like(s["z"])
    else:
        h["cache"] = moe.kv_cache(s["data"], c["fmt"], c["D"])
        if c["op"] == "cache":
            h["ws"] = torch.zeros(moe.STATUS_BYTES, dtype=torch.uint8, device=dev)
        else:
            nbytes = moe.moe_attn_workspace_size(c["H"] * c["G"], c["H"], c["D"])
            h["ws"] = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
            h["out"] = torch.empty_like(s["q"])
            h["lse"] = torch.empty(c["B"], c["H"] * c["G"], dtype=torch.float32, device=dev)
    return h


def _own(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    c, h = s["case"], s["handles"]
    moe = h["moe"]
    if c["op"] == "route":
        moe.moe_route_grouped(s["logits"], s["bias"], c["k"], h["cfg"], h["ids"], h["w"], h["ws"])
        return {"ids": h["ids"], "weights": h["w"]}
    if c["op"] == "norm":
        moe.moe_residual_norm(s["z"], s["res"], s["gate"], h["post"], c["alpha"], h["h"], h["pre"], h["y"])
        return {"h": h["h"]} if h["y"] is None else {"h": h["h"], "y": h["y"]}
    if c["op"] == "cache":
        moe.moe_kv_write(s["k"], s["v"], s["slots"], h["cache"], h["ws"])
        moe.moe_kv_read(h["cache"], s["slots"], s["k_out"], s["v_out"], h["ws"])
        return {"k": s["k_out"], "v": s["v_out"], "rows": _row_exponents(s["data"], c["fmt"])}
    moe.moe_attn_decode(s["q"], h["cache"], s["table"], s["lens"], h["out"], h["ws"], s["scale"], c["window"],
                        s["sinks"], h["lse"])
    return {"out": h["out"], "lse": h["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"route": _route, "norm": _norm, "cache": _cache, "attn": _attn}[state["case"]["op"]](state)


# -------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        b = T * E * (4 if case["logits"] == "fp32" else 2) + (4 * E if case["bias"] else 0) + 8 * T * k
        return {"bytes": b, "flops": 4 * T * E}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        a, r = (4 if case[n] == "fp32" else 2 for n in ("act", "res"))
        gate = {"none": 0, "full": T * H, "row": T, "col": H}[case["gate"]]
        vec = sum({"none": 0, "rms": 1, "layer": 2}[case[n]] for n in ("post", "pre"))
        y = 0 if case["pre"] == "none" else a
        return {"bytes": T * H * (a + 2 * r + y) + gate * a + 4 * H * vec, "flops": 10 * T * H}
    if case["op"] == "cache":
        T, H, D = case["T"], case["H"], case["D"]
        held = _record(case["fmt"], D)[1] / 16  # bytes of one token's key and value
        b = T * H * (2 * D * (4 if case["act"] == "fp32" else 2) + 2 * held + 4 * D) + 8 * T
        return {"bytes": b, "flops": 8 * T * H * D}
    H, G, D = case["H"], case["G"], case["D"]
    # the lengths vary with the seed: those of seed 0 stand for all
    n = sum(min(x, case["window"] or x) for x in _lens(case, 0))
    b = n * H * _record(case["fmt"], D)[1] / 16 + case["B"] * H * G * (4 * D + 4) + 4 * n / case["page"]
    return {"bytes": b, "flops": 4 * n * H * G * D}


# ------------------------------------------------------------------------------ in 64 bits, apart
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "route":
        T, E, n = case["T"], case["E"], case["groups"]
        l = s["logits"].to(f64).cpu()
        if case["score"] == "softmax":
            e = torch.exp(l - l.max(1, keepdim=True).values)
            p = e / e.sum(1, keepdim=True)
        else:
            p = 1 / (1 + torch.exp(-l))
        pb = p if s["bias"] is None else p + s["bias"].to(f64).cpu()
        rank = (l if s["bias"] is None else pb).numpy()
        gs, ids = E // n, []
        sorted_rows = np.sort((pb.numpy() if case["gscore"] == "top2" else rank).reshape(T, n, gs), axis=2)
        for t in range(T):
            row = sorted_rows[t]
            score = row[:, -1] + row[:, -2] if case["gscore"] == "top2" else row[:, -1]
            groups = sorted(range(n), key=lambda a: (-score[a], a))[:case["keep"]]
            r = rank[t]
            ids.append(sorted((a * gs + b for a in groups for b in range(gs)), key=lambda e: (-r[e], e))[:case["k"]])
        ids = torch.tensor(ids)
        w = p.gather(1, ids)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return {"ids": ids.to(torch.int32), "weights": w * case["factor"]}
    if case["op"] == "norm":
        def norm(x, kind, w, b):
            if kind == "none":
                return x
            mean = x.mean(1, keepdim=True) if kind == "layer" else 0.0
            y = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + EPS) * w.to(f64)
            return y if b is None else y + b.to(f64)
        gate = 1.0 if s["gate"] is None else s["gate"].to(f64)
        h = s["res"].to(f64) + case["alpha"] * gate * norm(s["z"].to(f64), case["post"], s["post_w"], s["post_b"])
        return {"h": h} if case["pre"] == "none" else {"h": h, "y": norm(h, case["pre"], s["pre_w"], s["pre_b"])}
    if case["op"] == "cache":
        return {n: _held(s[n].to(f64), case["fmt"]) for n in ("k", "v")} | {"rows": None}
    return _attn64(case, s)


def _nearest(x, grid):
    """x to the nearest value of +-grid (64 bits), ties to the even place, past the end to the last."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    a = x.abs().contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.where(a >= grid[-1], grid[-1], grid[pick]) * torch.sign(x)


def _held(x, fmt):
    """What the cache holds of x [n, H, D] (64 bits)."""
    if fmt in DTYPES:
        return x.to(DTYPES[fmt]).double()
    e4m3 = [(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)]
    amax = x.abs().amax(2, keepdim=True)
    pow2 = torch.tensor([2.0 ** e for e in range(-127, 128)], dtype=torch.float64, device=x.device)
    at = torch.searchsorted(pow2 * (448 if fmt == "fp8" else 2688), amax.contiguous())  # the first that is enough
    r = pow2[at.clamp(max=254)]
    if fmt == "fp8":
        return _nearest(x / r, e4m3) * r
    b = x.view(x.shape[0], x.shape[1], -1, 16)
    sc = _nearest(b.abs().amax(3, keepdim=True) / 6 / r[..., None], e4m3) * r[..., None]
    return (_nearest(torch.where(sc > 0, b / sc.clamp(min=1e-300), torch.zeros_like(b)), list(E2M1)) * sc).view(x.shape)


def _attn64(case, s):
    H, G, D, page, fmt = (case[n] for n in ("H", "G", "D", "page", "fmt"))
    row, rec = _record(fmt, D)
    lens, table, outs, lses = s["lens"].tolist(), s["table"].long(), [], []
    dev = s["q"].device
    pow2 = torch.tensor([2.0 ** e for e in range(-127, 129)], dtype=torch.float64, device=dev)
    # where piece p of row i lies: [16, row] byte positions within a section of codes
    at = torch.tensor([[(i * row + b) ^ 16 * (i & 7 if row > 64 else i & 6 if row > 32 else i // 2 & 2)
                        for b in range(row)] for i in range(16)], device=dev)
    for b, n in enumerate(lens):
        first = max(0, n - case["window"]) if case["window"] else 0
        p0 = first // page
        r = s["data"][table[b, p0:-(-n // page)]].transpose(0, 1).reshape(H, -1, rec)  # every head's records
        kv = []
        for part in (0, 1):
            codes = r[:, :, part * 16 * row:(part + 1) * 16 * row][:, :, at]  # [H, records, 16, row]
            if fmt in DTYPES:
                x = codes.view(DTYPES[fmt]).double()
            else:
                rows = pow2[r[:, :, rec - 32 + 16 * part:rec - 16 + 16 * part].int()]
                if fmt == "fp8":
                    x = codes.view(torch.float8_e4m3fn).double() * rows[..., None]
                else:
                    c = torch.stack((codes % 16, codes // 16), 4).flatten(3).double()
                    m = c % 8
                    mag = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
                    sc = r[:, :, 32 * row + part * D:32 * row + part * D + D].contiguous().view(torch.float8_e4m3fn)
                    sc = sc.double().view(H, -1, D // 16, 16).transpose(2, 3) * rows[..., None]
                    x = torch.where(c < 8, mag, -mag) * sc.repeat_interleave(16, 3)
            kv.append(x.reshape(H, -1, D)[:, first - p0 * page:n - p0 * page])
        q = s["q"][b].double().view(H, G, D)
        t = q @ kv[0].transpose(1, 2) * s["scale"]
        m = t.amax(2, keepdim=True)
        e = torch.exp(t - m)
        l = e.sum(2, keepdim=True)
        if s["sinks"] is not None:
            l = l + torch.exp(s["sinks"].double().view(H, G, 1) - m)
        outs.append((e @ kv[1] / l).view(H * G, D))
        lses.append((m + torch.log(l)).view(H * G))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
