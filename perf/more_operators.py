"""The operators between a decoder block's hidden states and its attention, measured: the plan of a batch (pages,
block tables, slots), rotary positions with and without the cache write, 4-bit quantisation of activations, and the
product of two 4-bit operands.

Every case is a dict of plain values; ``prepare`` makes its inputs on the GPU, ``run`` computes the operator either
in its plain form (elementary torch operations, ``own`` false) or through the library's entry points (``own``
true), ``exact`` computes it from the definition in 64 bits.

Definitions:

* plan: sequence b holds L tokens and gets n more (n < 0: it ends). Ended sequences' pages, ceil(L / page) of them,
  are put on the stack of free pages in the order of sequences and pages. Sequence b is served if L + n tokens fit
  its row of the block table, the pages that it and all before it need (ceil((L + n) / page) - ceil(L / page)) fit the
  stack or it needs none, and its last token is among the T rows. The pages come off the top of the stack in the order of
  sequences and pages. Token i of its new ones is at position L + i, in slot table[position / page] * page + position %
  page; rows of a sequence that is not served have slot -1 and position 0, rows past the last token slot -1, position
  0 and sequence -1.
* rope: pairs (a, b) of a head's first R columns, (i, i + R / 2) or (2 i, 2 i + 1), become (a c - b s, b c + a s) with
  c, s = m cos(p f_i), m sin(p f_i) at position p. f_i = base^(-2 i / R), scaled for long contexts: "linear" f / factor;
  "ntk" base * factor^(R / (R - 2)); "yarn" f / factor (1 - g) + f g, g = 1 - clamp((i - low) / (high - low), 0, 1), low and high =
  R ln(L / (2 pi beta)) / (2 ln base) for beta 32 and 1, m = 0.1 ln(factor) + 1; "llama3" by wavelength 2 pi / f: f below L / 4,
  f / factor above L, between them (1 - h) f / factor + h f, h = (L / wavelength - 1) / 3. With the cache: the rotated keys,
  unrounded, and the values are quantised into their slots.
* cache: blocks of 16 tokens of one head are one record: the K codes, the V codes, the K and V block scales (NVFP4), the K
  and V row exponents (FP8 and NVFP4). FP8: row scale r the least power of two with amax / r <= 448, codes E4M3 of x / r.
  NVFP4 as below, rows of one head.
* quantisation: NVFP4: row scale r the least power of two with amax / r <= 6 * 448, an E4M3 scale s of amax16 / r / 6 for
  every 16 values, codes E2M1 of x / r / s. MXFP4: for every 32 values the least power of two s with amax32 / s <= 6,
  codes E2M1 of x / s.
* product: out[t][n] = sum_k x[t][k] w[n][k] + bias[n], x quantised by the call, w quantised before.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
YARN_LEN = 4096  # context that the scaled frequencies come from


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one step of a decode batch: every sequence one token longer, now and then a new page
        {"name": "plan_decode", "op": "plan", "B": 64, "T": 64, "L": 8000, "page": 16, "width": 512, "ends": 0.0,
         "prompts": 0.0, "enough": True},
        # a step that mixes decode, new prompts and ended sequences, in a fixed number of token rows
        {"name": "plan_mixed", "op": "plan", "B": 500, "T": 65536, "L": 4000, "page": 32, "width": 256, "ends": 0.1,
         "prompts": 0.2, "enough": True},
        # one token of a gpt-oss-like layer, 64 query heads on 8, YaRN: latency
        {"name": "rope_one", "op": "rope", "T": 1, "H": 8, "G": 8, "D": 64, "rot": 64, "layout": "half",
         "scaling": "yarn", "base": 150000.0, "factor": 32.0, "far": 131072, "act": "bf16"},
        # a prefill chunk far into a long context, half of each head rotated, interleaved
        {"name": "rope_prefill", "op": "rope", "T": 8192, "H": 8, "G": 4, "D": 128, "rot": 64,
         "layout": "interleaved", "scaling": "llama3", "base": 500000.0, "factor": 8.0, "far": 1000000, "act": "bf16"},
        # a decode batch's rotation and write into a 4-bit cache
        {"name": "write_decode", "op": "write", "T": 64, "H": 8, "G": 8, "D": 64, "rot": 64, "layout": "half",
         "scaling": "yarn", "base": 150000.0, "factor": 32.0, "far": 131072, "act": "bf16", "fmt": "nvfp4", "page": 16,
         "pages": 2048},
        # a long prompt into an 8-bit cache
        {"name": "write_prompt", "op": "write", "T": 12345, "H": 8, "G": 4, "D": 128, "rot": 128, "layout": "half",
         "scaling": "none", "base": 10000.0, "factor": 1.0, "far": 12345, "act": "bf16", "fmt": "fp8", "page": 32,
         "pages": 1024},
        # the activations of a decode batch, width 2880
        {"name": "quant_decode", "op": "quant", "T": 64, "K": 2880, "fmt": "nvfp4", "act": "bf16"},
        # a prefill chunk of the concatenated heads, width 4096
        {"name": "quant_prefill", "op": "quant", "T": 8192, "K": 4096, "fmt": "mxfp4", "act": "bf16"},
        # the query, key and value projection of one token (64 + 2 * 8 heads of 64 from width 2880): latency
        {"name": "linear_one", "op": "linear", "T": 1, "N": 5120, "K": 2880, "fmt": "nvfp4", "act": "bf16",
         "bias": True},
        # the output projection of a ragged batch
        {"name": "linear_batch", "op": "linear", "T": 333, "N": 2880, "K": 4096, "fmt": "mxfp4", "act": "bf16",
         "bias": True},
        # the same projection of a prefill chunk
        {"name": "linear_prefill", "op": "linear", "T": 8192, "N": 5120, "K": 2880, "fmt": "nvfp4", "act": "bf16",
         "bias": True},
        # a wide model's projection: the tensor cores
        {"name": "linear_wide", "op": "linear", "T": 16384, "N": 8192, "K": 8192, "fmt": "nvfp4", "act": "bf16",
         "bias": False},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("plan", "rope", "write", "quant", "linear", "linear"))
    if op == "plan":
        page, B = rng.choice((16, 32, 64, 128)), _log(rng, 1, 1024)
        prompts = rng.choice((0.0, 0.1, 0.5, 1.0))
        width = rng.randint(1, 512)
        return {"op": op, "B": B, "T": B if prompts == 0.0 else _log(rng, max(B, 16), 65536),
                "L": max(1, _log(rng, 1, width * page) - 1), "page": page, "width": width,
                "ends": rng.choice((0.0, 0.1, 0.9)), "prompts": prompts, "enough": rng.random() < 0.7}
    if op in ("rope", "write"):
        D = rng.choice((64, 128, 256))
        scaling = rng.choice(("none", "linear", "ntk", "yarn", "llama3"))
        case = {"op": op, "T": _log(rng, 1, 12345), "H": rng.randint(1, 16), "G": rng.randint(1, 16), "D": D,
                "rot": rng.choice((D, D, D // 2, rng.randrange(4, D, 2))), "layout": rng.choice(("half", "interleaved")),
                "scaling": scaling, "base": rng.choice((10000.0, 150000.0, 500000.0)),
                "factor": 1.0 if scaling == "none" else rng.choice((2.0, 8.0, 32.0)), "far": _log(rng, 12345, 4000000),
                "act": rng.choice(("bf16", "bf16", "fp16", "fp32"))}
        while case["T"] > 1 and case["T"] * case["H"] * (case["G"] + 2) * D > 80_000_000:
            case["T"] = case["T"] * 3 // 4
        if op == "write":
            # 4 bits at the sizes of new tokens of a batch: among many millions of rotated keys a few lie so close to
            # a border between two codes that 32 bits may fall on either side
            case["fmt"] = rng.choice(("bf16", "fp16", "fp8")) if case["T"] > 256 else rng.choice(("bf16", "fp8", "nvfp4"))
            case["page"] = rng.choice((16, 32, 64, 128))
            case["pages"] = case["T"] // case["page"] + 2 + rng.randint(0, 200)
        return case
    K = 32 * _log(rng, 2, 256)
    case = {"op": op, "T": _log(rng, 1, 16384), "K": K, "fmt": rng.choice(("nvfp4", "mxfp4")),
            "act": rng.choice(("bf16", "bf16", "fp16"))}
    if op == "linear":
        case["N"] = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            case["N"] = max(64, case["N"] - case["N"] % 64)
        case["bias"] = rng.random() < 0.5
    return case


# ----------------------------------------------------------------------------------------- inputs
def _record(fmt, D):
    """(bytes of one head's row of codes, bytes of a record) of the cache."""
    if fmt in ("bf16", "fp16"):
        return 2 * D, 64 * D
    if fmt == "fp8":
        return D, 32 * D + 32
    return D // 2, 18 * D + 32


def _frequencies(case):
    """(frequencies in radians a position [rot / 2] in 64 bits, amplitude)."""
    R, base, factor = case["rot"], case["base"], case["factor"]
    i = np.arange(R // 2, dtype=np.float64)
    if case["scaling"] == "ntk":
        base = base * factor ** (R / (R - 2))
    f = base ** (-2.0 * i / R)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "yarn":
        low, high = (R * math.log(YARN_LEN / (2 * math.pi * beta)) / (2 * math.log(base)) for beta in (32.0, 1.0))
        low, high = max(low, 0.0), min(high, R - 1.0)
        keep = 1.0 - np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    if case["scaling"] == "llama3":
        smooth = np.clip((YARN_LEN * f / (2 * math.pi) - 1.0) / 3.0, 0.0, 1.0)
        return f / factor * (1 - smooth) + f * smooth, 1.0
    return f, 1.0


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    s = {"case": dict(case)}
    if case["op"] == "plan":
        B, T, page, width = case["B"], case["T"], case["page"], case["width"]
        r = torch.rand(4, B, generator=g, device=dev, dtype=torch.float64)
        lens = (case["L"] ** r[0]).round().long().clamp(1, max(1, width * page - 1))
        new = torch.ones_like(lens)
        prompt = r[1] < case["prompts"]
        if case["prompts"]:  # prompts of many lengths, empty sequences until now, about T tokens in all
            lens = torch.where(prompt, torch.zeros_like(lens), lens)
            want = (r[2] * 1.6 * T / max(1.0, case["prompts"] * B)).long().clamp(1, width * page)
            new = torch.where(prompt, want, new)
        new = torch.where(~prompt & (r[3] < case["ends"]), torch.full_like(new, -1), new)
        held = (lens + page - 1) // page
        need = int(((lens + new.clamp(min=0) + page - 1) // page - held).sum())
        used = int(held.sum())
        # pages of the cache; what is neither in the table nor free belongs to others
        pages = B * (case["L"] // page + 4) + 2 * T // page + 200
        count = need + 100 if case["enough"] else need * 3 // 4 + 1
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        first = held.cumsum(0) - held
        col = torch.arange(width, device=dev)
        in_use = col < held[:, None]
        s["table"] = torch.where(in_use, order[(first[:, None] + col).clamp(max=pages - 1)], -1).to(torch.int32)
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        s["free"][:count] = order[used:used + count]
        s["count"] = torch.tensor([count], dtype=torch.int32, device=dev)
        s["lens"], s["new"] = lens.to(torch.int32), new.to(torch.int32)
    elif case["op"] in ("rope", "write"):
        T, H, G, D = (case[n] for n in ("T", "H", "G", "D"))
        # queries, keys and values are parts of one projection's output; some channels of the keys are large
        qkv = randn(T, H * G + 2 * H, D)
        qkv[:, H * G:H * G + H, ::16] *= 8.0
        qkv = qkv.to(DTYPES[case["act"]])
        s["q"], s["k"], s["v"] = qkv.split((H * G, H, H), dim=1)
        far = case["far"]
        if T > far // 4 or case["op"] == "rope":  # a chunk that ends at the far position
            s["pos"] = torch.arange(far - T, far, device=dev).to(torch.int32)
        else:  # one token of each of many sequences
            s["pos"] = torch.randint(0, far, (T,), generator=g, device=dev, dtype=torch.int32)
        f, m = _frequencies(case)
        s["freq"], s["amp"] = torch.from_numpy(f).to(dev), m
        if case["op"] == "write":
            page = case["page"]
            s["data"] = torch.zeros(case["pages"], H, page // 16, _record(case["fmt"], D)[1], dtype=torch.uint8, device=dev)
            s["slots"] = torch.randperm(case["pages"], generator=g, device=dev)[torch.arange(T, device=dev) // page] * page
            s["slots"] = (s["slots"] + torch.arange(T, device=dev) % page).to(torch.int32)
    else:
        T, K = case["T"], case["K"]
        x = randn(T, K)
        x[:, torch.randperm(K, generator=g, device=dev)[:K // 64]] *= 12.0  # a few channels are large
        x *= torch.exp(randn(T, 1, std=0.7))  # and rows differ
        s["x"] = x.to(DTYPES[case["act"]])
        if case["op"] == "linear":
            N = case["N"]
            w = randn(N, K, std=K ** -0.5)
            if case["fmt"] == "nvfp4":  # as a checkpoint holds it: one scale for all rows, chosen from the largest value
                s["gscale"] = (w.abs().max() / 2688.0).reshape(1)
                b = w.view(N, K // 16, 16)
                sc = (b.abs().amax(2) / 6.0 / s["gscale"]).to(torch.float8_e4m3fn)
                d = (sc.float() * s["gscale"])[..., None]
                s["w_q"] = _pack(_e2m1(torch.where(d > 0, b / d, torch.zeros_like(b))).view(N, K))
                s["w_s"] = sc.view(torch.uint8)
            else:
                s["gscale"] = None
                s["w_q"], s["w_s"] = _mxfp4(w)
            s["bias"] = randn(N, std=0.1, dtype=s["x"].dtype) if case["bias"] else None
    return s


# -------------------------------------------------------------------------------------- plain form
def _plan(s):
    c = s["case"]
    B, T, page, width = c["B"], c["T"], c["page"], c["width"]
    dev, cap, total = s["lens"].device, c["width"] * c["page"], s["free"].numel()
    L, n, top = s["lens"].long(), s["new"].long(), s["count"].long()
    ends, grow = n < 0, n.clamp(min=0)
    held = (L + page - 1) // page
    col = torch.arange(width, device=dev)
    # ended sequences' pages onto the stack; what is not pushed goes to a place behind it
    back = torch.where(ends, held, torch.zeros_like(held))
    at = top + (back.cumsum(0) - back)[:, None] + col
    at = torch.where(col < back[:, None], at, torch.full_like(at, total))
    stack = torch.cat((s["free"], s["free"].new_zeros(1))).scatter(0, at.view(-1), s["table"].reshape(-1))[:total]
    top = top + back.sum()
    can = (n > 0) & (L + grow <= cap)
    need = torch.where(can, (L + grow + page - 1) // page - held, torch.zeros_like(held))
    last = grow.cumsum(0)
    served = can & ((need.cumsum(0) <= top) | (need == 0)) & (last <= T)
    before = need.cumsum(0) - need
    fresh = served[:, None] & (col >= held[:, None]) & (col < (held + need)[:, None])
    page_of = stack[(top - 1 - before[:, None] - (col - held[:, None])).clamp(0, total - 1)]
    table = torch.where(fresh, page_of, s["table"])
    # the rows
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(last, t, right=True)
    there = b < B
    b = b.clamp(max=B - 1)
    pos = L[b] + t - (last - grow)[b]
    ok = there & served[b]
    pos = torch.where(ok, pos, torch.zeros_like(pos))
    slots = torch.where(ok, table[b, pos // page].long() * page + pos % page, torch.full_like(pos, -1))
    out = {"slots": slots, "positions": pos, "seqs": torch.where(there, b, torch.full_like(b, -1)),
           "offsets": torch.cat((last.new_zeros(1), last)),
           "lens": torch.where(ends, torch.zeros_like(L), torch.where(served, L + grow, L)),
           "count": top - torch.where(served, need, torch.zeros_like(need)).sum(), "table": table, "free": stack}
    return {k: v.to(torch.int32) for k, v in out.items()}


def _rotated(x, pos, freq, amp, layout):
    """x [T, heads, D], rotated, in 32 bits; angles in 64."""
    R = 2 * freq.numel()
    a = pos.double()[:, None] * freq
    c, s = (torch.cos(a) * amp).float()[:, None, :], (torch.sin(a) * amp).float()[:, None, :]
    x = x.float()
    if layout == "half":
        u, v = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat((u * c - v * s, v * c + u * s), 2)
    else:
        u, v = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack((u * c - v * s, v * c + u * s), 3).flatten(2)
    return torch.cat((y, x[..., R:]), 2)


def _rope(s):
    lay = s["case"]["layout"]
    return {n: _rotated(s[n], s["pos"], s["freq"], s["amp"], lay).to(s[n].dtype) for n in ("q", "k")}


def _write(s):
    c = s["case"]
    q = _rotated(s["q"], s["pos"], s["freq"], s["amp"], c["layout"]).to(s["q"].dtype)
    k = _rotated(s["k"], s["pos"], s["freq"], s["amp"], c["layout"])
    _store(s["data"], s["slots"], c["page"], c["fmt"], c["D"], k, s["v"].float())
    k, v = _rows(s["data"], s["slots"], c["page"], c["fmt"], c["D"])
    return {"q": q, "k": k.bfloat16(), "v": v.bfloat16()}


def _places(slots, page, H, D, fmt, dev):
    """Byte positions in the cache of every slot's K codes [n, H, row], and of its records [n, H]."""
    row, rec = _record(fmt, D)
    slots = slots.long()
    i = slots % 16
    record = (slots // page)[:, None] * H + torch.arange(H, device=dev)
    record = (record * (page // 16) + (slots % page // 16)[:, None]) * rec
    f = i & 7 if row >= 128 else i & 6 if row == 64 else (i >> 1) & 2
    at = (i[:, None] * row + torch.arange(row, device=dev)) ^ (f[:, None] * 16)
    return record, record[:, :, None] + at[:, None, :]


def _scale_places(record, slots, fmt, D):
    """Byte positions of the K block scales [n, H, D / 16] of the slots, and of their K row exponents."""
    row, rec = _record(fmt, D)
    i = slots.long()[:, None] % 16
    blocks = record[:, :, None] + 32 * row + torch.arange(D // 16, device=record.device) * 16 + i[:, :, None]
    return blocks, record + rec - 32 + i


def _store(data, slots, page, fmt, D, k, v):
    record, kat = _places(slots, page, data.shape[1], D, fmt, data.device)
    row, flat = _record(fmt, D)[0], data.view(-1)
    if fmt in DTYPES:
        flat[kat] = k.to(DTYPES[fmt]).contiguous().view(torch.uint8)
        flat[kat + 16 * row] = v.to(DTYPES[fmt]).contiguous().view(torch.uint8)
        return
    blocks, rows = _scale_places(record, slots, fmt, D)
    quantise = _fp8 if fmt == "fp8" else _nvfp4
    kc, kb, kr = quantise(k)
    vc, vb, vr = quantise(v)
    flat[kat], flat[kat + 16 * row] = kc, vc
    if kb is not None:
        flat[blocks], flat[blocks + D] = kb, vb
    flat[rows], flat[rows + 16] = (kr + 127).to(torch.uint8), (vr + 127).to(torch.uint8)


def _rows(data, slots, page, fmt, D):
    """Keys and values of the slots, [n, H, D] in 32 bits."""
    record, kat = _places(slots, page, data.shape[1], D, fmt, data.device)
    row, flat = _record(fmt, D)[0], data.view(-1)
    k, v = flat[kat], flat[kat + 16 * row]
    if fmt in DTYPES:
        return k.view(DTYPES[fmt]).float(), v.view(DTYPES[fmt]).float()
    blocks, rows = _scale_places(record, slots, fmt, D)
    kr, vr = flat[rows].int() - 127, flat[rows + 16].int() - 127
    if fmt == "fp8":
        k, v = k.view(torch.float8_e4m3fn).float(), v.view(torch.float8_e4m3fn).float()
    else:
        k, v = _nvfp4_values(k, flat[blocks]), _nvfp4_values(v, flat[blocks + D])
    return _times_pow2(k, kr[..., None]), _times_pow2(v, vr[..., None])


def _times_pow2(x, e):
    """x 2^e in 32 bits, exact where it is no subnormal: e from -127 to 127, in two steps from the bits of
    powers of two (the device's exp2 and pow of whole numbers are not exact)."""
    half = e >> 1
    return x * ((half + 127) << 23).view(torch.float32) * ((e - half + 127) << 23).view(torch.float32)


def _least_pow2(amax, top):
    """The least e from -127 to 127 with amax / 2^e <= top."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1
    mt, et = math.frexp(top)
    return torch.where(amax > 0, e - et + (m > mt).int(), torch.full_like(e, -127)).clamp(-127, 127)


def _e2m1(x):
    """E2M1 codes of x, to the nearest, ties to the even code, the sign in bit 3."""
    a = x.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() +
            (a >= 3.5).int() + (a > 5.0).int())
    return code + 8 * torch.signbit(x).int()


def _pack(c):
    """Two codes a byte, the even one in the low half."""
    return (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8)


def _unpack(q):
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=q.device)
    return lut[torch.stack((q & 15, q >> 4), -1).int()].flatten(-2)


def _fp8(x):
    """Codes, None and row exponents of x [..., K] (32 bits)."""
    e = _least_pow2(x.abs().amax(-1, keepdim=True), 448.0)
    return _times_pow2(x, -e).to(torch.float8_e4m3fn).view(torch.uint8), None, e[..., 0]


def _nvfp4(x):
    """Codes [..., K / 2], block scales [..., K / 16] (bytes) and row exponents of x [..., K] (32 bits)."""
    e = _least_pow2(x.abs().amax(-1, keepdim=True), 2688.0)
    b = _times_pow2(x, -e).unflatten(-1, (-1, 16))
    sc = (b.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    d = sc.float()[..., None]
    return _pack(_e2m1(torch.where(d > 0, b / d, torch.zeros_like(b))).flatten(-2)), sc.view(torch.uint8), e[..., 0]


def _nvfp4_values(q, sc):
    return _unpack(q) * sc.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)


def _mxfp4(x):
    """Codes [T, K / 2] and block scales [T, K / 32] (exponents with 127 added) of x [T, K] (32 bits)."""
    b = x.unflatten(-1, (-1, 32))
    e = _least_pow2(b.abs().amax(-1), 6.0)
    return _pack(_e2m1(_times_pow2(b, -e[..., None])).flatten(-2)), (e + 127).to(torch.uint8)


def _mxfp4_values(q, sc):
    return _times_pow2(_unpack(q).unflatten(-1, (-1, 32)), sc.int()[..., None] - 127).flatten(-2)


def _held(x, fmt):
    """What is left of x [T, K] (32 bits) in 4 bits."""
    if fmt == "mxfp4":
        return _mxfp4_values(*_mxfp4(x))
    q, sc, e = _nvfp4(x)
    return _times_pow2(_nvfp4_values(q, sc), e[:, None])


def _quant(s):
    return {"x": _held(s["x"].float(), s["case"]["fmt"]).bfloat16()}


def _linear(s):
    c = s["case"]
    x = _held(s["x"].float(), c["fmt"])
    w = _mxfp4_values(s["w_q"], s["w_s"]) if c["fmt"] == "mxfp4" else _nvfp4_values(s["w_q"], s["w_s"]) * s["gscale"]
    out = x @ w.t()
    if s["bias"] is not None:
        out = out + s["bias"].float()
    return {"out": out.to(s["x"].dtype)}


# -------------------------------------------------------------------------------- the library's calls
def _handles(s):
    """What a program keeps beside its inputs: workspace, output buffers, the views and layouts of its weights."""
    import bit_block_scaled_gb300 as moe
    c, dev = s["case"], "cuda"
    h = {"moe": moe, "ws": torch.zeros(moe.STATUS_BYTES, dtype=torch.uint8, device=dev)}

    def ints(*shape):
        return torch.empty(shape, dtype=torch.int32, device=dev)
    if c["op"] == "plan":
        h.update(slots=ints(c["T"]), positions=ints(c["T"]), seqs=ints(c["T"]), offsets=ints(c["B"] + 1), lens=ints(c["B"]),
                 count=ints(1))
    elif c["op"] in ("rope", "write"):
        h["rope"] = moe.rope(c["rot"], c["layout"], c["base"], c["scaling"], c["factor"], YARN_LEN, truncate=False)
        h["q"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=dev)
        h["k"] = torch.empty(s["k"].shape, dtype=s["k"].dtype if c["op"] == "rope" else torch.bfloat16, device=dev)
        if c["op"] == "write":
            h["v"] = torch.empty_like(h["k"])
            h["cache"] = moe.kv_cache(s["data"], c["fmt"], c["D"])
    else:
        T, K, fmt = c["T"], c["K"], c["fmt"]
        h["x"] = moe.fp4(torch.empty(T, K // 2, dtype=torch.uint8, device=dev),
                         torch.empty(moe.moe_fp4_scale_bytes(fmt, T, K), dtype=torch.uint8, device=dev), fmt,
                         torch.empty(T, device=dev) if fmt == "nvfp4" else None)
        if c["op"] == "quant":
            h["out"] = torch.empty(T, K, dtype=torch.bfloat16, device=dev)
        else:
            h["out"] = torch.empty(T, c["N"], dtype=s["x"].dtype, device=dev)
            sc = torch.empty(moe.moe_fp4_scale_bytes(fmt, c["N"], K), dtype=torch.uint8, device=dev)
            moe.moe_fp4_pack_scales(s["w_s"], fmt, K, sc)
            h["w"] = moe.fp4(s["w_q"], sc, fmt, s["gscale"])
    return h


def _own(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    c, h = s["case"], s["handles"]
    moe, ws = h["moe"], h["ws"]
    if c["op"] == "plan":
        moe.moe_batch_plan(s["new"], s["lens"], s["table"], s["free"], s["count"], c["page"], h["slots"], h["lens"],
                           h["count"], ws, positions=h["positions"], seq_ids=h["seqs"], offsets=h["offsets"])
        return {n: h[n] for n in ("slots", "positions", "seqs", "offsets", "lens", "count")} | {"table": s["table"],
                                                                                             "free": s["free"]}
    if c["op"] == "rope":
        moe.moe_rope(h["rope"], s["pos"], s["q"], h["q"], s["k"], h["k"])
        return {"q": h["q"], "k": h["k"]}
    if c["op"] == "write":
        moe.moe_rope_kv_write(h["rope"], s["pos"], s["q"], h["q"], s["k"], s["v"], s["slots"], h["cache"], ws)
        moe.moe_kv_read(h["cache"], s["slots"], h["k"], h["v"], ws)
        return {"q": h["q"], "k": h["k"], "v": h["v"]}
    moe.moe_fp4_quantize(s["x"], h["x"])
    if c["op"] == "quant":
        moe.moe_fp4_dequantize(h["x"], h["out"])
        return {"x": h["out"]}
    moe.moe_fp4_linear(h["x"], h["w"], s["bias"], h["out"], ws)
    return {"out": h["out"]}


def run(state):
    if own:
        return _own(state)
    return {"plan": _plan, "rope": _rope, "write": _write, "quant": _quant, "linear": _linear}[state["case"]["op"]](state)


# -------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "plan":
        # lengths in and out, offsets, the rows; the pages are few beside them
        return {"bytes": 16 * case["B"] + 12 * case["T"], "flops": 0}
    if case["op"] in ("rope", "write"):
        T, H, G, D = (case[n] for n in ("T", "H", "G", "D"))
        size, q, k = 4 if case["act"] == "fp32" else 2, T * H * G * D, T * H * D
        b = 2 * q * size + 4 * T + 8 * case["rot"]
        if case["op"] == "rope":
            return {"bytes": b + 2 * k * size, "flops": 6 * (q + k) * case["rot"] // D}
        held = _record(case["fmt"], D)[1] / 16  # bytes of one token's key and value; they are read back, too
        return {"bytes": b + 2 * k * size + 4 * T + T * H * (2 * held + 4 * D), "flops": 6 * (q + k) + 8 * k}
    T, K = case["T"], case["K"]
    bits = 4 + 8 / (16 if case["fmt"] == "nvfp4" else 32)
    row = 4 if case["fmt"] == "nvfp4" else 0
    if case["op"] == "quant":
        return {"bytes": T * (2 * K + 2 * (K * bits / 8 + row) + 2 * K), "flops": 6 * T * K}
    N = case["N"]
    return {"bytes": 2 * T * K + 2 * T * (K * bits / 8 + row) + N * K * bits / 8 + 2 * T * N + 2 * N * case["bias"],
            "flops": 2 * T * N * K}


# ------------------------------------------------------------------------------ in 64 bits, apart
def _angles64(case, pos):
    """cos and sin with their amplitude, [T, 1, rot / 2] in 64 bits; frequencies one by one."""
    R, base, factor, fs, m = case["rot"], case["base"], case["factor"], [], 1.0
    for i in range(R // 2):
        f = math.exp(-2.0 * i / R * math.log(base))
        if case["scaling"] == "linear":
            f /= factor
        elif case["scaling"] == "ntk":
            f = math.exp(-2.0 * i / R * (math.log(base) + R / (R - 2) * math.log(factor)))
        elif case["scaling"] == "yarn":
            at = [R / 2 * math.log(YARN_LEN / (beta * 2 * math.pi)) / math.log(base) for beta in (32, 1)]
            lo, hi = max(0.0, at[0]), min(at[1], R - 1)
            share = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))  # of the stretched frequency
            f, m = f * (1 - share) + f / factor * share, 1 + math.log(factor) / 10
        elif case["scaling"] == "llama3":
            wave = 2 * math.pi / f
            if wave > YARN_LEN:
                f /= factor
            elif wave > YARN_LEN / 4:
                h = (YARN_LEN / wave - 1) / 3
                f = h * f + (1 - h) * f / factor
        fs.append(f)
    a = (pos.double()[:, None] * torch.tensor(fs, dtype=torch.float64, device=pos.device))[:, None]
    return m * torch.cos(a), m * torch.sin(a)


def _rotated64(case, x, pos):
    x, (c, s), R = x.double().clone(), _angles64(case, pos), case["rot"]
    i = torch.arange(R // 2, device=x.device)
    one, two = (i, i + R // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
    a, b = x[..., one], x[..., two]
    x[..., one], x[..., two] = a * c - b * s, b * c + a * s
    return x


def _nearest(x, grid):
    """x to the nearest value of +-grid (64 bits), ties to the even place, past the end to the last."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    a = x.abs().contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.where(a >= grid[-1], grid[-1], grid[pick]) * torch.sign(x)


def _held64(x, fmt):
    """What a format holds of the rows of x (64 bits)."""
    if fmt in DTYPES:
        return x.to(DTYPES[fmt]).double()
    e4m3 = [(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)]
    pow2 = torch.tensor([2.0 ** e for e in range(-127, 128)], dtype=torch.float64, device=x.device)

    def least(a, top):  # the first power of two that is enough
        return pow2[torch.searchsorted(pow2 * top, a.contiguous()).clamp(max=254)]
    if fmt == "mxfp4":
        b = x.unflatten(-1, (-1, 32))
        r = least(b.abs().amax(-1, keepdim=True), 6.0)
        return (_nearest(b / r, E2M1) * r).flatten(-2)
    r = least(x.abs().amax(-1, keepdim=True), 448.0 if fmt == "fp8" else 2688.0)
    if fmt == "fp8":
        return _nearest(x / r, e4m3) * r
    b = x.unflatten(-1, (-1, 16))
    sc = _nearest(b.abs().amax(-1, keepdim=True) / 6 / r[..., None], e4m3) * r[..., None]
    return (_nearest(torch.where(sc > 0, b / sc.clamp(min=1e-300), torch.zeros_like(b)), E2M1) * sc).flatten(-2)


def _weights64(s):
    q, c = s["w_q"], s["case"]
    code = torch.stack((q % 16, q // 16), 2).flatten(1).double()
    m = code % 8
    m = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    w = torch.where(code < 8, m, -m)
    if c["fmt"] == "mxfp4":
        return w * torch.pow(2.0, s["w_s"].double() - 127).repeat_interleave(32, 1)
    return w * s["w_s"].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * s["gscale"].double()


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {n: _rotated64(case, s[n], s["pos"]) for n in ("q", "k")}
    if case["op"] == "write":
        return {"q": _rotated64(case, s["q"], s["pos"]), "k": _held64(_rotated64(case, s["k"], s["pos"]), case["fmt"]),
                "v": _held64(s["v"].double(), case["fmt"])}
    x = torch.cat([_held64(part.double(), case["fmt"]) for part in s["x"].split(2048)])
    if case["op"] == "quant":
        return {"x": x}
    out = x @ _weights64(s).t()
    return {"out": out if s["bias"] is None else out + s["bias"].double()}
