"""Cases for timing and comparing the operators of attention over a cache of 4-bit keys and values.

Attention around linears that were exported by awq_quantize_pack and awq_export_fp16, between the QKV product and the
output product:

* rope:   rotary positions with one or several axes (text; time, height and width), and its gradient;
* cache:  new keys and values quantized as they are written to their slots of a paged cache, and read back from there;
* attend: attention of new tokens over the cached ones: single tokens, drafts of a few, prompts.

A cache holds groups of 128 consecutive channels of a head (the last one shorter) as codes 0 .. 15 with a float16 step and a
float16 offset; a code stands for offset + code * step. `own` selects the framework's entry points; otherwise `run` computes
the same in elementary torch operations, in 32 bits (angles and codes, which lie next to borders, in 64), rounded once at
the end.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 128
BIG = 65024.0  # values saturate here, inside float16's range
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one decoded token: 32 query and 8 key heads of 128 in one fused QKV row; only latency counts
        {"name": "rope-step", "op": "rope", "grad": False, "n": 1, "heads": 40, "d": 128, "rot": 128, "axes": 1, "style": "half", "dtype": "bf16"},
        # a long video prompt through the 70B layer's 64 query and 8 key heads: time, height and width
        {"name": "rope-video", "op": "rope", "grad": False, "n": 16384, "heads": 72, "d": 128, "rot": 128, "axes": 3, "style": "half", "dtype": "bf16"},
        # float32 training over images: two axes, heads of 80, adjacent pairs, an odd number of tokens
        {"name": "rope-grad-image", "op": "rope", "grad": True, "n": 4099, "heads": 16, "d": 80, "rot": 80, "axes": 2, "style": "pairs", "dtype": "f32"},
        # a decoded batch of 64 tokens, 8 key heads of 128
        {"name": "cache-step", "op": "cache", "n": 64, "kv_heads": 8, "d": 128, "page": 64, "dtype": "bf16", "out": "same", "dropped": 0.0},
        # the keys and values of a long prompt
        {"name": "cache-prompt", "op": "cache", "n": 32768, "kv_heads": 8, "d": 128, "page": 64, "dtype": "bf16", "out": "same", "dropped": 0.0},
        # float32, an odd number of tokens with padding among them, heads of 96, small pages
        {"name": "cache-odd", "op": "cache", "n": 5003, "kv_heads": 32, "d": 96, "page": 16, "dtype": "f32", "out": "same", "dropped": 0.1},
        # one decoded token of the 7B layer (32 heads with keys of their own) over a short context
        {"name": "attend-step", "op": "attend", "seqs": 1, "q": 1, "kv": 2047, "ragged": False, "heads": 32, "kv_heads": 32, "d": 128,
         "page": 64, "window": 0, "causal": True, "dtype": "bf16"},
        # a decoded batch of the 70B layer (64 heads on 8 key heads) over contexts of many lengths, an empty one among them
        {"name": "attend-batch", "op": "attend", "seqs": 64, "q": 1, "kv": 8192, "ragged": True, "heads": 64, "kv_heads": 8, "d": 128,
         "page": 64, "window": 0, "causal": True, "dtype": "bf16"},
        # one decoded token over a very long context
        {"name": "attend-long", "op": "attend", "seqs": 1, "q": 1, "kv": 131071, "ragged": False, "heads": 64, "kv_heads": 8, "d": 128,
         "page": 128, "window": 0, "causal": True, "dtype": "bf16"},
        # drafts of five tokens for each of 24 sequences, heads of 256, small pages, a sliding window
        {"name": "attend-draft", "op": "attend", "seqs": 24, "q": 5, "kv": 6001, "ragged": False, "heads": 16, "kv_heads": 8, "d": 256,
         "page": 16, "window": 2048, "causal": True, "dtype": "f16"},
        # short prompts of many lengths together, heads of 64
        {"name": "attend-prompts", "op": "attend", "seqs": 9, "q": 1500, "kv": 2000, "ragged": True, "heads": 32, "kv_heads": 8, "d": 64,
         "page": 32, "window": 0, "causal": True, "dtype": "f16"},
        # a chunk of 4096 tokens of a long prompt behind 8192 cached ones
        {"name": "attend-prompt", "op": "attend", "seqs": 1, "q": 4096, "kv": 12288, "ragged": False, "heads": 64, "kv_heads": 8, "d": 128,
         "page": 64, "window": 0, "causal": True, "dtype": "bf16"},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "attend", "attend"])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 128, 256, 2 * rng.randint(4, 128)])
        rot = d if rng.random() < 0.7 else 2 * rng.randint(1, d // 2)
        heads = rng.randint(1, 80)
        n = _spread(rng, 1, max(2, min(32768, (1 << 27) // (heads * d))))
        axes = rng.choice([1, 2, 3, 3]) if rot >= 8 else 1
        return {"op": op, "grad": rng.random() < 0.5, "n": n, "heads": heads, "d": d, "rot": rot, "axes": axes,
                "style": rng.choice(["half", "pairs"]), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    d = rng.choice([64, 128, 128, 256, 32 * rng.randint(1, 8)])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "cache":
        kv_heads = rng.choice([1, 2, 4, 8, 16, 32, rng.randint(1, 40)])
        n = _spread(rng, 1, max(2, min(32768, (1 << 25) // (kv_heads * d))))
        return {"op": op, "n": n, "kv_heads": kv_heads, "d": d, "page": page, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "out": rng.choice(["same", "same", "f32"]), "dropped": rng.choice([0.0, 0.0, 0.1])}
    kv_heads = rng.choice([1, 2, 4, 8, 16, 32])
    heads = min(64, kv_heads * rng.choice([1, 1, 2, 4, 5, 8, 16]))
    heads = max(kv_heads, heads // kv_heads * kv_heads)
    seqs = _spread(rng, 1, 96)
    q = rng.choice([1, 1, 1, rng.randint(2, 16), _spread(rng, 17, 4096)])
    kv = max(q, _spread(rng, 1, 131072))
    while seqs > 1 and (seqs * kv * kv_heads * d > 1 << 29 or seqs * q * kv * heads * d > 1 << 37):
        seqs = (seqs + 1) // 2 if seqs > 2 else 1
    while seqs * kv * kv_heads * d > 1 << 29:
        kv = max(q, kv // 2)
    while q > 1 and q * kv * heads * d > 1 << 38:
        q = (q + 1) // 2 if q > 2 else 1
    return {"op": op, "seqs": seqs, "q": q, "kv": kv, "ragged": seqs > 1 and rng.random() < 0.5, "heads": heads, "kv_heads": kv_heads, "d": d,
            "page": page, "window": rng.choice([0, 0, 0, _spread(rng, 16, 8192)]), "causal": rng.random() < 0.8,
            "dtype": rng.choice(["bf16", "f16"])}


def _lengths(c):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    if not c["ragged"]:
        return [c["q"]] * c["seqs"], [c["kv"]] * c["seqs"]
    rng = random.Random(c["seqs"] * c["kv"])
    q = [c["q"] if c["q"] <= 16 else rng.randint(max(1, c["q"] // 16), c["q"]) for _ in range(c["seqs"])]
    kv = [max(a, rng.randint(c["kv"] // 8, c["kv"])) for a in q]
    q[0], kv[0] = c["q"], c["kv"]
    if c["q"] == 1:
        kv[-1] = 0  # a padded sequence: its token sees nothing
    elif c["seqs"] > 2:
        q[-1] = 0  # a sequence without new tokens
    return q, kv


# ---------------------------------------------------------------- inputs


def _frequencies(c):
    """float32 frequencies of the rotated pairs and each pair's axis."""
    half = c["rot"] // 2
    i = torch.arange(half, dtype=torch.float64)
    if c["axes"] == 2:  # each axis with frequencies of its own
        first = (half + 1) // 2
        axis = (i >= first).to(torch.int32)
        freq = 10000.0 ** (-(i - first * axis) / max(first, 1))
    else:
        freq = 1000000.0 ** (-i / half)
        axis = ((i >= half // 4).to(torch.int32) + (i >= half // 4 + (half - half // 4) // 2).to(torch.int32)) * int(c["axes"] == 3)
    return freq.float().cuda(), axis.to(torch.int32).cuda()


def _positions(c, g):
    """int32 [axes, n]: running tokens of a text, or the places of a grid behind one."""
    i = torch.arange(c["n"], device="cuda")
    start = int(torch.randint(0, 200000, (1,), generator=g, device="cuda"))
    if c["axes"] == 1:
        return (i + start).to(torch.int32)[None].contiguous()
    wide = max(1, min(48, int(math.sqrt(c["n"]))))
    high = max(1, min(30, c["n"] // wide))
    grid = [start + i // (wide * high), start + i // wide % high, start + i % wide]
    return torch.stack(grid[3 - c["axes"]:]).to(torch.int32)


def _heads(g, n, heads, d, t):
    """Keys or values: normal, a few channels of each head far wider and off zero."""
    x = torch.randn((n, heads, d), generator=g, device="cuda")
    wide = (torch.rand((heads, d), generator=g, device="cuda") < 0.03).float()
    x = x * (1 + 3 * wide) + 4 * wide * torch.randn((heads, d), generator=g, device="cuda")
    return x.to(t)


def _empty_cache(pages, kv_heads, d, page):
    """What a program keeps: codes [pages, 2, kv_heads, page, d / 2] and (step, offset) [pages, 2, kv_heads, groups, page, 2]."""
    groups = (d + GROUP - 1) // GROUP
    return (torch.zeros((pages, 2, kv_heads, page, d // 2), dtype=torch.uint8, device="cuda"),
            torch.zeros((pages, 2, kv_heads, groups, page, 2), dtype=torch.float16, device="cuda"))


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "rope":
        s["x"] = torch.randn((c["n"], c["heads"], c["d"]), generator=g, device="cuda").to(t)
        s["positions"] = _positions(c, g)
        s["inv_freq"], s["axis"] = _frequencies(c)
        return s
    d, kvh, page = c["d"], c["kv_heads"], c["page"]
    if c["op"] == "cache":
        n = c["n"]
        s["k"], s["v"] = _heads(g, n, kvh, d, t), _heads(g, n, kvh, d, t)
        pages = (n + page - 1) // page + 3
        s["codes"], s["params"] = _empty_cache(pages, kvh, d, page)
        # runs of a sequence's tokens over pages anywhere; a padded token has no slot
        at = torch.arange(n, device="cuda") + int(torch.randint(0, page, (1,), generator=g, device="cuda"))
        slots = torch.randperm(pages, generator=g, device="cuda")[at // page] * page + at % page
        s["slots"] = torch.where(torch.rand(n, generator=g, device="cuda") < c["dropped"], -1, slots)
        out = torch.float32 if c["out"] == "f32" else t
        s["k_out"], s["v_out"] = (torch.zeros((n, kvh, d), dtype=out, device="cuda") for _ in range(2))
        return s
    s["q_len"], s["kv_len"] = _lengths(c)
    offsets = [0]
    for a in s["q_len"]:
        offsets.append(offsets[-1] + a)
    s["q"] = (1.5 * torch.randn((offsets[-1], c["heads"], d), generator=g, device="cuda")).to(t)
    wide = max(1, max((a + page - 1) // page for a in s["kv_len"]))
    pages = sum((a + page - 1) // page for a in s["kv_len"]) + 1
    s["codes"], s["params"] = _empty_cache(pages, kvh, d, page)
    step = max(1, (1 << 26) // (2 * kvh * page * d))
    for at in range(0, pages, step):  # a cache full of quantized tokens
        m = min(step, pages - at)
        x = _heads(g, m * page, 2 * kvh, d, torch.float32).view(m, page, 2, kvh, d).permute(0, 2, 3, 1, 4)
        for lo in range(0, d, GROUP):
            part = x[..., lo:lo + GROUP]
            low, high = part.amin(-1, keepdim=True), part.amax(-1, keepdim=True)
            size = ((high - low) / 15).half()
            codes = ((part - low.half()) / size).round().clamp(0, 15).to(torch.uint8)
            s["codes"][at:at + m, ..., lo // 2:(lo + GROUP) // 2] = codes[..., 0::2] | (codes[..., 1::2] << 4)
            s["params"][at:at + m, :, :, lo // GROUP] = torch.cat([size, low.half()], -1)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["seqs"], wide), -1, dtype=torch.int32, device="cuda")
    used = 0
    for i, a in enumerate(s["kv_len"]):
        m = (a + page - 1) // page
        table[i, :m] = order[used:used + m]
        used += m
    s["table"] = table
    s["kv_lens"] = torch.tensor(s["kv_len"], dtype=torch.int32, device="cuda")
    # sequences with the same number of new tokens need no offsets
    s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda") if len(set(s["q_len"])) > 1 else None
    s["scale"] = 1 / math.sqrt(d)
    return s


# ---------------------------------------------------------------- the plain forms


def _rope(s):
    c, t = s["case"], s["x"].dtype
    half = c["rot"] // 2
    angle = s["positions"].double()[s["axis"].long()].t() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["grad"]:
        sin = -sin
    x = s["x"].float()
    y = x.clone()
    if c["style"] == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    return {"x": y.to(t)}


def _to_half(v):
    """float64 to float16, rounded once (a conversion by way of float32 would round twice)."""
    e = torch.frexp(v).exponent.clamp(min=-13)
    unit = ((e.long() + (1023 - 11)) << 52).view(torch.float64)  # 2^(e - 11) by its bits
    return (torch.round(v / unit) * unit).half()


def _write(s, x, which):
    slots, page = s["slots"], s["case"]["page"]
    kept = slots >= 0
    p, r = (slots // page)[kept], (slots % page)[kept]
    x = x[kept].double().clamp(-BIG, BIG)
    for lo in range(0, x.shape[2], GROUP):
        part = x[..., lo:lo + GROUP]
        low, high = part.amin(-1, keepdim=True), part.amax(-1, keepdim=True)
        step, offset = _to_half((high - low) / torch.full_like(high, 15.0)), _to_half(low)
        codes = torch.where(step > 0, (part - offset.double()) / step.double(), 0.0).round().clamp(0, 15).to(torch.uint8)
        s["codes"][p, which, :, r, lo // 2:(lo + GROUP) // 2] = codes[..., 0::2] | (codes[..., 1::2] << 4)
        s["params"][p, which, :, lo // GROUP, r] = torch.cat([step, offset], -1)


def _values(codes, params):
    """float32 values of codes [..., m, d / 2] with params [..., groups, m, 2]."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    step, offset = params.float().transpose(-3, -2).repeat_interleave(GROUP, -2)[..., :q.shape[-1], :].unbind(-1)
    return offset + q * step


def _cache(s):
    page, slots = s["case"]["page"], s["slots"]
    _write(s, s["k"], 0)
    _write(s, s["v"], 1)
    kept = slots >= 0
    p, r = (slots // page).clamp(min=0), slots % page
    out = {}
    for which, name in enumerate(("k", "v")):
        x = _values(s["codes"][p, which, :, r], s["params"][p, which, :, :, r].transpose(1, 2))
        out[name] = torch.where(kept[:, None, None], x.to(s[name + "_out"].dtype), s[name + "_out"])
    return out


def _seen(c, first, last, q_len, kv_len, device):
    """Which cached tokens the new tokens first .. last - 1 of a sequence see."""
    at = torch.arange(first, last, device=device)[:, None] + (kv_len - q_len)
    j = torch.arange(kv_len, device=device)
    seen = j <= at if c["causal"] else torch.ones_like(j <= at)
    return seen & (j > at - c["window"]) if c["window"] else seen


def _attend(s):
    c, out = s["case"], torch.zeros_like(s["q"])
    group, page, first = c["heads"] // c["kv_heads"], c["page"], 0
    for i, (n, m) in enumerate(zip(s["q_len"], s["kv_len"])):
        if n and m:
            pages = s["table"][i, :(m + page - 1) // page].long()
            kv = _values(s["codes"][pages], s["params"][pages]).permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :m]
            step = max(1, (1 << 30) // (group * m))
            for lo in range(0, n, step):
                hi = min(n, lo + step)
                seen = _seen(c, lo, hi, n, m, out.device)
                for h in range(c["kv_heads"]):
                    q = s["q"][first + lo:first + hi, h * group:(h + 1) * group].float().transpose(0, 1)
                    x = torch.where(seen, torch.matmul(q.reshape(-1, c["d"]), kv[0, h].t().contiguous()).view(group, hi - lo, m) * s["scale"], -math.inf)
                    top = x.amax(-1, keepdim=True)
                    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
                    total = p.sum(-1, keepdim=True)
                    y = torch.matmul(p.reshape(-1, m), kv[1, h]).view(group, hi - lo, c["d"]) / torch.where(total > 0, total, 1.0)
                    out[first + lo:first + hi, h * group:(h + 1) * group] = y.transpose(0, 1).to(out.dtype)
        first += n
    return {"out": out}


# ---------------------------------------------------------------- the framework's calls


def _own(s):
    from post_quantization_mean_amd import attn
    c = s["case"]
    if c["op"] == "rope":
        call = attn.awq_rope_backward if c["grad"] else attn.awq_rope
        return {"x": call(s["x"], s["positions"], s["inv_freq"], axis=s["axis"] if c["axes"] > 1 else None, style=c["style"])}
    if c["op"] == "cache":
        attn.awq_kv4_write(s["k"], s["v"], s["codes"], s["params"], s["slots"])
        k, v = attn.awq_kv4_read(s["codes"], s["params"], s["slots"], out=(s["k_out"], s["v_out"]))
        return {"k": k, "v": v}
    return {"out": attn.awq_kv4_attention(s["q"], s["codes"], s["params"], s["table"], s["kv_lens"], q_offsets=s["offsets"],
                                          scale=s["scale"], causal=c["causal"], window=c["window"], max_kv=max(s["kv_len"]))}


def run(state):
    if own:
        return _own(state)
    return {"rope": _rope, "cache": _cache, "attend": _attend}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the least work, and the definition in 64 bits


def _pairs(c):
    """(pairs of a new and a cached token that see each other, cached tokens that any new token sees)."""
    pairs = tokens = 0
    for n, m in zip(*_lengths(c)):
        if not n or not m:
            continue
        w = c["window"] or m + n
        for i in (range(n) if c["causal"] or c["window"] else ()):
            at = m - n + i
            pairs += max(0, (at + 1 if c["causal"] else m) - max(0, at + 1 - w))
        if not c["causal"] and not c["window"]:
            pairs += n * m
        tokens += m - max(0, m - n + 1 - w)
    return pairs, tokens


def work(case):
    c = case
    b = SIZES[c["dtype"]]
    if c["op"] == "rope":
        n = c["n"]
        return {"bytes": 2 * n * c["heads"] * c["d"] * b + 4 * n * c["axes"] + 4 * c["rot"], "flops": 3 * n * c["heads"] * c["rot"]}
    d = c["d"]
    row = d // 2 + 4 * ((d + GROUP - 1) // GROUP)  # bytes of a token's codes, step and offset in one head
    if c["op"] == "cache":
        kept = c["n"] * (1 - c["dropped"])
        out = 4 if c["out"] == "f32" else b
        return {"bytes": int(2 * kept * c["kv_heads"] * (d * b + 2 * row + d * out) + 16 * c["n"]), "flops": int(2 * kept * c["kv_heads"] * d * 8)}
    pairs, tokens = _pairs(c)
    return {"bytes": int(2 * tokens * c["kv_heads"] * row + 2 * sum(_lengths(c)[0]) * c["heads"] * d * b + 4 * tokens / c["page"]),
            "flops": int(4 * pairs * c["heads"] * d)}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        x = s["x"].double()
        y, half = x.clone(), c["rot"] // 2
        turn = -1.0 if c["grad"] else 1.0
        for i in range(half):
            a, b = (i, i + half) if c["style"] == "half" else (2 * i, 2 * i + 1)
            angle = turn * s["positions"][int(s["axis"][i])].double() * float(s["inv_freq"][i])
            z = torch.polar(torch.ones_like(angle), angle)[:, None] * torch.complex(x[..., a], x[..., b])
            y[..., a], y[..., b] = z.real, z.imag
        return {"x": y}
    if c["op"] == "cache":
        out = {}
        kept = (s["slots"] >= 0).cpu().numpy()
        for name in ("k", "v"):
            x = s[name].double().cpu().numpy().clip(-BIG, BIG)
            y = s[name + "_out"].double().cpu().numpy()
            for lo in range(0, c["d"], GROUP):
                part = x[..., lo:lo + GROUP]
                low = part.min(-1, keepdims=True)
                step = ((part.max(-1, keepdims=True) - low) / 15).astype(np.float16).astype(np.float64)
                low = low.astype(np.float16).astype(np.float64)
                code = np.rint(np.divide(part - low, step, out=np.zeros_like(part), where=step > 0)).clip(0, 15)
                y[..., lo:lo + GROUP] = np.where(kept[:, None, None], low + code * step, y[..., lo:lo + GROUP])
            out[name] = torch.from_numpy(y).cuda()
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, page, start = c["heads"] // c["kv_heads"], c["page"], 0
    for i, (n, m) in enumerate(zip(s["q_len"], s["kv_len"])):
        pages = s["table"][i, :(m + page - 1) // page].long()
        for h in range(c["kv_heads"] if n and m else 0):
            kv = []
            for which in (0, 1):
                codes = s["codes"][pages, which, h].flatten(0, 1)[:m]
                params = s["params"][pages, which, h].transpose(1, 2).flatten(0, 1)[:m].double()
                x = torch.empty((m, c["d"]), dtype=torch.float64, device="cuda")
                x[:, 0::2], x[:, 1::2] = codes % 16, codes // 16
                for lo in range(0, c["d"], GROUP):
                    x[:, lo:lo + GROUP] = x[:, lo:lo + GROUP] * params[:, lo // GROUP, :1] + params[:, lo // GROUP, 1:]
                kv.append(x)
            for lo in range(0, n, max(1, (1 << 27) // m)):
                hi = min(n, lo + max(1, (1 << 27) // m))
                seen = _seen(c, lo, hi, n, m, "cuda")
                for a in range(h * group, (h + 1) * group):
                    score = (s["q"][start + lo:start + hi, a].double() @ kv[0].t()) * s["scale"]
                    p = torch.softmax(score.masked_fill(~seen, -math.inf), -1)
                    out[start + lo:start + hi, a] = torch.where(seen.any(1, keepdim=True), p, 0.0) @ kv[1]
        start += n
    return {"out": out}
