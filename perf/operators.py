"""Cases for timing and comparing the operators of a 4-bit mixture-of-experts block.

The block around experts that were exported by awq_quantize_pack and awq_export_fp16:

* norm:    the RMS norms before and after the block, fused with the gate and the residual scale;
* route:   tokens sorted by expert, gathered into expert order (with the per-channel multipliers 1 / s of
           each expert, which cannot be folded into a norm that all experts share), and combined back with
           the router's weights;
* experts: the products of the sorted rows with each expert's 4-bit weights, plain or with the gated
           activation of a stacked gate/up pair.

Each comes forward and as its gradient. `own` selects the framework's entry points; otherwise `run` computes the same
in elementary torch operations, in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

GROUP = 128
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one decoded token through a 4096-wide block: the smallest call, where only its latency counts
        {"name": "norm-step", "op": "norm", "grad": False, "n": 1, "d": 4096, "dtype": "bf16", "gate": "channel"},
        # a long prompt through an 8192-wide block
        {"name": "norm-prompt", "op": "norm", "grad": False, "n": 8192, "d": 8192, "dtype": "bf16", "gate": "channel"},
        # a training batch of a 4096-wide block; the gate is a learned vector, so its gradient sums over tokens
        {"name": "norm-grad", "op": "norm", "grad": True, "n": 8192, "d": 4096, "dtype": "bf16", "gate": "channel"},
        # float32 training with a gate of each token's own, at an odd width and an odd number of tokens
        {"name": "norm-grad-odd", "op": "norm", "grad": True, "n": 1531, "d": 4097, "dtype": "f32", "gate": "token"},
        # one decoded token that goes to 8 of 64 narrow experts
        {"name": "route-step", "op": "route", "grad": False, "n": 1, "top_k": 8, "experts": 64, "d": 2048,
         "dtype": "bf16", "scaled": True, "dropped": 0.0, "skew": 0.0},
        # a prompt over 2 of 8 wide experts
        {"name": "route-prompt", "op": "route", "grad": False, "n": 16384, "top_k": 2, "experts": 8, "d": 4096,
         "dtype": "bf16", "scaled": True, "dropped": 0.0, "skew": 0.3},
        # the gradients of a batch over 8 of 64 experts, some slots dropped by a capacity limit or padding
        {"name": "route-grad", "op": "route", "grad": True, "n": 8191, "top_k": 8, "experts": 64, "d": 2048,
         "dtype": "bf16", "scaled": True, "dropped": 0.05, "skew": 0.5},
        # one decoded token through the gate/up pair of 2 of 8 experts of the 7B MLP's widths
        {"name": "experts-step", "op": "experts", "grad": False, "n": 1, "top_k": 2, "experts": 8, "d_in": 4096,
         "d_out": 22016, "act": "silu", "dtype": "bf16", "out": "same", "dropped": 0.0, "skew": 0.0},
        # a decoded batch over 4 of 32 narrow experts: a few rows for each
        {"name": "experts-batch", "op": "experts", "grad": False, "n": 48, "top_k": 4, "experts": 32, "d_in": 2048,
         "d_out": 2048, "act": "silu", "dtype": "bf16", "out": "same", "dropped": 0.0, "skew": 0.5},
        # a prompt through the gate/up pair of 2 of 8 experts
        {"name": "experts-prompt", "op": "experts", "grad": False, "n": 4096, "top_k": 2, "experts": 8, "d_in": 4096,
         "d_out": 22016, "act": "silu", "dtype": "bf16", "out": "same", "dropped": 0.0, "skew": 0.1},
        # the down projection of a shorter prompt with an odd number of tokens, float16, float32 out
        {"name": "experts-down", "op": "experts", "grad": False, "n": 1027, "top_k": 2, "experts": 8, "d_in": 11008,
         "d_out": 4096, "act": "none", "dtype": "f16", "out": "f32", "dropped": 0.02, "skew": 0.2},
        # the gradient of a batch's rows through the frozen gate/up weights
        {"name": "experts-grad", "op": "experts", "grad": True, "n": 4096, "top_k": 2, "experts": 8, "d_in": 4096,
         "d_out": 22016, "act": "none", "dtype": "bf16", "out": "same", "dropped": 0.0, "skew": 0.1},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "route", "experts", "experts"])
    grad = rng.random() < (0.5 if op != "experts" else 0.3)
    if op == "norm":
        d = rng.choice([128 * rng.randint(1, 224), 8 * rng.randint(8, 1024), rng.randint(1, 8200)])
        n = _spread(rng, 1, max(2, min(16384, (1 << 25) // d)))
        return {"op": op, "grad": grad, "n": n, "d": d, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "gate": rng.choice(["channel", "token", "none"])}
    experts = rng.choice([4, 8, 16, 32, 60, 64, 128])
    top_k = rng.randint(1, min(8, experts))
    tail = {"dropped": rng.choice([0.0, 0.0, 0.1]), "skew": round(rng.choice([0.0, rng.uniform(0.0, 0.8)]), 3)}
    if op == "route":
        d = rng.choice([128 * rng.randint(1, 64), 8 * rng.randint(8, 512), rng.randint(1, 4100)])
        n = _spread(rng, 1, max(2, min(16384, (1 << 26) // (d * top_k))))
        return {"op": op, "grad": grad, "n": n, "top_k": top_k, "experts": experts, "d": d,
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "scaled": rng.random() < 0.7, **tail}
    act = "none" if grad else rng.choice(["silu", "relu", "none"])
    d_in = 128 * rng.choice([rng.randint(1, 16), rng.randint(8, 48), rng.randint(32, 88)])
    widest = min(11008, (1 << 28) // (experts * d_in))  # an expert layer of at most 2^28 weights
    d_out = max(64, 2 * rng.randint(32, max(33, widest // 2)))
    if grad:
        d_out += d_out % 8 and 8 - d_out % 8
    n = _spread(rng, 1, max(2, min(8192, (1 << 38) // (top_k * d_in * d_out))))
    return {"op": op, "grad": grad, "n": n, "top_k": top_k, "experts": experts, "d_in": d_in, "d_out": d_out, "act": act,
            "dtype": rng.choice(["bf16", "bf16", "f16"]), "out": rng.choice(["same", "same", "f32"]), **tail}


# ---------------------------------------------------------------- inputs


def _activations(g, n, d, dtype):
    """Activations with a few outlier channels, as the calibrated layers see them."""
    x = torch.randn((n, d), generator=g, device="cuda")
    channel = 1.0 + 15.0 * (torch.rand(d, generator=g, device="cuda") < 0.004).float()
    return (x * channel).to(dtype)


def _expert_ids(g, c):
    """[n, top_k] distinct experts of each token (int64, as a top-k returns them), dropped slots -1."""
    n, k, e = c["n"], c["top_k"], c["experts"]
    noise = -torch.log(-torch.log(torch.rand((n, e), generator=g, device="cuda").clamp(1e-9, 1 - 1e-7)))
    popular = -c["skew"] * torch.log(torch.arange(1, e + 1, device="cuda", dtype=torch.float32))
    ids = torch.topk(noise + popular[torch.randperm(e, generator=g, device="cuda")], k, dim=1).indices
    return torch.where(torch.rand((n, k), generator=g, device="cuda") < c["dropped"], -1, ids)


def _sorted(ids, experts):
    """The stable order of the slots by expert: (offsets [experts + 1], order, position), int32; -1 where dropped."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=ids.device)).to(torch.int32)
    at = torch.arange(flat.numel(), device=ids.device, dtype=torch.int32)
    valid = at < offsets[experts]
    position = torch.empty_like(at)
    position[order] = torch.where(valid, at, -1)
    return offsets, torch.where(valid, order.to(torch.int32), -1), position.reshape(ids.shape)


def _weights(g, experts, d_out, d_in):
    """An export's codes, float16 steps (as bits) and packed zero points: normal weights on a 4-bit grid."""
    groups = d_in // GROUP
    q = torch.randn((experts, d_out, d_in), generator=g, device="cuda")
    q = q.mul_(2.6).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
    codes = q[..., 0::2] | (q[..., 1::2] << 4)
    spread = torch.rand((experts, d_out, groups), generator=g, device="cuda")
    steps = ((0.5 + spread) * 0.4 / math.sqrt(d_in)).to(torch.float16).view(torch.int16)
    z = torch.randint(6, 10, (experts, d_out, 2 * ((groups + 1) // 2)), generator=g, device="cuda", dtype=torch.uint8)
    return codes, steps, (z[..., 0::2] | (z[..., 1::2] << 4)).contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "norm":
        n, d = c["n"], c["d"]
        s["y"], s["residual"] = _activations(g, n, d, t), _activations(g, n, d, t)
        s["w_pre"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(t)
        s["w_post"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(t)
        s["gate"] = {"channel": lambda: torch.randn(d, generator=g, device="cuda").to(t),
                     "token": lambda: torch.randn((n, d), generator=g, device="cuda").to(t),
                     "none": lambda: None}[c["gate"]]()
        s["res_scale"] = 0.5
        if c["grad"]:
            s["d_res"] = torch.randn((n, d), generator=g, device="cuda").to(t)
            s["d_h"] = torch.randn((n, d), generator=g, device="cuda").to(t)
        return s
    s["ids"] = _expert_ids(g, c)
    n_rows = c["n"] * c["top_k"]
    if c["op"] == "route":
        d = c["d"]
        # what a program keeps: the experts' input multipliers, and the buffers of the expert-ordered rows, whose
        # part behind the last sorted row stays as it was
        s["in_scales"] = torch.exp(0.5 * torch.randn((c["experts"], d), generator=g, device="cuda")) if c["scaled"] else None
        s["weights"] = torch.softmax(torch.randn((c["n"], c["top_k"]), generator=g, device="cuda"), 1)
        s["rows"] = torch.zeros((n_rows, d), dtype=t, device="cuda")
        s["expert_out"] = _activations(g, n_rows, d, t)
        if c["grad"]:
            s["offsets"], s["order"], s["position"] = _sorted(s["ids"], c["experts"])
            s["d_out"] = torch.randn((c["n"], d), generator=g, device="cuda").to(t)
            s["d_rows_in"] = torch.randn((n_rows, d), generator=g, device="cuda").to(t)
        else:
            s["x"] = _activations(g, c["n"], d, t)
        return s
    s["offsets"], _, _ = _sorted(s["ids"], c["experts"])
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())  # the widest expert's rows (the plain form pads to it)
    s["codes"], s["steps"], s["zeros"] = _weights(g, c["experts"], c["d_out"], c["d_in"])
    out_t = torch.float32 if c["out"] == "f32" else t
    if c["grad"]:
        s["x"] = torch.randn((n_rows, c["d_out"]), generator=g, device="cuda").to(t)
        s["y"] = torch.zeros((n_rows, c["d_in"]), dtype=out_t, device="cuda")
    else:
        s["x"] = _activations(g, n_rows, c["d_in"], t)
        wide = c["d_out"] if c["act"] == "none" else c["d_out"] // 2
        s["y"] = torch.zeros((n_rows, wide), dtype=out_t, device="cuda")
    return s


# ---------------------------------------------------------------- the plain forms


def _norm(s):
    c, t = s["case"], s["y"].dtype
    y, r, w2 = s["y"].float(), s["residual"].float(), s["w_pre"].float()
    unit = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
    gate = s["res_scale"] if s["gate"] is None else s["res_scale"] * s["gate"].float()
    z = unit * s["w_post"].float()
    res = r + gate * z
    rstd2 = torch.rsqrt(res.square().mean(1, keepdim=True) + EPS)
    if not c["grad"]:
        return {"residual": res.to(t), "h": (res * rstd2 * w2).to(t)}
    dh, unit2 = s["d_h"].float(), res * rstd2
    dw2 = dh * w2
    dres = s["d_res"].float() + rstd2 * (dw2 - unit2 * (dw2 * unit2).mean(1, keepdim=True))
    rstd1 = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
    dz = dres * gate
    dw1 = dz * s["w_post"].float()
    out = {"d_residual": dres.to(t), "d_y": (rstd1 * (dw1 - unit * (dw1 * unit).mean(1, keepdim=True))).to(t),
           "d_w_pre": (dh * unit2).sum(0), "d_w_post": (dz * unit).sum(0)}
    if s["gate"] is not None:
        dgate = s["res_scale"] * dres * z
        out["d_gate"] = dgate.sum(0) if s["gate"].dim() == 1 else dgate.to(t)
    return out


def _route(s):
    c = s["case"]
    offsets, order, position = _sorted(s["ids"], c["experts"])
    valid = order >= 0
    slot = order.clamp(min=0).long()
    picked = s["x"][slot // c["top_k"]].float()
    if s["in_scales"] is not None:
        picked = picked * s["in_scales"][s["ids"].reshape(-1)[slot].clamp(min=0)]
    rows = torch.where(valid[:, None], picked.to(s["x"].dtype), s["rows"])
    back = s["expert_out"][position.clamp(min=0).long()].float() * s["weights"][..., None]
    out = torch.where((position >= 0)[..., None], back, 0.0).sum(1).to(s["x"].dtype)
    return {"offsets": offsets, "order": order, "position": position, "rows": rows, "out": out}


def _route_grad(s):
    c, t = s["case"], s["d_out"].dtype
    order, position = s["order"], s["position"]
    valid, slot = order >= 0, order.clamp(min=0).long()
    d_rows = s["d_out"][slot // c["top_k"]].float() * s["weights"].reshape(-1)[slot][:, None]
    d_rows = torch.where(valid[:, None], d_rows.to(t), s["rows"])
    at = position.clamp(min=0).long()
    kept = (position >= 0)[..., None]
    dots = (s["d_out"].float()[:, None] * s["expert_out"][at].float()).sum(2)
    d_x = s["d_rows_in"][at].float()
    if s["in_scales"] is not None:
        d_x = d_x * s["in_scales"][s["ids"].clamp(min=0)]
    return {"d_rows": d_rows, "d_weights": torch.where(kept[..., 0], dots, 0.0),
            "d_x": torch.where(kept, d_x, 0.0).sum(1).to(t)}


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _dequantized(codes, steps, zeros, t):
    """[.., d_out, d_in] weights (q - zero) * step, rounded once to the operands' 16-bit type, as float32."""
    q = _nibbles(codes).float().unflatten(-1, (-1, GROUP))
    z = _nibbles(zeros)[..., :q.shape[-2]].float()
    w = (q - z[..., None]) * steps.view(torch.float16).float()[..., None]
    return w.flatten(-2).to(t).float()


def _experts(s):
    """Rows of the same expert side by side, padded to the widest; with no more rows than experts, each row for itself."""
    c, x, offsets = s["case"], s["x"], s["offsets"].long()
    experts, n = c["experts"], x.shape[0]
    at = torch.arange(n, device=x.device)
    e = torch.searchsorted(offsets[1:], at, right=True).clamp(max=experts - 1)
    if n <= experts:
        w = _dequantized(s["codes"][e], s["steps"][e], s["zeros"][e], x.dtype)
        y = torch.bmm(x.float()[:, None], w if c["grad"] else w.transpose(1, 2))[:, 0]
    else:
        w = _dequantized(s["codes"], s["steps"], s["zeros"], x.dtype)
        pad = offsets[:-1, None] + torch.arange(max(s["most"], 1), device=x.device)
        y = torch.bmm(x[pad.clamp(max=n - 1)].float(), w if c["grad"] else w.transpose(1, 2))
        y = y[e, (at - offsets[e]).clamp(0, y.shape[1] - 1)]
    if c["act"] != "none":
        gate, up = y.chunk(2, 1)
        y = (gate * torch.sigmoid(gate) if c["act"] == "silu" else gate.clamp(min=0)) * up
    return {"y": torch.where((at < offsets[experts])[:, None], y.to(s["y"].dtype), s["y"])}


# ---------------------------------------------------------------- the framework's calls


def _own(s):
    from post_quantization_mean_amd import moe
    c = s["case"]
    if c["op"] == "norm":
        if c["grad"]:
            return moe.awq_block_norm_backward(s["y"], s["residual"], s["d_res"], s["d_h"], w_pre=s["w_pre"], w_post=s["w_post"],
                                               gate=s["gate"], res_scale=s["res_scale"], eps=EPS)
        return moe.awq_block_norm(s["y"], s["residual"], w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"],
                                  res_scale=s["res_scale"], eps=EPS)
    if c["op"] == "route":
        scaled = {} if s["in_scales"] is None else {"expert_ids": s["ids"], "in_scales": s["in_scales"]}
        if c["grad"]:
            r = moe.awq_moe_combine_backward(s["d_out"], s["expert_out"], s["position"], s["weights"], out={"d_rows": s["rows"]})
            return {**r, "d_x": moe.awq_moe_gather_backward(s["d_rows_in"], s["position"], **scaled)}
        plan = moe.awq_moe_sort(s["ids"], c["experts"])
        rows = moe.awq_moe_gather(s["x"], plan["position"], out=s["rows"], **scaled)
        return {**plan, "rows": rows, "out": moe.awq_moe_combine(s["expert_out"], plan["position"], s["weights"])}
    if c["grad"]:
        return {"y": moe.awq_w4a16_grouped_gemm_backward(s["x"], s["codes"], s["steps"], s["zeros"], s["offsets"], dx=s["y"])}
    return {"y": moe.awq_w4a16_grouped_gemm(s["x"], s["codes"], s["steps"], s["zeros"], s["offsets"],
                                            act=None if c["act"] == "none" else c["act"], y=s["y"])}


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "norm":
        return _norm(state)
    if c["op"] == "route":
        return _route_grad(state) if c["grad"] else _route(state)
    return _experts(state)


# ---------------------------------------------------------------- the least work, and the definition in 64 bits


def _distinct(c):
    """Expected number of experts that get a row."""
    share = [(i + 1) ** -c["skew"] for i in range(c["experts"])]
    kept = c["top_k"] * (1 - c["dropped"]) / sum(share)
    return sum(1 - (1 - min(1.0, p * kept)) ** c["n"] for p in share)


def work(case):
    c = case
    b, n = SIZES[c["dtype"]], c["n"]
    if c["op"] == "norm":
        token, channel = c["gate"] == "token", c["gate"] == "channel"
        if c["grad"]:
            wide = 6 + 2 * token  # y, residual, d_res, d_h, d_y, d_residual; the gate and its gradient
            return {"bytes": c["d"] * (n * wide * b + (2 + channel) * (b + 4)), "flops": 40 * n * c["d"]}
        return {"bytes": c["d"] * (n * (4 + token) * b + (2 + channel) * b), "flops": 14 * n * c["d"]}
    slots = n * c["top_k"]
    kept = slots * (1 - c["dropped"])
    if c["op"] == "route":
        d = c["d"]
        scales = 4 * d * _distinct(c) if c["scaled"] else 0
        if c["grad"]:  # d_out once, d_rows written, expert_out and d_rows_in read, d_x written, positions and weights
            return {"bytes": int(d * b * (2 * n + 3 * kept) + scales + slots * 16), "flops": int(6 * kept * d)}
        return {"bytes": int(d * b * (2 * n + 2 * kept) + scales + slots * 24), "flops": int(3 * kept * d)}
    layer = c["d_in"] * c["d_out"]
    weights = _distinct(c) * layer * (0.5 + 2.5 / GROUP)
    wide = c["d_out"] if c["act"] == "none" else c["d_out"] // 2
    out_b = 4 if c["out"] == "f32" else b
    rows_in, rows_out = (c["d_out"], c["d_in"]) if c["grad"] else (c["d_in"], wide)
    return {"bytes": int(weights + kept * (rows_in * b + rows_out * out_b)), "flops": int(2 * kept * layer)}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        y, r = s["y"].double(), s["residual"].double()
        a, w = s["w_post"].double(), s["w_pre"].double()
        k = torch.full_like(y, s["res_scale"]) if s["gate"] is None else s["res_scale"] * s["gate"].double().expand_as(y)
        n1 = (y.pow(2).sum(1, True) / c["d"] + EPS).sqrt()
        res = r + k * (y / n1) * a
        n2 = (res.pow(2).sum(1, True) / c["d"] + EPS).sqrt()
        if not c["grad"]:
            return {"residual": res, "h": res / n2 * w}
        gh = s["d_h"].double() * w
        gres = s["d_res"].double() + gh / n2 - res * (gh * res).sum(1, True) / (c["d"] * n2 ** 3)
        gz = gres * k * a
        out = {"d_residual": gres, "d_y": gz / n1 - y * (gz * y).sum(1, True) / (c["d"] * n1 ** 3),
               "d_w_pre": (s["d_h"].double() * res / n2).sum(0), "d_w_post": (gres * k * y / n1).sum(0)}
        if s["gate"] is not None:
            gg = s["res_scale"] * gres * y / n1 * a
            out["d_gate"] = gg.sum(0) if s["gate"].dim() == 1 else gg
        return out
    ids = s["ids"].reshape(-1)
    experts, slots = c["experts"], ids.numel()
    if c["op"] == "route":
        # the place of a slot: the slots of lower experts and the earlier ones of its own, counted
        places, count = torch.full((slots,), -1, dtype=torch.int32, device=ids.device), 0
        order = torch.full((slots,), -1, dtype=torch.int32, device=ids.device)
        offsets = [0]
        for e in range(experts):
            mine = (ids == e).nonzero()[:, 0]
            places[mine] = torch.arange(count, count + mine.numel(), dtype=torch.int32, device=ids.device)
            order[count:count + mine.numel()] = mine.to(torch.int32)
            count += mine.numel()
            offsets.append(count)
        token = order[:count].long() // c["top_k"]
        scale = None if s["in_scales"] is None else s["in_scales"].double()
        if c["grad"]:
            d_rows = s["rows"].double().clone()
            d_rows[:count] = s["d_out"].double()[token] * s["weights"].double().reshape(-1)[order[:count].long()][:, None]
            d_w = torch.zeros(slots, dtype=torch.float64, device=ids.device)
            d_w[order[:count].long()] = (s["d_out"].double()[token] * s["expert_out"][:count].double()).sum(1)
            back = s["d_rows_in"][:count].double()
            if scale is not None:
                back = back * scale[ids[order[:count].long()]]
            d_x = torch.zeros((c["n"], c["d"]), dtype=torch.float64, device=ids.device).index_add_(0, token, back)
            return {"d_rows": d_rows, "d_weights": d_w.reshape(c["n"], -1), "d_x": d_x}
        rows = s["rows"].double().clone()
        rows[:count] = s["x"].double()[token]
        if scale is not None:
            rows[:count] *= scale[ids[order[:count].long()]]
        weighed = s["expert_out"][:count].double() * s["weights"].double().reshape(-1)[order[:count].long()][:, None]
        out = torch.zeros((c["n"], c["d"]), dtype=torch.float64, device=ids.device).index_add_(0, token, weighed)
        return {"offsets": torch.tensor(offsets, dtype=torch.int32, device=ids.device), "order": order,
                "position": places.reshape(c["n"], -1), "rows": rows, "out": out}
    y = s["y"].double().clone()
    ends = s["offsets"].tolist()
    for e in range(experts):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        low, high = (s["codes"][e] & 15).double(), (s["codes"][e] >> 4).double()
        q = torch.empty((c["d_out"], c["d_in"]), dtype=torch.float64, device=y.device)
        q[:, 0::2], q[:, 1::2] = low, high
        g = torch.arange(c["d_in"], device=y.device) // GROUP
        zb = s["zeros"][e][:, g // 2]
        z = torch.where(g % 2 == 0, zb & 15, zb >> 4).double()
        step = s["steps"][e].view(torch.float16).double()[:, g]
        w = ((q - z) * step).to(s["x"].dtype).double()
        part = s["x"][lo:hi].double() @ (w if c["grad"] else w.t())
        if c["act"] != "none":
            gate, up = part[:, :c["d_out"] // 2], part[:, c["d_out"] // 2:]
            part = (gate / (1 + torch.exp(-gate)) if c["act"] == "silu" else torch.relu(gate)) * up
        y[lo:hi] = part
    return {"y": y}
