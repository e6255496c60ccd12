"""Inputs shared by the tests of attention over the 4-bit cache."""
import numpy as np
import torch

from oracle import awq_attn as A


def random_cache(rng, n_pages, n_kv, d, page, exact=False):
    """(codes, params) of a cache full of quantized tokens: any codes, steps and offsets of normal keys and values; with
    `exact` steps are powers of two and offsets eighths, so that every number is a float16 and scores are sums without
    rounding."""
    g = (d + 127) // 128
    codes = rng.integers(0, 256, (n_pages, 2, n_kv, page, d // 2)).astype(np.uint8)
    shape = (n_pages, 2, n_kv, g, page)
    if exact:
        step, offset = 2.0 ** rng.integers(-4, -1, shape), rng.integers(-16, 9, shape) / 8
    else:
        step, offset = rng.uniform(0.15, 0.45, shape), rng.uniform(-3.5, -1.5, shape)
    return codes, np.stack([step, offset], -1).astype(np.float16)


def cache_dev(codes, params, apart=0):
    """The cache on the device; with `apart`, pages that many elements apart more than they are large."""
    c, p = torch.from_numpy(codes).cuda(), torch.from_numpy(params).cuda()
    if not apart:
        return c, p
    out = []
    for t, gap in ((c, 16 * apart), (p, 8 * apart)):
        wide = torch.full((t.shape[0], t[0].numel() + gap), 7, dtype=t.dtype, device="cuda")
        part = wide[:, :t[0].numel()].unflatten(1, t.shape[1:])
        part.copy_(t)
        out.append(part)
    return tuple(out)


def paged(rng, kv_len, page, spare=2, wide=0):
    """(table, pages): each sequence's pages anywhere in the cache, -1 past its end."""
    used = [(m + page - 1) // page for m in kv_len]
    pages = sum(used) + spare
    order = rng.permutation(pages)
    table = np.full((len(kv_len), max(used + [1]) + wide), -1, np.int32)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = order[at:at + n]
        at += n
    return table, pages


def attention_bound(q, codes, params, table, kv_len, q_offsets, scale, causal, window, out, exact=False):
    """How far the kernels' outputs may be from the definition, [n, heads, d] (without the output's own rounding).

    Keys and values are rounded to float16, 2^-11 of each number; scores are sums of d float32 products, each addition off
    by at most 2^-24 of the sum of magnitudes (exact inputs have neither error). A score that is off by e makes a weight off by 2 e,
    its share of the sum included; a numerator's rounding towards zero adds 2^-10, twice for the same reason; numerators below
    2^-31 of the largest are lost. Sums over n tokens are float32. All relative to the sum of |weight * value|."""
    n, heads, d = q.shape
    group = heads // codes.shape[2]
    bound = np.zeros((n, heads, d))
    size, pages = codes.shape[3], codes.shape[0]
    for s in range(len(kv_len)):
        first, last = int(q_offsets[s]), int(q_offsets[s + 1])
        m = int(kv_len[s])
        if not m or last <= first:
            continue
        j = np.arange(m)
        page = table[s][j // size]
        there = (page >= 0) & (page < pages)
        k, v = A.cached(codes, params, np.where(there, page, 0), j % size)
        for i in range(first, last):
            p = m - (last - first) + i - first
            at = np.flatnonzero(there & ((j <= p) if causal else True) & ((j > p - window) if window else True))
            if not len(at):
                continue
            for h in range(heads):
                kk, vv = k[at, h // group], v[at, h // group]
                x = kk @ q[i, h] * scale
                w = np.exp(x - x.max())
                w /= w.sum()
                e = 0.0 if exact else np.max(np.abs(kk) @ np.abs(q[i, h])) * abs(scale) * (2.0 ** -11 + d * 2.0 ** -24)
                size_of = w @ np.abs(vv)
                # exp of a float32: the score times log2(e) is rounded twice
                e += (np.max(np.abs(x)) + 1) * 2.0 ** -22
                bound[i, h] = size_of * (2 * e + 2.0 ** -9 + (0 if exact else 2.0 ** -11) + len(at) * 2.0 ** -24) \
                    + len(at) * 2.0 ** -31 * np.abs(vv).max(0)
    return bound
