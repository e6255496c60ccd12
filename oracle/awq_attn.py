"""CPU oracle of attention over the 4-bit cache (include/awq_attn.h): rotary positions and their gradient, the cache's
quantizer, and attention, in numpy float64 from their definitions.

TEST INFRASTRUCTURE, NOT PRODUCT CODE. The GPU library never calls it and shares no code with it.

Readings:
* An axis entry outside [0, n_axes) turns its pair by the angle 0.
* A cache's group is 128 consecutive channels of a head, the last one shorter. Numbers beyond +-65024 are taken as that; a
  group with a NaN or an infinity stands for NaNs, and so does one whose step or offset is not finite.
* A row that sees nothing has zeros and lse = -infinity. A NaN that a row does not see leaves it alone.
"""
from __future__ import annotations

import numpy as np

GROUP = 128
LARGEST = 65024.0


def rope(x, positions, inv_freq, axis, pairs, scale, backward=False):
    """x [n, heads, d]; positions [axes, n]; inv_freq [half]; axis [half] or None."""
    x = np.asarray(x, np.float64)
    half = len(inv_freq)
    y = x.copy()
    for i in range(half):
        at = 0 if axis is None else int(axis[i])
        pos = np.asarray(positions)[at].astype(np.float64) if 0 <= at < len(positions) else np.zeros(x.shape[0])
        angle = pos * np.float64(inv_freq[i])
        c, s = scale * np.cos(angle)[:, None], scale * np.sin(angle)[:, None]
        if backward:
            s = -s
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def quantize(x):
    """(codes uint8 [..., d], step float16 [..., groups], offset float16 [..., groups])."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    codes, steps, offsets = np.zeros(x.shape, np.uint8), [], []
    for lo in range(0, d, GROUP):
        part = x[..., lo:lo + GROUP]
        bad = ~np.isfinite(part).all(-1)
        part = np.where(bad[..., None], 0.0, part).clip(-LARGEST, LARGEST)
        low = part.min(-1)
        step, offset = ((part.max(-1) - low) / 15.0).astype(np.float16), low.astype(np.float16)
        s64 = step.astype(np.float64)[..., None]
        q = np.rint((part - offset.astype(np.float64)[..., None]) / np.where(s64 > 0, s64, 1.0))
        codes[..., lo:lo + GROUP] = np.where((s64 > 0) & ~bad[..., None], q.clip(0, 15), 0).astype(np.uint8)
        steps.append(np.where(bad, np.float16("nan"), step))
        offsets.append(np.where(bad, np.float16("nan"), offset))
    return codes, np.stack(steps, -1).astype(np.float16), np.stack(offsets, -1).astype(np.float16)


def dequantize(codes, step, offset):
    """float64 [..., d] of codes [..., d] with step and offset [..., groups]."""
    s, o = np.asarray(step, np.float64), np.asarray(offset, np.float64)
    bad = ~(np.isfinite(s) & np.isfinite(o))
    s, o = np.where(bad, np.nan, s), np.where(bad, np.nan, o)
    d = codes.shape[-1]
    return np.asarray(codes, np.float64) * np.repeat(s, GROUP, -1)[..., :d] + np.repeat(o, GROUP, -1)[..., :d]


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(b):
    return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)


def cached(codes, params, page, place):
    """float64 [..., n_kv, d] keys and values of places of pages: codes [pages, 2, kv, size, d/2], params
    [pages, 2, kv, groups, size, 2]."""
    out = []
    for which in (0, 1):
        p = np.stack([params[a, which, :, :, b] for a, b in zip(page, place)])
        c = np.stack([codes[a, which, :, b] for a, b in zip(page, place)])
        out.append(dequantize(unpack(c), p[..., 0], p[..., 1]))
    return out


def attention(q, codes, params, table, kv_len, q_offsets, scale, causal, window, out=None, lse=None):
    """(out [n, heads, d], lse [n, heads]); rows of no sequence keep what `out` and `lse` hold (zeros, -infinity)."""
    q = np.asarray(q, np.float64)
    n, heads, d = q.shape
    pages, _, kv, size, _ = codes.shape
    group = heads // kv
    out = np.zeros((n, heads, d)) if out is None else np.array(out, np.float64)
    lse = np.full((n, heads), -np.inf) if lse is None else np.array(lse, np.float64)
    for s in range(len(kv_len)):
        first = min(max(int(q_offsets[s]), 0), n)
        last = min(max(int(q_offsets[s + 1]), first), n)
        m = min(max(int(kv_len[s]), 0), table.shape[1] * size)
        j = np.arange(m)
        page = table[s][j // size].astype(np.int64)
        there = (page >= 0) & (page < pages)
        if m:
            k, v = cached(codes, params, np.where(there, page, 0), j % size)
        for i in range(last - first):
            p = m - (last - first) + i
            seen = there & ((j <= p) if causal else True) & ((j > p - window) if window else True)
            at = np.flatnonzero(seen)
            for h in range(heads):
                if not len(at):
                    out[first + i, h], lse[first + i, h] = 0.0, -np.inf
                    continue
                with np.errstate(invalid="ignore"):
                    x = k[at, h // group] @ q[first + i, h] * scale
                    top = x.max()
                    e = np.exp(x - top)
                    out[first + i, h] = e @ v[at, h // group] / e.sum()
                    lse[first + i, h] = top + np.log(e.sum())
    return out, lse
