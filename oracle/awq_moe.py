"""CPU oracle of the 4-bit mixture-of-experts block (include/awq_moe.h): the norms around the block, the
order of the slots by expert, gather and combine, the experts' products, and the gradients, in numpy
float64 from their definitions.

TEST INFRASTRUCTURE, NOT PRODUCT CODE. The GPU library never calls it and shares no code with it.

Readings:
* A slot is t * top_k + j; an id outside [0, n_experts) drops it. Within an expert slots ascend.
* Rows that no slot names keep what they held; a token without kept slots gets zeros.
* The experts' weights are dequantized and rounded to the rows' type as in oracle/awq_w4a16.py.
"""
from __future__ import annotations

import numpy as np

from oracle import awq_w4a16 as Q


# ---------------------------------------------------------------- norms


def block_norm(y, residual, w_pre, w_post, gate, res_scale, eps):
    """(r', h); y, w_pre, w_post, gate may be None (h is None without w_pre)."""
    r = np.asarray(residual, np.float64)
    if y is not None:
        z = np.asarray(y, np.float64)
        if w_post is not None:
            z = z / np.sqrt(np.mean(z * z, 1, keepdims=True) + eps) * w_post
        r = r + res_scale * (z if gate is None else gate * z)
    h = None if w_pre is None else r / np.sqrt(np.mean(r * r, 1, keepdims=True) + eps) * w_pre
    return r, h


def block_norm_backward(y, residual, w_pre, w_post, gate, res_scale, eps, d_res, d_h):
    """dict of d_residual, d_y, d_w_pre, d_w_post, d_gate (those whose input is there)."""
    r, _ = block_norm(y, residual, None, w_post, gate, res_scale, eps)
    D = np.zeros_like(r) if d_res is None else np.asarray(d_res, np.float64)
    out = {}
    if w_pre is not None:
        n2 = np.sqrt(np.mean(r * r, 1, keepdims=True) + eps)
        u2, gh = r / n2, d_h * w_pre
        out["d_w_pre"] = np.sum(d_h * u2, 0)
        D = D + (gh - u2 * np.mean(gh * u2, 1, keepdims=True)) / n2
    out["d_residual"] = D
    if y is None:
        return out
    y = np.asarray(y, np.float64)
    n1 = np.sqrt(np.mean(y * y, 1, keepdims=True) + eps) if w_post is not None else 1.0
    u1 = y / n1
    z = u1 if w_post is None else u1 * w_post
    if gate is not None:
        dg = res_scale * D * z
        out["d_gate"] = dg if np.ndim(gate) == 2 else np.sum(dg, 0)
    dz = res_scale * D * (1.0 if gate is None else gate)
    if w_post is None:
        out["d_y"] = dz
    else:
        out["d_w_post"] = np.sum(dz * u1, 0)
        t = dz * w_post
        out["d_y"] = (t - u1 * np.mean(t * u1, 1, keepdims=True)) / n1
    return out


# ---------------------------------------------------------------- tokens by expert and back


def sort_slots(ids, n_experts):
    """(offsets [n_experts + 1], order [slots], position like ids), int32."""
    flat = np.asarray(ids).reshape(-1)
    order = np.full(flat.size, -1, np.int32)
    position = np.full(flat.size, -1, np.int32)
    offsets = np.zeros(n_experts + 1, np.int32)
    at = 0
    for e in range(n_experts):
        for s in np.flatnonzero(flat == e):
            order[at], position[s] = s, at
            at += 1
        offsets[e + 1] = at
    return offsets, order, position.reshape(np.shape(ids))


def gather(x, position, ids, in_scales, rows):
    rows = np.array(rows, np.float64)
    for t, j in np.argwhere((position >= 0) & (position < rows.shape[0])):
        rows[position[t, j]] = np.asarray(x[t], np.float64) * (1.0 if in_scales is None else in_scales[ids[t, j]])
    return rows


def combine(rows, position, weights):
    """weights [n, k], or [n, k, d] multipliers of every channel."""
    n, k = position.shape
    out = np.zeros((n, rows.shape[1]))
    for t, j in np.argwhere((position >= 0) & (position < rows.shape[0])):
        out[t] += weights[t, j] * np.asarray(rows[position[t, j]], np.float64)
    return out


def gather_backward(d_rows, position, ids, in_scales):
    w = np.ones(position.shape + (1,)) if in_scales is None else np.asarray(in_scales, np.float64)[np.maximum(ids, 0)]
    return combine(d_rows, position, w)


def combine_backward(d_out, rows, position, weights, d_rows):
    d_rows, d_w = np.array(d_rows, np.float64), np.zeros(position.shape)
    for t, j in np.argwhere((position >= 0) & (position < rows.shape[0])):
        d_rows[position[t, j]] = weights[t, j] * np.asarray(d_out[t], np.float64)
        d_w[t, j] = np.dot(np.asarray(d_out[t], np.float64), np.asarray(rows[position[t, j]], np.float64))
    return d_rows, d_w


# ---------------------------------------------------------------- the experts' products


def act_product(g, u, act):
    with np.errstate(over="ignore"):
        return (g / (1.0 + np.exp(-g)) if act == "silu" else np.maximum(g, 0.0)) * u


def grouped(x, weights, offsets, y, act=None, backward=False):
    """weights: per expert the float64 [d_out, d_in] values rounded to the operand type. Rows from
    offsets[-1] on keep y's values."""
    y = np.array(y, np.float64)
    for e, w in enumerate(weights):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        part = np.asarray(x[lo:hi], np.float64) @ (w if backward else w.T)
        if act is not None:
            half = w.shape[0] // 2
            part = act_product(part[:, :half], part[:, half:], act)
        y[lo:hi] = part
    return y


def expert_weights(codes, steps_bits, zeros_u4, operand):
    """Per expert the dequantized [d_out, d_in] matrix, rounded to the operand type (float64 values)."""
    d_in = 2 * codes.shape[2]
    return [Q.dequant_deploy(c, s, z, d_in, operand) for c, s, z in zip(codes, steps_bits, zeros_u4)]
