"""Layer norm, rotary positions and the expert permutation in float64 NumPy: each formula written out.

Inputs are float64 arrays of the very values the library reads (a bf16 or FP32 tensor converted exactly).  Each
function returns the exact results and, beside each floating result, `mag`: per element the sum of the magnitudes that
its FP32 evaluation rounds, so that a tolerance is a number of units of 2^-24 of it.
"""
from __future__ import annotations

import math

import numpy as np


def layer_norm(x, gain=None, bias=None, gain_offset=0.0, eps=1e-6):
    """(y, mag): mag has the centred element's own size and the size of the elements whose mean was taken off."""
    w = 1.0 if gain is None else gain + gain_offset
    m = x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - m) * r * w
    mag = np.abs(y) + np.abs(x).mean(-1, keepdims=True) * r * np.abs(w)
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    return y, mag


def layer_norm_bwd(x, dy, gain=None, gain_offset=0.0, eps=1e-6):
    """((dx, mag), (dgain, mag), (dbias, mag))."""
    w = 1.0 if gain is None else gain + gain_offset
    m = x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    n, g = (x - m) * r, dy * w
    gn = (g * n).mean(-1, keepdims=True)
    dx = r * (g - g.mean(-1, keepdims=True) - n * gn)
    off = np.abs(x).mean(-1, keepdims=True) * r  # what the mean's rounding is a part of, in units of n
    gm, gnm = np.abs(g).mean(-1, keepdims=True), np.abs(g * n).mean(-1, keepdims=True)
    mag = r * (np.abs(g) + gm + (np.abs(n) + off) * (gnm + off * gm))
    dgain = (dy * n).sum(0)
    return (dx, mag), (dgain, (np.abs(dy) * (np.abs(n) + off)).sum(0)), (dy.sum(0), np.abs(dy).sum(0))


def rope_positions(tokens, seqlen=None, cu_seqlens=None):
    """Position of each token: modulo seqlen, or from the start of its document."""
    t = np.arange(tokens)
    if cu_seqlens is None:
        return t % seqlen
    cu = np.asarray(cu_seqlens, dtype=np.int64)
    return t - cu[np.searchsorted(cu, t, side="right") - 1]


def rope(x, positions, inv_freq, pairing, scale=1.0, backward=False):
    """(y, mag) of x [tokens, heads, d]; angles in extended precision (64 bits of mantissa and a reduction by them)."""
    angle = np.asarray(positions, dtype=np.longdouble)[:, None] * np.asarray(inv_freq, dtype=np.longdouble)
    c = (scale * np.cos(angle)).astype(np.float64)[:, None, :]
    s = (scale * np.sin(angle)).astype(np.float64)[:, None, :] * (-1.0 if backward else 1.0)
    n = len(inv_freq)
    i = np.arange(n)
    first, second = (i, i + n) if pairing == "half" else (2 * i, 2 * i + 1)
    a, b = x[..., first], x[..., second]
    y, mag = x.copy(), np.zeros_like(x)  # what is not rotated is copied
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    mag[..., first] = mag[..., second] = abs(scale) * (np.abs(a) + np.abs(b))
    return y, mag


def rope_frequencies(rotary_dim, base, scaling="none", factor=1.0, low=1.0, high=4.0, original_context=0.0):
    rd = float(rotary_dim)
    if scaling == "base" and rotary_dim > 2:
        base = base * factor ** (rd / (rd - 2))
    f = [base ** (-2 * i / rd) for i in range(rotary_dim // 2)]
    if scaling == "linear":
        return np.array([v / factor for v in f])
    if scaling in ("bands", "ramp"):
        out = []
        at = lambda turns: rd * math.log(original_context / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        for i, v in enumerate(f):
            if scaling == "bands":
                k = (original_context / (2 * math.pi / v) - low) / (high - low)
            else:
                i0, i1 = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rotary_dim - 1)
                k = 1 - (i - i0) / max(i1 - i0, 0.001)
            k = min(max(k, 0.0), 1.0)
            out.append((1 - k) * v / factor + k * v)
        return np.array(out)
    return np.array(f)


def expert_sort(ids, num_experts):
    """(group_offsets, row_of_slot, slot_of_row) of integer ids [tokens, top_k]."""
    flat = [int(e) for e in np.asarray(ids).reshape(-1)]
    slots_of = [[s for s, e in enumerate(flat) if e == expert] for expert in range(num_experts)] if len(flat) < 2000 else None
    if slots_of is None:
        slots_of = [[] for _ in range(num_experts)]
        for s, e in enumerate(flat):
            if 0 <= e < num_experts:
                slots_of[e].append(s)
    slot_of_row = np.full(len(flat), -1, dtype=np.int64)
    row_of_slot = np.full(len(flat), -1, dtype=np.int64)
    offsets, row = [0], 0
    for group in slots_of:
        for s in group:
            slot_of_row[row], row_of_slot[s] = s, row
            row += 1
        offsets.append(row)
    return np.array(offsets), row_of_slot.reshape(np.asarray(ids).shape), slot_of_row


def expert_combine(rows, row_of_slot, weights=None):
    """(y, mag): each token's weighted sum of its rows; a slot whose row is not among them adds nothing."""
    tokens, top_k = row_of_slot.shape
    y = np.zeros((tokens, rows.shape[1]))
    mag = np.zeros_like(y)
    for t in range(tokens):
        for j in range(top_k):
            r = row_of_slot[t, j]
            if 0 <= r < rows.shape[0]:
                term = rows[r] * (1.0 if weights is None else weights[t, j])
                y[t] += term
                mag[t] += np.abs(term)
    return y, mag


def expert_combine_bwd(rows, dy, row_of_slot, weights=None):
    """(drows, mag) with NaN in the rows that no slot names, and (dweights, mag)."""
    drows = np.full(rows.shape, np.nan)
    dw = np.zeros(row_of_slot.shape)
    dmag = np.zeros(row_of_slot.shape)
    for t in range(row_of_slot.shape[0]):
        for j in range(row_of_slot.shape[1]):
            r = row_of_slot[t, j]
            if 0 <= r < rows.shape[0]:
                drows[r] = dy[t] * (1.0 if weights is None else weights[t, j])
                dw[t, j], dmag[t, j] = (dy[t] * rows[r]).sum(), np.abs(dy[t] * rows[r]).sum()
    return (drows, np.abs(drows)), (dw, dmag)
