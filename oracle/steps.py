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
