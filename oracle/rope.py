"""Rotary positions in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Pair i of a 64-value vector, (2i, 2i+1) when interleaved and (i, i+32)
otherwise, is turned by position * inv_freq[i] ("DeepSeek R1 Architecture &
Deployment Guide", section 1.1: k_R = RoPE(W^KR h)).  Readings: the guide gives
neither layout nor base; 10000 is the usual base.  The scaling for long
contexts is YaRN's: pairs that turn beta_fast times or more over the original
length keep their frequency, pairs that turn fewer than beta_slow times have it
divided by the factor, a ramp in the pair's number joins them.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(base=10000.0, factor=1.0, original=4096, beta_fast=32.0, beta_slow=1.0, dim=64):
    f = [base ** (-2.0 * i / dim) for i in range(dim // 2)]

    def pair(turns):
        # base^(-2 i / dim) original = 2 pi turns, solved for i
        return dim * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))

    low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), dim - 1)
    out = []
    for i, x in enumerate(f):
        ramp = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        out.append(x / factor * ramp + x * (1 - ramp))
    return out


def rotate(x, positions, inv_freq, interleaved, scale=1.0, inverse=False):
    """x [rows, ..., 64] float64, positions [rows] -> the rotated vectors."""
    angle = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq)
    if inverse:
        angle = -angle
    angle = angle.reshape((x.shape[0],) + (1,) * (x.ndim - 2) + (32,))
    c, s = scale * np.cos(angle), scale * np.sin(angle)
    out = np.empty(x.shape)
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    with np.errstate(invalid="ignore"):
        out[..., first] = x[..., first] * c - x[..., second] * s
        out[..., second] = x[..., first] * s + x[..., second] * c
    return out
