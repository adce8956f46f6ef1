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


def to_bf16(x):
    """float64 -> the nearest bf16 value, ties to even, in one rounding (normal numbers)."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(np.ldexp(m, 8)), e - 8)


def fp32_bound(x, want, interleaved, scale=1.0):
    """How far bf16 values may be off `want` = rotate(x, ...) that were rotated in fp32 and rounded once.  Cosine and sine
    times the scale are off by 2^-23 of it, the two products and their sum by 2^-24 each of the pair's |a| + |b|: together
    under 2^-21; half a bf16 step is 2^-8 of the value at most."""
    a, b = (np.abs(x[..., 0::2]), np.abs(x[..., 1::2])) if interleaved else (np.abs(x[..., :32]), np.abs(x[..., 32:]))
    pair = np.repeat(a + b, 2, -1) if interleaved else np.concatenate([a + b, a + b], -1)
    fp32 = 2.0 ** -21 * abs(scale) * pair
    return fp32 + 2.0 ** -8 * (np.abs(want) + fp32)
