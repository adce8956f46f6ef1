"""Encoding of cache rows in float64, written from the published formats.

TEST INFRASTRUCTURE ONLY (see the package docstring).

A group of G values (G = 32 for e4m3 rows, 16 for e2m1 rows) shares the scale
2^k, k the smallest integer with max|v| <= M 2^k, M the format's largest
magnitude (448 for OCP E4M3FN, 6 for OCP MX E2M1), k = 0 for a group of
zeros; the codes are v / 2^k rounded to nearest, ties to even.  Readings:
k is kept in [-127, 119] (e4m3) or [-127, 125] (e2m1), where codes saturate,
so that every stored value is finite in bf16; a group that holds an infinity
or a NaN takes the NaN scale byte 255 and zero codes.  The layouts are those
fp8_codec and fp4_codec decode.
"""
from __future__ import annotations

import numpy as np

from .fp8_codec import float64_to_e4m3fn

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TOP = {"fp8": (448.0, 32, 119), "fp4": (6.0, 16, 125)}


def float64_to_e2m1(x: np.ndarray) -> np.ndarray:
    """Nearest of the eight magnitudes by distance, ties to the even code."""
    x = np.asarray(x, dtype=np.float64)
    d = np.abs(np.abs(x)[..., None] - E2M1)
    best = d.min(-1, keepdims=True)
    tied = d == best                      # one or two neighbouring codes
    low = tied.argmax(-1)
    two = tied.sum(-1) == 2
    code = np.where(two & (low % 2 == 1), low + 1, low)
    return (code + 8 * np.signbit(x)).astype(np.uint8)


def encode_groups(x: np.ndarray, kind: str):
    """[n, m] float64 -> (codes [n, m], scale bytes [n, m / G])."""
    top, group, k_hi = TOP[kind]
    g = np.asarray(x, dtype=np.float64).reshape(x.shape[0], -1, group)
    finite = np.isfinite(g).all(-1)
    g = np.where(finite[..., None], g, 0.0)
    amax = np.abs(g).max(-1)
    with np.errstate(divide="ignore"):
        k = np.ceil(np.log2(amax / top))
    k = np.where(amax == 0, 0, k)
    # log2 may round across an integer: settle k by its definition
    k = np.where(amax > top * np.exp2(k), k + 1, k)
    k = np.where((amax > 0) & (amax <= top * np.exp2(k - 1)), k - 1, k)
    k = np.clip(k, -127, k_hi).astype(np.int64)
    scaled = np.clip(g / np.exp2(k.astype(np.float64))[..., None], -top, top)
    codes = float64_to_e4m3fn(scaled) if kind == "fp8" else float64_to_e2m1(scaled)
    codes = np.where(finite[..., None], codes, 0).astype(np.uint8)
    return codes.reshape(x.shape), np.where(finite, k + 127, 255).astype(np.uint8)


def encode_rows(c_kv: np.ndarray, k_rope: np.ndarray, fmt: str) -> np.ndarray:
    """c_kv [n, 512], k_rope [n, 64] float64 -> rows of a quantised format
    ("fp8", "fp4", "fp8_v41", "fp4_v41") as uint8."""
    latent = c_kv[:, :448] if fmt.endswith("v41") else c_kv
    codes, scales = encode_groups(np.concatenate([latent, k_rope], -1), fmt[:3])
    if fmt.startswith("fp4"):
        codes = codes[:, 0::2] | (codes[:, 1::2] << 4)
    return np.concatenate([codes, scales], -1)
