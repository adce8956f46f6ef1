"""Frequencies from bases and factors that fp32 does not hold."""
import ctypes

import pytest

from mla_latent_kv_05_gb300 import _build, binding
from oracle import rope


@pytest.mark.parametrize("kw", [dict(base=10000.1), dict(factor=1.3), dict(base=1e6 + 0.3, factor=2.7, original_tokens=32768),
                                dict(factor=4.1, beta_fast=32.7, beta_slow=1.1), dict(factor=4.0, original_tokens=4)])
def test_arguments_are_taken_in_64_bits(kw):
    _build.build()
    binding.load()
    want = rope.frequencies(**{("original" if k == "original_tokens" else k): v for k, v in kw.items()})
    got = binding.mla_rope_frequencies(**kw)
    # a power and a logarithm, each off by a few units of the last place; a base that is first rounded to fp32 is off by
    # up to 2^-25 of it, which turns the second pair by 4e-3 at position 160,000
    assert got == pytest.approx(want, rel=1e-13)
    assert max(abs(x - y) for x, y in zip(got, want)) * 163840 < 1e-8


def test_both_entries_agree_and_refuse():
    lib = binding.load()
    a, b = (ctypes.c_double * 32)(), (ctypes.c_double * 32)()
    four = ctypes.c_double * 4
    assert lib.mla_rope_frequencies(500000.0, 8.0, 8192, 32.0, 1.0, a) == 0
    assert lib.mla_rope_frequencies_f64(four(500000.0, 8.0, 32.0, 1.0), 8192, b) == 0
    assert list(a) == list(b)
    assert lib.mla_rope_frequencies_f64(None, 8192, b) == -1 and lib.mla_rope_frequencies(1e4, 1.0, 4096, 32.0, 1.0, None) == -1
    assert lib.mla_rope_frequencies_f64(four(1e4, 1.0, 32.0, 1.0), 8192, None) == -1
    for bad in ((1.0, 1, 32, 1), (1e4, 0.999999999, 32, 1), (1e4, 1, 1, 1), (1e4, 1, 32, 0), (float("nan"), 1, 32, 1),
                (float("inf"), 1, 32, 1), (1e4, float("inf"), 32, 1), (1e4, 1, float("inf"), 1)):
        assert lib.mla_rope_frequencies_f64(four(*bad), 8192, b) == -1, bad
    assert lib.mla_rope_frequencies_f64(four(1e4, 1, 32, 1), 0, b) == -1
