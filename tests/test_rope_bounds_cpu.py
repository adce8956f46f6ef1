"""What the rotation's outputs are held to: a rotation in fp32 is within its bound, and not always the append's bits."""
import numpy as np
import pytest
import torch

import __graft_entry__
from oracle import rope


def in_fp32(x, pos, f, interleaved):
    """The rotation with fp32 cosines, sines, products and sums (numpy's own roundings), rounded to bf16."""
    angle = pos[:, None] * np.asarray(f)
    c, s = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    a, b, y = x[:, first].astype(np.float32), x[:, second].astype(np.float32), np.empty(x.shape, dtype=np.float32)
    y[:, first], y[:, second] = a * c - b * s, a * s + b * c
    return torch.from_numpy(y).to(torch.bfloat16).double().numpy()


def vectors(seed, rows):
    return torch.randn((rows, 64), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("interleaved", [True, False])
def test_fp32_is_within_the_bound_and_not_the_exact_bits(interleaved):
    f, differ = rope.frequencies(factor=40.0), 0
    for seed in range(40):
        x, pos = vectors(seed, 90), np.arange(90)
        want = rope.rotate(x, pos, f, interleaved)
        got = in_fp32(x, pos, f, interleaved)
        assert (np.abs(got - want) <= rope.fp32_bound(x, want, interleaved)).all()
        differ += not np.array_equal(got, rope.to_bf16(want))
    assert differ > 0          # a check for equal bits would refuse a right kernel


def test_the_bound_refuses_a_value_that_is_off():
    f, x, pos = rope.frequencies(), vectors(7, 50), np.arange(50)
    want = rope.rotate(x, pos, f, True)
    got = in_fp32(x, pos, f, True)
    big = np.abs(want) > 0.1
    for wrong in (got * (1 + 2.0 ** -6), in_fp32(x, pos + 1, f, True), in_fp32(x, -pos, f, True), x):
        assert not (np.abs(wrong - want) <= rope.fp32_bound(x, want, True))[big].all()


def test_to_bf16_is_the_nearest():
    x = np.concatenate([vectors(3, 20).ravel(), [1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -40, 0.0, -1.5]])
    assert np.array_equal(rope.to_bf16(x[:-5]), x[:-5])
    assert rope.to_bf16(x[-5:]).tolist() == [1.0, 1 + 2.0 ** -6, 1 + 2.0 ** -7, 0.0, -1.5]


def test_the_smoke_check_takes_either_rounding():
    f, near = rope.frequencies(factor=40.0), 0
    for seed in range(40):
        x, pos = vectors(seed, 90), np.arange(90)
        want = rope.rotate(x, pos, f, True)
        t, exact, fp32 = (torch.from_numpy(y) for y in (x, rope.to_bf16(want), in_fp32(x, pos, f, True)))
        __graft_entry__.check_rotation(exact, t, f, exact=True)
        __graft_entry__.check_rotation(exact, t, f)
        __graft_entry__.check_rotation(fp32, t, f)
        if not torch.equal(fp32, exact):
            near += 1
            with pytest.raises(RuntimeError):
                __graft_entry__.check_rotation(fp32, t, f, exact=True)
    assert near > 0
    with pytest.raises(RuntimeError):
        __graft_entry__.check_rotation(t, t, f)
