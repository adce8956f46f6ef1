"""The size of the backward pass's workspace, which programs allocate for their largest call and keep."""
import random

import pytest

from mla_latent_kv_05_gb300 import _build, binding


@pytest.fixture(scope="module")
def size():
    _build.build()
    binding.load()
    return binding.mla_workspace_size_prefill_backward


# on both sides of the key tiles from which eight heads' RoPE sums are kept together (75 and 76, with 0, 1, 8 sequences)
EDGES = [(1, 4096, 5000), (1, 4096, 9599), (1, 4096, 9600), (1, 4096, 16384), (0, 10, 9727), (0, 10, 9728), (8, 8192, 8700),
         (8, 8192, 8704), (1, 9500, 9500), (1, 9728, 9728), (1, 4323, 7265), (8, 7098, 18990), (75, 75, 75), (76, 76, 76),
         (1, 1, 38400), (1, 1, 38912), (1, 1, 39000)]


def test_a_workspace_for_more_serves_less(size):
    for a in EDGES:
        for b in EDGES:
            if all(x <= y for x, y in zip(a, b)):
                assert size(*a) <= size(*b), (a, b)


@pytest.mark.parametrize("seed", range(4))
def test_sizes_grow_in_every_count(size, seed):
    r = random.Random(seed)
    for _ in range(5000):
        large = [round(2 ** r.uniform(0, top)) for top in (10, 16, 17)]
        small = [x if r.random() < 0.4 else r.randint(x // 2, x) for x in large]
        assert size(*small) <= size(*large), (small, large)


@pytest.mark.parametrize("batch", [0, 1, 7, 64])
def test_sizes_never_fall_from_one_key_to_the_next(size, batch):
    for nq in (0, 1, 300, 4096):
        last = 0
        for nk in range(8000, 10200):
            n = size(batch, nq, nk)
            assert n >= last, (batch, nq, nk)
            last = n


TILE = 128 * 2 * 128 * 128   # bytes of a tile of scores' gradients, all heads


def tiles(nq, nk):
    return sum(-(-q // 128) * -(-k // 128) for q, k in zip(nq, nk))


# what the gradients of scores may take beyond what these lengths need: the counts do not tell the lengths
@pytest.mark.parametrize("nq,nk,most", [([100] * 16, [100] * 16, 200), ([33, 7, 1, 20, 5], [33, 7, 1, 20, 5], 5), ([1] * 64, [500] * 64, 256),
                                        ([777] * 3, [777] * 3, 384), ([4096], [4096], 1024)],
                         ids=["16 x 100", "short", "64 queries", "777", "4096"])
def test_room_for_scores_is_near_what_the_counts_can_need(size, nq, nk, most):
    n = size(len(nq), sum(nq), sum(nk))
    # the rest: fp32 sums of the RoPE part (16 KiB a key), statistics (128 KiB a tile of queries), lists
    rest = 16384 * sum(nk) + 131072 * (sum(nq) // 128 + len(nq)) + 65536
    assert tiles(nq, nk) * TILE <= n <= most * TILE + rest


@pytest.mark.parametrize("seed", range(4))
def test_room_for_scores_is_enough(size, seed):
    r = random.Random(seed)

    def lengths(n, top):
        return [r.choice((0, 1, 127, 128, 129, round(2 ** r.uniform(0, top)))) for _ in range(n)]

    for _ in range(3000):
        n = round(2 ** r.uniform(0, 7))
        top = r.uniform(1, 12)
        nq, nk = lengths(n, top), lengths(n, top)
        if r.random() < 0.3:
            nk = nq
        rest = size(n, sum(nq), 0) + size(0, 0, sum(nk))   # no scores at all (each has a header of under 4 KiB)
        assert size(n, sum(nq), sum(nk)) >= min(tiles(nq, nk), 1024) * TILE + rest - 4096 - 16 * n, (nq, nk)
