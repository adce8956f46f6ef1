"""Backward pass: one workspace, sized for the largest call, serves smaller ones between its uses."""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from plain_backward import check
from test_gpu_backward import SCALE, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("large,small", [(([200], [9800]), ([190], [9590])), (([130, 40], [9000, 900]), ([129], [9599])),
                                         (([1300], [1300]), ([64] * 20, [64] * 20))], ids=["9800", "two", "many"])
def test_a_kept_workspace(cuda_device, large, small):
    """9,728 keys and more keep RoPE sums of eight heads together, fewer of two."""
    batch = max(len(large[0]), len(small[0]))
    ws = binding.alloc_workspace_prefill_backward(batch, sum(large[0]), sum(large[1]))
    a, b = make(*large, seed=1), make(*small, seed=2)
    first = run(a, workspace=ws)
    check(run(b, workspace=ws), b, True, SCALE)
    for x, y in zip(run(a, workspace=ws), first):
        assert torch.equal(x, y)
    check(first, a, True, SCALE)
    assert binding.mla_get_status(ws) == 0
