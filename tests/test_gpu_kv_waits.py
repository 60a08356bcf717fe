"""gdn_attn_decode with bounds on its waits (gdn_set_wait_limit) from one poll to
more than any wait takes: wherever a wait runs out first, the call ends with
nothing of its own left in flight (no GDN_FLAG_DRAIN), says so, and the next call
is right; a call whose waits all end is right itself."""
from __future__ import annotations

import pytest
import torch

from gated_deltanet_linear_sm_gb300 import binding
from tests.test_gpu_kv import SENTINEL, Case

pytestmark = pytest.mark.gpu


def _sweep(dev, kind, D, window):
    # (72 rows of a cache head: units of 64 and of 8; sequences of one tile and of many, most with an edge tile)
    c = Case(dev, [3000, 500, 77, 0, 1300], [4, 1, 2, 1, 3], 36, 2, D, kind, page=64, seed=D)
    seen = set()
    for limit in (1, 2, 4, 8, 16, 32, 64, 128, 256, 512, 1024, 4096, 1 << 20):
        for _ in range(3):
            c.status.zero_()
            c.out.view(torch.int16).fill_(SENTINEL)
            binding.set_wait_limit(limit)
            try:
                c.run(window=window)
            finally:
                binding.set_wait_limit(0)
            status = int(c.status)
            assert status in (0, binding.GDN_FLAG_TIMEOUT)
            seen.add(status)
            if status == 0:
                c.check(window=window)
    assert seen == {0, binding.GDN_FLAG_TIMEOUT}
    c.status.zero_()
    c.out.view(torch.int16).fill_(SENTINEL)
    c.run(window=window)
    assert int(c.status) == 0
    c.check(window=window)


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_wait_that_runs_out_anywhere(cuda_device, kind, D):
    _sweep(cuda_device, kind, D, 0)


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("D,window", [(192, 0), (256, 0), (256, 100)])
def test_a_wait_that_runs_out_between_the_blocks_of_a_head_dim(cuda_device, kind, D, window):
    """Head dims of two blocks: the values of a tile at a sequence's end (with a window: of every tile) are two loads on one barrier."""
    _sweep(cuda_device, kind, D, window)
