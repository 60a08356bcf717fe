"""Calls of the prompt convolution and the state-space layer beside those of test_gpu_ssm.py."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_ssm import Conv, Scan, _bits

pytestmark = pytest.mark.gpu


def test_prompts_without_rows_in_this_chunk_keep_their_slots(cuda_device):
    """A sequence that sits a chunk out, with another slot to write than to read: neither slot changes, and the next
    chunk reads the one that it would have read."""
    c = Conv(cuda_device, [5, 0, 40, 0], 264, 4, seed=70, history=[0, 2, 4, 6])
    c.conv_out = [1, 3, 5, 7]
    before = c.pool.clone()
    c.run()
    c.check(before)
    assert torch.equal(_bits(c.pool[[2, 3, 6, 7]]), _bits(before[[2, 3, 6, 7]])) and int(c.status) == 0
    for lens in ([50, 0, 140, 0], [1500, 0, 0, 900]):                   # whole, and cut into segments
        s = Scan(cuda_device, lens, 2, 1, 64, 64, "f32", seed=71, read=[0, 2, 4, 6])
        s.write = [1, 3, 5, 7]
        before = s.pool.clone()
        s.run()
        s.check(before)
        idle = [k for i, n in enumerate(lens) if n == 0 for k in (2 * i, 2 * i + 1)]
        assert torch.equal(_bits(s.pool[idle]), _bits(before[idle])) and int(s.status) == 0
