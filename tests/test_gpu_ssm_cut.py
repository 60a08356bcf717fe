"""gdn_ssm_prefill of prompts that are cut into segments."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from gated_deltanet_linear_sm_gb300 import binding, ops
from tests.test_gpu_ssm import Scan

pytestmark = pytest.mark.gpu


def _workspace(s):
    """Bytes that the call takes for its segments (0: the prompts are not cut)."""
    return gdn.ssm_prefill_workspace(ops._ssm_dims(len(s.lens), s.N, s.H, s.G, s.P, s.S, s.pool, s.dt, s.z, s.out), s.dev)


@pytest.mark.parametrize("what", ["read", "write", "rows"])
def test_bad_data_behind_the_first_32_sequences_is_reported(cuda_device, what):
    """A slot or rows out of range in a late sequence: its flag, and every other sequence as it should be."""
    s = Scan(cuda_device, [1000] * 39 + [400], 1, 1, 64, 64, "f32", seed=60)
    assert _workspace(s) > 0
    before = s.pool.clone()
    if what == "rows":
        bad, flag = 39, binding.GDN_FLAG_TOKEN_ROW
        s.cu[40] = s.N + 1                                              # the last one ends behind the rows
    else:
        bad, flag = 35, binding.GDN_FLAG_SLOT_RANGE
        (s.read if what == "read" else s.write)[bad] = s.pool.shape[0]
    s.run()
    s.check(before, skipped=[bad])
    assert int(s.status) == flag
