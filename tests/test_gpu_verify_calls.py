"""Calls of gdn_verify_drafts beside those of test_gpu_verify.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from gated_deltanet_linear_sm_gb300 import binding
from tests.test_gpu_verify import DT, Batch, _host, _i32

pytestmark = pytest.mark.gpu


def test_one_request_with_tables_of_different_widths(cuda_device):
    """One sequence has no stride between sequences: its drafts and numbers may be of any length from T-1 on."""
    b = Batch(cuda_device, [4], 4, 301, "f32", seed=20)
    b.run()
    b.check()
    want = b.out.clone()
    b.tokens = torch.cat([b.tokens, _i32([[5, 6, 7]], cuda_device)], 1)
    b.accept_u = torch.cat([b.accept_u, torch.zeros(1, 1, device=cuda_device)], 1)
    b.draft = torch.cat([b.draft, b.draft[:, :2]], 1)
    b.run()
    b.check()
    assert torch.equal(b.out, want)
    two = Batch(cuda_device, [4, 4], 4, 301, "f32", seed=21)
    two.tokens = torch.cat([two.tokens, two.tokens], 1)
    with pytest.raises(ValueError, match="same row stride"):
        two.run()
