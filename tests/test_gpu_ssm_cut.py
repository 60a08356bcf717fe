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


def test_decays_of_long_parts_are_added_exactly(cuda_device):
    """Parts of 220 chunks whose decays are all alike, such that an FP32 sum of their logarithms rounds the same
    way again and again (by 4e-5 to 6e-5 a part, four parts): what is left of the initial state, without inputs.

    Relative error: the logarithm of a token in FP32 (softplus, product, rate: 8 roundings), 2^-21 |l|; the last
    segment's 144 chunks, each a factor 2^l within 2^-22 and two roundings; five parts' exp2f (two steps each)
    and their logarithms up to 32, rounded once (2^-20)."""
    H, T, dev = 64, 131072, cuda_device
    level = torch.tensor([-7.40625, -7.5, -7.375, -8.0]).bfloat16().repeat(H // 4)
    x = torch.zeros(T, H, 64, dtype=torch.bfloat16, device=dev)
    B = torch.randn(T, 1, 64, generator=torch.Generator(device=dev).manual_seed(1), device=dev).bfloat16()
    dt = level.to(dev).expand(T, H).contiguous()
    zero = torch.zeros(H, dtype=torch.bfloat16, device=dev)
    pool = torch.rand(2, H, 64, 64, generator=torch.Generator(device=dev).manual_seed(2), device=dev) + 0.5
    start = pool[0].double()
    out = torch.empty_like(x)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    d = ops._ssm_dims(1, T, H, 1, 64, 64, pool, dt, None, out)
    assert gdn.ssm_prefill_workspace(d, dev) == 5 * H * (64 * 64 + 1) * 4     # two segments of two parts, and the start
    i32 = dict(dtype=torch.int32, device=dev)
    gdn.gdn_ssm_prefill(x, B, B, dt, None, torch.zeros(H, device=dev), zero, None, pool, torch.tensor([0], **i32),
                        torch.tensor([1], **i32), torch.tensor([0, T], **i32), out, status=status)
    assert int(status) == 0
    l = T * torch.log1p(torch.exp(level.double())).to(dev)
    want = start * torch.exp(-l)[:, None, None]
    bound = l * 2.0 ** -21 + 144 * (2.0 ** -22 + 2 * 2.0 ** -24) + 5 * (2 * 2.0 ** -23 + 2.0 ** -20)
    err = ((pool[1].double() - want).abs() / want).amax((1, 2))
    assert (err <= bound).all(), (err.max(), bound.max())
