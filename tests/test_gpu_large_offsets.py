"""Rows and slots that lie more than 2^31 elements into their tensors: the bits
of the same call on compact tensors.  (Up to some 40 GB of device memory.)"""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from tests.test_gpu_ssm import Conv, Scan, Step, _bits, _i32
from tests.test_gpu_verify import Batch

pytestmark = pytest.mark.gpu

FAR = 2 ** 31


def _spread(t, stride):
    """The rows of t `stride` elements apart, so that the last of them are beyond 2^31 elements."""
    flat = torch.zeros((t.shape[0] - 1) * stride + t[0].numel(), dtype=t.dtype, device=t.device)
    wide = flat.as_strided((t.shape[0], *t.shape[1:]), (stride, *t.stride()[1:]))
    wide.copy_(t)
    assert (t.shape[0] - 1) * stride > FAR
    return wide


def test_convolution(cuda_device):
    a = Conv(cuda_device, [3, 700, 1, 397], 264, 4, seed=80)
    b = Conv(cuda_device, [3, 700, 1, 397], 264, 4, seed=80)
    b.x, b.y = _spread(a.x, 2_000_000), _spread(a.y, 2_000_000)
    # slots far into their pool
    b.pool = torch.zeros(FAR // (6 * 264) + 20, 6, 264, dtype=torch.bfloat16, device=cuda_device)
    base = b.pool.shape[0] - a.slots
    b.pool[base:] = a.pool
    b.conv_in, b.conv_out = ([k + base if k >= 0 else k for k in v] for v in (a.conv_in, a.conv_out))
    before = a.pool.clone()
    a.run()
    a.check(before)
    b.run()
    assert torch.equal(_bits(a.y), _bits(b.y)) and torch.equal(_bits(a.pool), _bits(b.pool[base:]))
    assert int(b.status) == 0


@pytest.mark.parametrize("lens", [[130, 300, 70], [1500, 40]])
def test_scan(cuda_device, lens):
    """Whole, and cut into segments."""
    a = Scan(cuda_device, lens, 2, 1, 64, 128, "f32", seed=81, packed=False)
    b = Scan(cuda_device, lens, 2, 1, 64, 128, "f32", seed=81, packed=False)
    stride = 2 ** 31 // (a.N - 30) // 8 * 8
    for k in ("x", "B", "C", "z", "dt", "out"):
        setattr(b, k, _spread(getattr(a, k), stride))
    b.pool = torch.zeros(FAR // (2 * 128 * 64) + 20, 2, 128, 64, device=cuda_device)
    base = b.pool.shape[0] - a.pool.shape[0]
    b.pool[base:] = a.pool
    b.read, b.write = ([k + base if k >= 0 else k for k in v] for v in (a.read, a.write))
    before = a.pool.clone()
    a.run()
    a.check(before)
    b.run()
    assert torch.equal(_bits(a.out), _bits(b.out)) and torch.equal(_bits(a.pool), _bits(b.pool[base:]))
    assert int(b.status) == 0


@pytest.mark.parametrize("state", ["f32", "bf16"])
def test_step(cuda_device, state):
    a = Step(cuda_device, [3, 1, 4, 2], 4, 2, 1, 64, 64, state, acc=[1, 4, 2, 3], seed=82)
    b = Step(cuda_device, [3, 1, 4, 2], 4, 2, 1, 64, 64, state, acc=[1, 4, 2, 3], seed=82)
    stride = 2 ** 31 // (a.N - 3) // 8 * 8
    for k in ("xbc", "z", "dt", "out"):
        setattr(b, k, _spread(getattr(a, k), stride))
    b.pool = torch.zeros(FAR // (2 * 64 * 64) + 40, 2, 64, 64, dtype=a.pool.dtype, device=cuda_device)
    base = b.pool.shape[0] - a.pool.shape[0]
    b.pool[base:] = a.pool
    b.idx = a.idx + base
    rows, D = a.conv_pool.shape[1:]
    b.conv_pool = torch.zeros(FAR // (rows * D) + 20, rows, D, dtype=torch.bfloat16, device=cuda_device)
    cbase = b.conv_pool.shape[0] - a.conv_pool.shape[0]
    b.conv_pool[cbase:] = a.conv_pool
    b.conv_in, b.conv_out = ([k + cbase if k >= 0 else k for k in v] for v in (a.conv_in, a.conv_out))
    a.go()
    b.run()
    assert int(b.status) == 0
    assert torch.equal(_bits(a.out), _bits(b.out)) and torch.equal(_bits(a.pool), _bits(b.pool[base:]))
    assert torch.equal(_bits(a.conv_pool), _bits(b.conv_pool[cbase:]))


@pytest.mark.parametrize("draft", [True, False])
def test_verification(cuda_device, draft):
    a = Batch(cuda_device, [3, 4, 1], 4, 5003, "bf16", draft=draft, seed=83)
    a.run()
    a.check()
    out, acc = a.out.clone(), a.acc.clone()
    a.out.fill_(-7)
    a.acc.fill_(-7)
    a.target = _spread(a.target, 2 ** 31 // 6 + 1)
    if draft:
        a.draft = _spread(a.draft, 2 ** 30 + 3)
    a.run()
    torch.cuda.synchronize()
    assert torch.equal(a.out, out) and torch.equal(a.acc, acc) and int(a.status) == 0


def test_tables(cuda_device):
    """A slot table of more than 2^31 entries."""
    S, R, B = 60000, 36000, 5
    dev = cuda_device
    slots = torch.zeros(R, S, dtype=torch.int32, device=dev)
    assert slots.numel() > FAR
    want = torch.randint(0, 2 ** 31 - 1, (B, S), dtype=torch.int32, device=dev)
    request = [R - 1, 3, R - 2, 0, R - 5]
    slots[_i32(request, dev).long()] = want
    accepted = torch.zeros(R, dtype=torch.int32, device=dev)
    accepted[_i32(request, dev).long()] = _i32([1, 2, 3, 4, 5], dev)
    cu, acc = (torch.empty(n, dtype=torch.int32, device=dev) for n in (B + 1, B))
    indx, idx = torch.empty(10, dtype=torch.int32, device=dev), torch.empty(B, S, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    gdn.gdn_step_tables(_i32([1, 2, 3, 0, 4], dev), slots, cu, indx, idx, acc, accepted=accepted, request=_i32(request, dev),
                        status=status)
    assert torch.equal(idx, want) and acc.tolist() == [1, 2, 3, 4, 5] and cu.tolist() == [0, 1, 3, 6, 6, 10]
    assert indx.tolist() == list(range(10)) and int(status) == 0
