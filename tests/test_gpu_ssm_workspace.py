"""The workspace that a prepared gdn_ssm_prefill takes by itself belongs to the
stream of each launch: nothing else is given its memory before the launch has
run, whichever stream prepared the call and however long the call object lives."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from gated_deltanet_linear_sm_gb300 import ops
from tests.test_gpu_ssm import Scan, _bits

pytestmark = pytest.mark.gpu

SLEEP = 20_000_000      # cycles, some 10 ms: far longer than the host takes to overwrite memory


def _cut_scan(dev):
    """A prompt that is cut into segments, its results, and the bytes of workspace that takes."""
    s = Scan(dev, [1500], 2, 1, 64, 128, "f32", seed=50)
    need = gdn.ssm_prefill_workspace(ops._ssm_dims(1, s.N, 2, 1, 64, 128, s.pool, s.dt, s.z, s.out), dev)
    assert need > 0
    s.run()
    want = s.out.clone(), s.pool.clone()
    s.out.zero_()
    s.pool[s.write[0]] = 0
    torch.cuda.synchronize()
    return s, want, need


def _overwrite(dev, need):
    """Every block of that size that the current stream may be given (NaN: what reads it shows)."""
    return [torch.empty(need // 4 + k, device=dev).fill_(float("nan")) for k in range(-8, 1)]


def _same(s, want):
    torch.cuda.synchronize()
    assert torch.equal(_bits(s.out), _bits(want[0])) and torch.equal(_bits(s.pool), _bits(want[1]))
    assert int(s.status) == 0


@pytest.mark.parametrize("handle", [False, True])
def test_call_dropped_while_it_runs_on_another_stream(cuda_device, handle):
    s, want, need = _cut_scan(cuda_device)
    side = torch.cuda.Stream()
    args = s.args()                                     # (the caller's own tensors live on)
    call = gdn.prepare_ssm_prefill(*args, status=s.status)
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    call(side.cuda_stream if handle else side)
    del call
    held = _overwrite(cuda_device, need)
    _same(s, want)
    assert len(held) == 9 and len(args) == 13


def test_call_prepared_behind_work_that_still_runs(cuda_device):
    """The preparing stream still writes memory that it has given back: another stream's launch must not get it."""
    s, want, need = _cut_scan(cuda_device)
    side = torch.cuda.Stream()
    args = s.args()
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    held = _overwrite(cuda_device, need)
    del held
    call = gdn.prepare_ssm_prefill(*args, status=s.status)
    call(side)
    _same(s, want)


def test_graphs_of_one_call_outlive_it(cuda_device):
    """Two graphs that captured one prepared call hold a workspace each."""
    s, want, need = _cut_scan(cuda_device)
    args = s.args()
    call = gdn.prepare_ssm_prefill(*args, status=s.status)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            call()
    del call
    held = _overwrite(cuda_device, need)
    for g in graphs:
        s.out.zero_()
        g.replay()
        _same(s, want)
    assert len(held) == 9


def test_given_workspace_is_the_one_that_is_used(cuda_device):
    s, want, need = _cut_scan(cuda_device)
    room = torch.full((need + 32,), 0x5a, dtype=torch.uint8, device=cuda_device)
    s.run(workspace=room[16:16 + need])
    _same(s, want)
    assert (room[:16] == 0x5a).all() and (room[16 + need:] == 0x5a).all() and not (room[16:16 + need] == 0x5a).all()
    with pytest.raises(ValueError, match="expected workspace"):
        s.run(workspace=room[:need - 1])
