"""gdn_ssm_prefill of prompts that are cut into segments.

Which prompts are cut and how is an estimate's choice (152 SMs); the tests that
want one form check by the workspace that they got it."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from gated_deltanet_linear_sm_gb300 import binding, ops
from tests.test_gpu_ssm import MARK, Scan, _bits

pytestmark = pytest.mark.gpu


def _workspace(s):
    """Bytes that the call takes for its segments (0: the prompts are not cut)."""
    return gdn.ssm_prefill_workspace(ops._ssm_dims(len(s.lens), s.N, s.H, s.G, s.P, s.S, s.pool, s.dt, s.z, s.out), s.dev)


def _check(s, before):
    """Scan.check on the GPU, for prompts of tens of thousands of tokens: the recurrence token by token in 64
    bits, with the sums of absolute values that the bounds are relative to."""
    f = torch.float64
    dt = s.dt.to(f) + s.dt_bias.to(f)
    d = torch.nn.functional.softplus(dt, threshold=40.0)
    a = torch.exp(-torch.exp(s.A_log.to(f)) * d)
    x, B, C = s.x.to(f), s.B.to(f), s.C.to(f)
    D = s.D.to(f) if s.D is not None else torch.zeros(s.H, dtype=f, device=s.dev)
    z = s.z.to(f) if s.z is not None else None
    kept, done = list(range(s.pool.shape[0])), torch.zeros(s.N, dtype=torch.bool, device=s.dev)
    for i, n in enumerate(s.lens):
        if n <= 0:
            continue
        S = before[s.read[i]].to(f) if s.read[i] >= 0 else torch.zeros(s.H, s.S, s.P, dtype=f, device=s.dev)
        M = S.abs()
        y, my = (torch.empty(n, s.H, s.P, dtype=f, device=s.dev) for _ in range(2))
        lo = int(s.cu[i])
        for t in range(n):
            r = lo + t
            b, c = (v[r].repeat_interleave(s.H // s.G, 0)[:, :, None] for v in (B, C))
            add = b * (d[r][:, None] * x[r])[:, None, :]
            S = S * a[r][:, None, None] + add
            M = M * a[r][:, None, None] + add.abs()
            y[t], my[t] = (c * S).sum(1), (c.abs() * M).sum(1)
        rows = slice(lo, lo + n)
        y, my = y + D[:, None] * x[rows], my + (D[:, None] * x[rows]).abs()
        if z is not None:
            gate = z[rows] * torch.sigmoid(z[rows])
            y, my = y * gate, my * gate.abs()
        err = (s.out[rows].to(f) - y).abs()
        assert (err <= 2.0 ** -8 * y.abs() + 2.0 ** -15 * my + 2.0 ** -17 * y.abs()).all(), f"sequence {i} outputs"
        done[rows] = True
        if s.write[i] >= 0:
            half = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[s.state]
            tol = half * S.abs() + 2.0 ** -16 * M + (2.0 ** -25 if s.state == "f16" else 0.0)
            assert ((s.pool[s.write[i]].to(f) - S).abs() <= tol).all(), f"sequence {i} state"
            kept.remove(s.write[i])
    assert (s.out[~done] == s.out.new_tensor(MARK)).all()
    assert torch.equal(_bits(s.pool[kept]), _bits(before[kept]))
    assert int(s.status) == 0


@pytest.mark.parametrize("lens,H,G,S,state,chunks,parts,kw", [
    ([2000], 64, 8, 64, "f32", 8, 4, {}),                               # four parts of two chunks
    ([4096], 32, 4, 128, "bf16", 8, 2, {}),                             # two parts of four chunks
    ([8192], 16, 1, 64, "f16", 7, 1, dict(gate=False)),                 # parts of seven chunks
    ([30000], 1, 1, 128, "f32", 6, 1, dict(skip=False)),                # a segment that starts from 40 parts
    ([700, 2100, 96, 1200], 16, 2, 128, "f32", 6, 2, {}),               # long, short and uncut prompts together
    ([1, 7000, 250, 0, 300, 129, 128, 127, 385, 60, 500, 120], 8, 8, 64, "f32", 6, 2, dict(strong=True)),
    ([6000, 1000, 3000], 24, 3, 128, "bf16", 20, 4, dict(packed=False)),
])
def test_every_form_of_the_cut_against_the_definition(cuda_device, lens, H, G, S, state, chunks, parts, kw):
    s = Scan(cuda_device, lens, H, G, 64, S, state, seed=sum(lens), **kw)
    before_last = s.N // (chunks * 128)                                 # segments that are not a sequence's last, at most
    room = before_last * parts + min(before_last, len(lens))
    assert _workspace(s) == room * H * (S * 64 + 1) * 4
    before = s.pool.clone()
    s.run()
    _check(s, before)


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


@pytest.mark.parametrize("cu", [[0, 3000, 2700, 3000, 0, 3000],         # the third one's parts begin at the room's last place
                                [0, 3000, 0, 3000, 0, 3000], [0, 2990, 10, 3000, 20, 2000]])
def test_overlapping_offsets_touch_nothing_outside(cuda_device, cu):
    """Offsets that go back (against the caller contract) claim more rows than there are: a flag, and whatever is
    computed stays inside the workspace, the rows, the heads and the slots, and comes from what was written."""
    s = Scan(cuda_device, [3000], 2, 1, 64, 64, "f32", seed=61)
    n = 5
    cu = torch.tensor(cu, dtype=torch.int32, device=s.dev)
    slots = torch.arange(2, 2 + n, dtype=torch.int32, device=s.dev)
    wide = torch.full((s.N + 8, 4, 64), MARK, dtype=torch.bfloat16, device=s.dev)
    pool = torch.full((n + 4, 2, 64, 64), 0.25, dtype=s.pool.dtype, device=s.dev)
    need = gdn.ssm_prefill_workspace(ops._ssm_dims(n, s.N, 2, 1, 64, 64, pool, s.dt, s.z, s.out), s.dev)
    assert need == 28 * 2 * (64 * 64 + 1) * 4                           # 23 parts and 5 initial states
    room = torch.full((need + 8192,), 0xff, dtype=torch.uint8, device=s.dev)     # (NaN)
    inside = torch.zeros(wide.shape, dtype=torch.bool, device=s.dev)
    inside[4:4 + s.N, 1:3] = True
    mark = wide.new_tensor(MARK)
    for _ in range(4):
        room.fill_(0xff)
        s.status.zero_()
        gdn.gdn_ssm_prefill(s.x, s.B, s.C, s.dt, s.z, s.A_log, s.dt_bias, s.D, pool, torch.full_like(slots, -1), slots, cu,
                            wide[4:4 + s.N, 1:3], workspace=room[4096:4096 + need], status=s.status)
        torch.cuda.synchronize()
        assert int(s.status) == binding.GDN_FLAG_TOKEN_ROW
        assert (room[:4096] == 0xff).all() and (room[4096 + need:] == 0xff).all()
        assert torch.isfinite(room[4096:4096 + need].view(torch.float32)[:2 * 64 * 64]).all()     # the first initial states
        assert (wide[~inside] == mark).all() and torch.isfinite(wide.float()).all()
        assert (wide[inside] != mark).any()
        assert (pool[[0, 1, n + 2, n + 3]] == 0.25).all() and torch.isfinite(pool).all()
