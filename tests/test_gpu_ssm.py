"""gdn_conv_prefill, gdn_ssm_prefill and gdn_ssm_decode against their
definitions in 64 bits, token by token.

Tolerances, each a bound on what the arithmetic may do:
  bf16 results     half a step, 2^-8 of the value, on top of the FP32 error;
  FP32 arithmetic  an error relative to the sum M of the absolute values of the
                   terms that make an element up.  A term passes through at
                   most: its operands as two bf16 parts (2^-18), a decay with
                   exponent error |l| 2^-21 on a weight e^-|l| (x e^-x <= 0.37,
                   so below 2^-22), FP32 sums of up to 128 terms a chunk on the
                   tensor cores, 8 partial sums of 16 that may truncate
                   (2^-23 each, so 2^-20), and the same again for each product
                   that it passes through (two for an output).  Together below
                   2^-16 M for a state and 2^-15 M for an output; silu adds
                   (5 + 1.2 |z|) 2^-23 of the value, below 2^-17 for |z| < 40.
  16-bit states    half a step more: 2^-8 (bf16), 2^-11 (fp16; 2^-25 absolute
                   among its subnormals).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from gated_deltanet_linear_sm_gb300 import binding, ops
from tests import ops_ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
MARK = -12345.0          # what no result is (exact in bf16 after rounding: compared as bits)


def _i32(v, dev):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)


def _h(t):
    return None if t is None else t.double().cpu().numpy()


def _bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def _close(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.max(err - tol):.3g} above its bound"


# ---- the convolution over prompts ------------------------------------------------


class Conv:
    def __init__(self, dev, lens, D, W, seed=0, bias=True, gap=0, history=None, state_len=None, pad_x=0, pad_y=0, shift=0):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.lens, self.D, self.W = lens, D, W
        self.cu = gap + np.concatenate([[0], np.cumsum(lens)])
        self.N = int(self.cu[-1]) + gap
        wide = torch.full((max(self.N, 1), D + pad_x + shift), float("nan"))
        wide[:, shift:shift + D] = torch.randn(max(self.N, 1), D, generator=g)
        self.x = wide.bfloat16().to(dev)[:self.N, shift:shift + D]
        self.w = (torch.randn(D, W, generator=g) * 0.5).bfloat16().to(dev)
        self.bias = (torch.randn(D, generator=g) * 0.3).bfloat16().to(dev) if bias else None
        self.slots = 2 * B + 3
        self.pool = torch.randn(self.slots, state_len or W + 2, D, generator=g).bfloat16().to(dev)
        self.conv_in = history if history is not None else [2 * i if i % 3 != 1 else -1 for i in range(B)]
        self.conv_out = [2 * i + 1 if i % 4 != 3 else -1 for i in range(B)]
        self.y = torch.full((max(self.N, 1), D + pad_y), MARK, dtype=torch.bfloat16, device=dev)[:self.N, :D]
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.dev = dev

    def run(self, **kw):
        gdn.gdn_conv_prefill(self.x, self.w, self.bias, self.pool, _i32(self.conv_in, self.dev),
                             _i32(self.conv_out, self.dev), _i32(self.cu, self.dev), self.y, status=self.status, **kw)
        torch.cuda.synchronize()

    def check(self, before, skipped=()):
        W = self.W
        x, w, bias, old = _h(self.x), _h(self.w), _h(self.bias), _h(before)
        want_pool = before.clone()
        rows = np.zeros(self.N, bool)
        got = _h(self.y)
        for i, n in enumerate(self.lens):
            if n <= 0 or i in skipped:
                continue
            a = int(self.cu[i])
            past = old[self.conv_in[i], 1:W] if self.conv_in[i] >= 0 else np.zeros((W - 1, self.D))
            ext = np.concatenate([past, x[a:a + n]])
            y, m = ops_ref.conv_rows(ext, w, bias)
            # taps: 5 roundings of the terms; the slope of silu is below 1.1; exp and the division
            tol = 2.0 ** -8 * np.abs(y) + 1.1 * 6 * 2.0 ** -24 * m + 2.0 ** -17 * np.abs(y)
            _close(got[a:a + n], y, tol, f"sequence {i}")
            rows[a:a + n] = True
            if self.conv_out[i] >= 0:
                want_pool[self.conv_out[i], :W] = torch.from_numpy(ext[-W:] if W <= len(ext) else
                                                                   np.concatenate([np.zeros((1, self.D)), ext])).to(want_pool)
        assert torch.equal(_bits(self.pool), _bits(want_pool))
        mark = torch.tensor(MARK, dtype=torch.bfloat16).double().item()
        assert (got[~rows] == mark).all()


@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("D", [8, 132, 1280])
def test_conv_against_definition(cuda_device, W, D):
    """Lengths from 0 and 1 to several runs, history or none, slots written or not; rows of no sequence stay."""
    c = Conv(cuda_device, [1, 0, 2, 3, 4, 5, 70, 130, 1, 9], D, W, seed=D + W, gap=3, bias=W != 2)
    before = c.pool.clone()
    c.run()
    c.check(before)
    assert int(c.status) == 0


@pytest.mark.parametrize("kw", [dict(pad_x=4, pad_y=12), dict(pad_x=8, pad_y=8), dict(shift=4), dict(shift=8, pad_y=8)])
def test_conv_strides_and_alignment(cuda_device, kw):
    c = Conv(cuda_device, [33, 5, 200], 264, 4, seed=4, **kw)
    before = c.pool.clone()
    c.run()
    c.check(before)


@pytest.mark.parametrize("lens", [[1] * 40, [3000, 1, 1], [1, 2, 3] * 30])
def test_conv_run_lengths(cuda_device, lens):
    """Many one-token sequences, and long prompts cut into runs at every offset from their start."""
    c = Conv(cuda_device, lens, 4352, 4, seed=len(lens))
    before = c.pool.clone()
    c.run()
    c.check(before)


@pytest.mark.parametrize("W", [1, 2, 3, 4])
def test_conv_of_many_rows_equals_its_slices(cuda_device, W):
    """Enough rows and channels for 8 channels a thread: the bits of the same call on slices of the channels,
    which are too few for that; and their definition on some channels."""
    lens = [1, 2, 3, 700, 0, 5, 64, 1209, 4, 33]
    D = 6464
    c = Conv(cuda_device, lens, D, W, seed=40 + W, gap=3)
    assert c.N * (D // 8) >= 20 * 512 * torch.cuda.get_device_properties(cuda_device).multi_processor_count
    before = c.pool.clone()
    c.run()
    assert int(c.status) == 0
    for lo in range(0, D, 1616):
        cut = slice(lo, lo + 1616)
        part = Conv(cuda_device, lens, 1616, W, seed=1, gap=3)
        part.x, part.w, part.bias = c.x[:, cut], c.w[cut].contiguous(), c.bias[cut].contiguous()
        part.pool = before[:, :, cut].contiguous()
        old = part.pool.clone()
        part.run()
        if lo == 0:
            part.check(old)
        assert torch.equal(_bits(part.y), _bits(c.y[:, cut])) and torch.equal(_bits(part.pool), _bits(c.pool[:, :, cut]))


@pytest.mark.parametrize("seed", range(8))
def test_conv_of_random_sizes(cuda_device, seed):
    rng = np.random.default_rng(seed)
    n = int(rng.choice([1, 2, 5, 60]))
    lens = rng.integers(0, int(rng.choice([3, 9, 200])), n).tolist()
    lens[0] += 1
    c = Conv(cuda_device, lens, 4 * int(rng.integers(1, 300)), int(rng.integers(1, 5)), seed=seed, bias=bool(rng.random() < 0.6),
             gap=int(rng.integers(0, 5)), pad_x=4 * int(rng.integers(0, 4)), pad_y=4 * int(rng.integers(0, 4)),
             shift=int(rng.choice([0, 0, 4, 8])))
    before = c.pool.clone()
    c.run()
    c.check(before)
    assert int(c.status) == 0


def test_conv_in_place_and_in_chunks(cuda_device):
    """A prompt in three chunks, its slot updated in place, gives the bits of the whole prompt."""
    D, W = 520, 4
    whole = Conv(cuda_device, [301], D, W, seed=11, history=[-1])
    whole.run()
    pool = whole.pool.clone()
    y = torch.empty_like(whole.y)
    at = 0
    for n in (2, 129, 170):
        cu = _i32([0, n], cuda_device)
        slot = _i32([0], cuda_device)
        gdn.gdn_conv_prefill(whole.x[at:at + n], whole.w, whole.bias, pool, _i32([-1], cuda_device) if at == 0 else slot, slot,
                             cu, y[at:at + n])
        at += n
    assert torch.equal(_bits(y), _bits(whole.y))
    assert torch.equal(_bits(pool[0, :W]), _bits(whole.pool[1, :W]))


def test_conv_bad_data_is_reported_and_skipped(cuda_device):
    c = Conv(cuda_device, [5, 6, 7], 256, 4, seed=12)
    before = c.pool.clone()
    c.conv_in[1] = c.slots
    c.run()
    c.check(before, skipped=[1])
    assert int(c.status) == binding.GDN_FLAG_SLOT_RANGE
    c = Conv(cuda_device, [5, 6, 7], 256, 4, seed=12)
    c.x, c.y, c.N = c.x[:17], c.y[:17], 17                              # the last sequence ends behind the rows
    c.run()
    c.check(before, skipped=[2])
    assert int(c.status) == binding.GDN_FLAG_TOKEN_ROW


def test_conv_of_infinite_and_nan_inputs_stays_in_its_rows(cuda_device):
    c = Conv(cuda_device, [9, 20, 9], 256, 4, seed=13, history=[-1, -1, -1])
    before = c.pool.clone()
    clean = Conv(cuda_device, [9, 20, 9], 256, 4, seed=13, history=[-1, -1, -1])
    clean.run()
    c.x[9 + 19] = float("nan")
    c.x[9 + 10] = float("inf")
    c.run()
    same = [r for r in range(38) if r not in range(19, 23) and r != 28]
    assert torch.equal(_bits(c.y[same]), _bits(clean.y[same]))
    assert not torch.isfinite(c.y[28]).any() and torch.equal(before[0], c.pool[0])


# ---- the state-space layer -----------------------------------------------------


class Layer:
    """Random parameters and rows of a layer; decays from nearly 1 to nearly 0."""

    def __init__(self, dev, N, H, G, P, S, state, gate=True, skip=True, seed=0, slots=8, strong=False):
        g = torch.Generator().manual_seed(seed)
        self.dev, self.N, self.H, self.G, self.P, self.S, self.state = dev, N, H, G, P, S, state
        rate = torch.exp(torch.rand(H, generator=g) * 4.6 - 6.9)
        self.dt = (torch.randn(N, H, generator=g) * (3.0 if strong else 0.6)).bfloat16().to(dev)
        self.dt_bias = (torch.log(torch.expm1(rate)) if not strong else torch.randn(H, generator=g) * 3).bfloat16().to(dev)
        self.A_log = torch.log(torch.rand(H, generator=g) * 15 + 1).to(dev)
        self.D = (torch.randn(H, generator=g) + 1).to(dev) if skip else None
        self.z = (torch.randn(N, H, P, generator=g) * 2).bfloat16().to(dev) if gate else None
        self.out = torch.full((N, H, P), MARK, dtype=torch.bfloat16, device=dev)
        self.pool = (torch.randn(slots, H, S, P, generator=g) * 0.3).to(DT[state]).to(dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.gen = g

    def gates(self):
        d = ops_ref.softplus(_h(self.dt) + _h(self.dt_bias))
        return d, np.exp(-np.exp(_h(self.A_log)) * d)

    def heads(self, v):
        """[G, S] -> [H, S]"""
        return np.repeat(v, self.H // self.G, axis=0)

    def state_tol(self, S, M):
        return HALF_STEP[self.state] * np.abs(S) + 2.0 ** -16 * M + (2.0 ** -25 if self.state == "f16" else 0.0)

    def out_tol(self, y, my):
        return 2.0 ** -8 * np.abs(y) + 2.0 ** -15 * my + 2.0 ** -17 * np.abs(y)


class Scan(Layer):
    def __init__(self, dev, lens, H, G, P, S, state, gap=0, read=None, packed=True, **kw):
        self.lens = lens
        self.cu = gap + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        n = len(lens)
        super().__init__(dev, int(self.cu[-1]) + gap, H, G, P, S, state, slots=2 * n + 2, **kw)
        row = H * P + 2 * G * S
        x = torch.randn(self.N, row, generator=self.gen)
        self.packed = (x * torch.sigmoid(x)).bfloat16().to(dev)
        self.x = self.packed[:, :H * P].view(self.N, H, P)
        self.B = self.packed[:, H * P:H * P + G * S].view(self.N, G, S)
        self.C = self.packed[:, H * P + G * S:].view(self.N, G, S)
        if not packed:
            self.x, self.B, self.C = (v.contiguous() for v in (self.x, self.B, self.C))
        self.read = read if read is not None else [2 * i if i % 3 != 1 else -1 for i in range(n)]
        self.write = [2 * i + 1 if i % 4 != 3 else -1 for i in range(n)]

    def args(self):
        return (self.x, self.B, self.C, self.dt, self.z, self.A_log, self.dt_bias, self.D, self.pool,
                _i32(self.read, self.dev), _i32(self.write, self.dev), _i32(self.cu, self.dev), self.out)

    def run(self, **kw):
        gdn.gdn_ssm_prefill(*self.args(), status=self.status, **kw)
        torch.cuda.synchronize()

    def check(self, before, skipped=()):
        d, a = self.gates()
        x, B, C, z = _h(self.x), _h(self.B), _h(self.C), _h(self.z)
        D = _h(self.D) if self.D is not None else np.zeros(self.H)
        got, old = _h(self.out), _h(before)
        done = np.zeros(self.N, bool)
        kept = list(range(self.pool.shape[0]))
        for i, n in enumerate(self.lens):
            if n <= 0 or i in skipped:
                continue
            S = old[self.read[i]] if self.read[i] >= 0 else np.zeros((self.H, self.S, self.P))
            M = np.abs(S)
            want, tol = np.empty((n, self.H, self.P)), np.empty((n, self.H, self.P))
            for t in range(n):
                r = int(self.cu[i]) + t
                gate = ops_ref.silu(z[r]) if z is not None else np.ones((self.H, self.P))
                S, M, want[t], my = ops_ref.layer_step(S, M, a[r], d[r], self.heads(B[r]), self.heads(C[r]), x[r], D, gate)
                tol[t] = self.out_tol(want[t], my)
            lo = int(self.cu[i])
            _close(got[lo:lo + n], want, tol, f"sequence {i} outputs")
            done[lo:lo + n] = True
            if self.write[i] >= 0:
                _close(_h(self.pool[self.write[i]]), S, self.state_tol(S, M), f"sequence {i} state")
                kept.remove(self.write[i])
        mark = torch.tensor(MARK, dtype=torch.bfloat16).double().item()
        assert (got[~done] == mark).all()
        assert torch.equal(_bits(self.pool[kept]), _bits(before[kept]))


@pytest.mark.parametrize("state", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("S", [64, 128])
def test_scan_of_ragged_prompts(cuda_device, state, S):
    """Lengths around every tile border, history or none, slots written or not."""
    s = Scan(cuda_device, [1, 0, 7, 127, 128, 129, 64, 300, 2, 33], 2, 1, 64, S, state, gap=5, seed=S)
    before = s.pool.clone()
    s.run()
    s.check(before)
    assert int(s.status) == 0


@pytest.mark.parametrize("H,G,P", [(1, 1, 64), (4, 2, 64), (3, 3, 128), (6, 1, 192), (2, 2, 256), (8, 4, 128)])
def test_scan_head_layouts(cuda_device, H, G, P):
    s = Scan(cuda_device, [150, 40], H, G, P, 128, "f32", seed=H * P)
    before = s.pool.clone()
    s.run()
    s.check(before)


@pytest.mark.parametrize("kw", [dict(gate=False), dict(skip=False), dict(gate=False, skip=False), dict(packed=False),
                                dict(strong=True)])
def test_scan_options(cuda_device, kw):
    """Without the gate, without D, from separate tensors, and with decays from 1 to 0 within a token."""
    s = Scan(cuda_device, [260, 19], 4, 2, 64, 64, "f32", seed=21, **kw)
    before = s.pool.clone()
    s.run()
    s.check(before)


@pytest.mark.parametrize("lens", [[1500], [700, 1, 900, 350]])
def test_scan_of_long_prompts(cuda_device, lens):
    s = Scan(cuda_device, lens, 2, 1, 64, 128, "f32", seed=sum(lens))
    before = s.pool.clone()
    s.run()
    s.check(before)


def test_scan_strided_rows_and_output(cuda_device):
    """z, dt and out inside wider tensors (NaN around them; the rest of out's rows is left alone)."""
    s = Scan(cuda_device, [140, 30], 2, 1, 64, 64, "bf16", seed=5)
    wide = torch.full((s.N, 3, 64), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    wide[:, 1:] = s.z
    s.z = wide[:, 1:]
    dt = torch.full((s.N, 5), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    dt[:, 2:4] = s.dt
    s.dt = dt[:, 2:4]
    out = torch.full((s.N, 4, 64), MARK, dtype=torch.bfloat16, device=cuda_device)
    s.out = out[:, 1:3]
    before = s.pool.clone()
    s.run()
    s.check(before)
    assert (out[:, [0, 3]] == out.new_tensor(MARK)).all()


def test_scan_in_chunks_and_in_place(cuda_device):
    """A prompt in three calls, its FP32 slot updated in place, agrees with the whole one (twice the bound of a call)."""
    s = Scan(cuda_device, [400], 2, 1, 64, 128, "f32", seed=6, read=[-1])
    s.run()
    pool = s.pool.clone()
    out = torch.empty_like(s.out)
    at = 0
    for n in (100, 201, 99):
        r = slice(at, at + n)
        gdn.gdn_ssm_prefill(s.x[r], s.B[r], s.C[r], s.dt[r], s.z[r], s.A_log, s.dt_bias, s.D, pool,
                            _i32([-1 if at == 0 else 0], cuda_device), _i32([0], cuda_device), _i32([0, n], cuda_device), out[r])
        at += n
    whole = Scan(cuda_device, [400], 2, 1, 64, 128, "f32", seed=6, read=[-1])
    before = whole.pool.clone()
    whole.out, whole.pool = out, torch.cat([before[:1], pool[:1], before[2:]])
    whole.check(before)


@pytest.mark.parametrize("state", ["f32", "f16"])
def test_scan_of_cut_prompts_in_place(cuda_device, state):
    """Prompts long enough to be cut into segments, their slots updated in place: the bits of the same prompts
    whose states go to other slots (a segment never reads a slot that the sequence's last one may have written)."""
    lens = [1900, 40, 1300, 700]
    a = Scan(cuda_device, lens, 3, 1, 64, 128, state, seed=18, read=[0, 2, -1, 6])
    b = Scan(cuda_device, lens, 3, 1, 64, 128, state, seed=18, read=[0, 2, -1, 6])
    a.write, b.write = [1, 3, 5, 7], [0, 2, 5, 6]
    d = ops._ssm_dims(4, a.N, 3, 1, 64, 128, a.pool, a.dt, a.z, a.out)
    assert gdn.ssm_prefill_workspace(d, cuda_device) > 0                # they are cut
    before = a.pool.clone()
    a.run()
    a.check(before)
    for _ in range(5):
        b.pool.copy_(before)
        b.run()
        assert torch.equal(_bits(a.out), _bits(b.out))
        for i in range(4):
            assert torch.equal(_bits(a.pool[a.write[i]]), _bits(b.pool[b.write[i]]))


def _random_scan(dev, seed):
    """Sizes from short prompts to ones that are cut, with and without every option."""
    rng = np.random.default_rng(1000 + seed)
    n = int(rng.choice([1, 1, 2, 3, 7, 40]))
    total = int(np.exp(rng.uniform(np.log(20), np.log(2600))))
    lens = rng.multinomial(total, rng.dirichlet(np.ones(n) * float(rng.choice([0.3, 1.0, 20.0])))).tolist()
    G = int(rng.choice([1, 1, 2, 3]))
    H = G * int(rng.choice([1, 2, 4]))
    read = [2 * i if rng.random() < 0.7 else -1 for i in range(n)]
    s = Scan(dev, lens, H, G, 64 * int(rng.choice([1, 1, 2])), int(rng.choice([64, 128])), str(rng.choice(["f32", "bf16", "f16"])),
             gap=int(rng.integers(0, 9)), read=read, packed=bool(rng.random() < 0.5), gate=bool(rng.random() < 0.6),
             skip=bool(rng.random() < 0.6), strong=bool(rng.random() < 0.3), seed=seed)
    s.write = [(r if r >= 0 and rng.random() < 0.5 else 2 * i + 1) if rng.random() < 0.9 else -1 for i, r in enumerate(read)]
    return s


@pytest.mark.parametrize("seed", range(12))
def test_scan_of_random_sizes(cuda_device, seed):
    s = _random_scan(cuda_device, seed)
    before = s.pool.clone()
    s.run()
    s.check(before)
    assert int(s.status) == 0


def test_scan_keeps_infinite_and_nan_rows_to_their_sequence(cuda_device):
    """Rows of NaN and infinity in the neighbouring sequences, and behind the last one, reach nobody else."""
    lens = [130, 70, 129]
    clean = Scan(cuda_device, lens, 2, 1, 64, 64, "f32", seed=8, gap=4)
    dirty = Scan(cuda_device, lens, 2, 1, 64, 64, "f32", seed=8, gap=4)
    clean.run()
    for lo, hi, v in ((0, 4, float("nan")), (134, 204, float("inf")), (333, 337, float("nan"))):
        dirty.packed[lo:hi] = v
        dirty.z[lo:hi] = v
        dirty.dt[lo:hi] = v
    dirty.run()
    rows = [r for r in range(337) if not 134 <= r < 204]
    assert torch.equal(_bits(dirty.out[rows]), _bits(clean.out[rows]))
    for i in (0, 2):
        assert torch.equal(_bits(dirty.pool[dirty.write[i]]), _bits(clean.pool[clean.write[i]]))
    assert not torch.isfinite(dirty.pool[dirty.write[1]].float()).any()


def test_scan_bad_data_is_reported_and_skipped(cuda_device):
    s = Scan(cuda_device, [50, 60, 70], 2, 1, 64, 64, "f32", seed=10)
    before = s.pool.clone()
    s.read[0] = s.pool.shape[0]
    s.run()
    s.check(before, skipped=[0])
    assert int(s.status) == binding.GDN_FLAG_SLOT_RANGE
    s = Scan(cuda_device, [50, 60, 70], 2, 1, 64, 64, "f32", seed=10)
    s.cu[2] = s.N + 1                                                   # the second ends behind the rows; the third is empty
    s.lens = [50, 60, 0]
    s.run()
    s.check(before, skipped=[1])
    assert int(s.status) & binding.GDN_FLAG_TOKEN_ROW


def test_scan_captured_beside_another_and_repeatable(cuda_device):
    """Two captured prefills with their own workspaces, replayed on two streams at once, give the bits of direct calls."""
    a = Scan(cuda_device, [900, 40], 2, 1, 64, 128, "f32", seed=14)
    b = Scan(cuda_device, [700], 4, 2, 64, 64, "bf16", seed=15)
    a.run()
    b.run()
    want = [(s.out.clone(), s.pool.clone()) for s in (a, b)]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    keep = []
    for s, st in zip((a, b), streams):
        call = gdn.prepare_ssm_prefill(*s.args(), status=s.status)
        keep.append(call)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call()
        graphs.append(g)
    for _ in range(3):
        for s in (a, b):
            s.out.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, (out, pool) in zip((a, b), want):
            assert torch.equal(_bits(s.out), _bits(out)) and torch.equal(_bits(s.pool), _bits(pool))
    a.out.zero_()
    torch.cuda.synchronize()
    a.run(stream=streams[0])
    a.out.cpu()
    b.run(stream=streams[1].cuda_stream)
    assert torch.equal(_bits(a.out), _bits(want[0][0])) and torch.equal(_bits(b.pool), _bits(want[1][1]))


@pytest.mark.parametrize("lens", [[700], [260, 90]])
def test_scan_wait_that_runs_out_is_reported(cuda_device, lens):
    """With a bound of one poll the tensor-core waits give up: a status bit and no state written, the GPU
    stays usable, and the next call with the default bound is right."""
    s = Scan(cuda_device, lens, 2, 1, 64, 128, "f32", seed=16)
    before = s.pool.clone()
    binding.set_wait_limit(1)
    try:
        s.run()
    finally:
        binding.set_wait_limit(0)
    assert int(s.status) & binding.GDN_FLAG_TIMEOUT and not int(s.status) & binding.GDN_FLAG_DRAIN
    assert torch.equal(_bits(s.pool), _bits(before))
    s.status.zero_()
    s.run()
    s.check(before)
    assert int(s.status) == 0


def test_scan_of_overlapping_offsets_stays_inside_its_memory(cuda_device):
    """Offsets that go back (against the caller contract) claim more rows than there are: nothing outside the
    rows and slots is touched, and every output row is finite."""
    s = Scan(cuda_device, [3000], 2, 1, 64, 64, "f32", seed=17)
    pool = torch.zeros(12, 2, 64, 64, device=cuda_device)
    n = 9
    cu = _i32([0, 3000, 0, 10, 3000, 0, 20, 3000, 0, 3000], cuda_device)
    gdn.gdn_ssm_prefill(s.x, s.B, s.C, s.dt, s.z, s.A_log, s.dt_bias, s.D, pool, _i32([-1] * n, cuda_device),
                        _i32(list(range(n)), cuda_device), cu, s.out, status=s.status)
    torch.cuda.synchronize()
    assert torch.isfinite(s.out.float()).all() and (pool[9:] == 0).all()


# ---- the step -------------------------------------------------------------------


class Step(Layer):
    def __init__(self, dev, q_lens, T, H, G, P, S, state, W=4, acc=None, gather=False, bias=True, seed=0, **kw):
        self.q, self.T, self.W = q_lens, T, W
        n = len(q_lens)
        rng = np.random.default_rng(seed)
        self.cu = np.concatenate([[0], np.cumsum(q_lens)])
        rows = int(self.cu[-1])
        N = rows + (4 if gather else 0)
        super().__init__(dev, N, H, G, P, S, state, seed=seed, slots=n * T + 3, **kw)
        D = H * P + 2 * G * S
        g = self.gen
        self.xbc = torch.randn(N, D, generator=g).bfloat16().to(dev)
        self.w = (torch.randn(D, W, generator=g) * 0.5).bfloat16().to(dev)
        self.bias = (torch.randn(D, generator=g) * 0.2).bfloat16().to(dev) if bias else None
        self.conv_pool = torch.randn(2 * n + 1, W - 1 + T + 1, D, generator=g).bfloat16().to(dev)
        self.conv_in = [i if i % 3 != 2 else -1 for i in range(n)]
        self.conv_out = [n + i if i % 4 != 1 else -1 for i in range(n)]
        self.idx = rng.permutation(n * T + 3)[:n * T].reshape(n, T)
        self.acc = list(rng.integers(0, T + 1, n)) if acc is None else acc
        self.indx = rng.permutation(N)[:rows] if gather else None

    def run(self, **kw):
        gdn.gdn_ssm_decode(self.xbc, self.w, self.bias, self.conv_pool, _i32(self.conv_in, self.dev),
                           _i32(self.conv_out, self.dev), self.dt, self.z, self.A_log, self.dt_bias, self.D, self.pool,
                           _i32(self.idx, self.dev), _i32(self.acc, self.dev), _i32(self.cu, self.dev), self.out, G=self.G,
                           spec_token_indx=None if self.indx is None else _i32(self.indx, self.dev), status=self.status, **kw)
        torch.cuda.synchronize()

    def check(self, pool0, conv0, skipped=()):
        H, G, P, S_, W = self.H, self.G, self.P, self.S, self.W
        d, a = self.gates()
        D = _h(self.D) if self.D is not None else np.zeros(H)
        x, w, bias, z = _h(self.xbc), _h(self.w), _h(self.bias), _h(self.z)
        got, old = _h(self.out), _h(pool0)
        done = np.zeros(self.N, bool)
        conv_want = conv0.clone()
        kept = set(range(self.pool.shape[0]))
        for i, n in enumerate(self.q):
            back = max(int(self.acc[i]), 1)
            if n <= 0 or i in skipped or self.idx[i][back - 1] < 0:
                continue
            rows = [int(self.indx[k]) if self.indx is not None else int(k) for k in range(self.cu[i], self.cu[i] + n)]
            raw = torch.cat([conv0[self.conv_in[i], back:back + W - 1] if self.conv_in[i] >= 0 else
                             conv0.new_zeros(W - 1, conv0.shape[2]), self.xbc[rows]])
            if self.conv_out[i] >= 0:
                conv_want[self.conv_out[i], :W - 1 + n] = raw
            u, m = ops_ref.conv_rows(_h(raw), w, bias)
            e = 1.1 * 6 * 2.0 ** -24 * m + 2.0 ** -18 * np.abs(u)       # the convolution's own FP32 error
            S = old[self.idx[i][back - 1]]
            M = np.abs(S)
            for t in range(n):
                r = rows[t]
                xs, Bt, Ct = u[t, :H * P].reshape(H, P), u[t, H * P:H * P + G * S_].reshape(G, S_), u[t, H * P + G * S_:].reshape(G, S_)
                ex, eB, eC = e[t, :H * P].reshape(H, P), e[t, H * P:H * P + G * S_].reshape(G, S_), e[t, H * P + G * S_:].reshape(G, S_)
                gate = ops_ref.silu(z[r]) if z is not None else np.ones((H, P))
                S, M, y, my = ops_ref.layer_step(S, M, a[r], d[r], self.heads(Bt), self.heads(Ct), xs, D, gate)
                # errors of B, C and x that reach the state and the output, taken into M and my in units of the bounds
                extra = (self.heads(eB)[:, :, None] * np.abs(d[r][:, None] * xs)[:, None, :]
                         + np.abs(self.heads(Bt))[:, :, None] * (d[r][:, None] * ex)[:, None, :])
                M = M + extra * 2.0 ** 16
                my = (np.einsum("hn,hnp->hp", np.abs(self.heads(Ct)), M) + np.abs(D[:, None] * xs)) * np.abs(gate)
                my = my + (np.einsum("hn,hnp->hp", self.heads(eC), np.abs(S)) + np.abs(D)[:, None] * ex) * np.abs(gate) * 2.0 ** 15
                _close(got[r], y, self.out_tol(y, my), f"sequence {i} token {t}")
                done[r] = True
                slot = int(self.idx[i][t])
                if 0 <= slot < self.pool.shape[0]:
                    _close(_h(self.pool[slot]), S, self.state_tol(S, M), f"sequence {i} state {t}")
                    kept.discard(slot)
        mark = torch.tensor(MARK, dtype=torch.bfloat16).double().item()
        assert (got[~done] == mark).all()
        k = sorted(kept)
        assert torch.equal(_bits(self.pool[k]), _bits(pool0[k]))
        assert torch.equal(_bits(self.conv_pool), _bits(conv_want))

    def go(self, skipped=(), flag=0, **kw):
        pool, conv = self.pool.clone(), self.conv_pool.clone()
        self.run(**kw)
        self.check(pool, conv, skipped)
        assert int(self.status) == flag


@pytest.mark.parametrize("state", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("S", [64, 128])
def test_step_of_ragged_drafts(cuda_device, state, S):
    Step(cuda_device, [8, 1, 3, 0, 5, 8], 8, 4, 2, 64, S, state, seed=S).go()


@pytest.mark.parametrize("H,G,P", [(1, 1, 64), (6, 3, 128), (4, 1, 192), (2, 2, 256)])
def test_step_single_token(cuda_device, H, G, P):
    """The form for single tokens: one slot column, the state updated in place."""
    Step(cuda_device, [1, 1, 1], 1, H, G, P, 128, "bf16", acc=[1, 0, 1], seed=H + P).go()


@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("bias", [True, False])
def test_step_widths(cuda_device, W, bias):
    Step(cuda_device, [3, 4, 1, 2], 4, 2, 1, 64, 64, "f32", W=W, bias=bias, gather=True, seed=W).go()


@pytest.mark.parametrize("kw", [dict(gate=False), dict(skip=False), dict(strong=True)])
def test_step_options(cuda_device, kw):
    Step(cuda_device, [2, 4], 4, 2, 1, 64, 128, "f32", seed=31, **kw).go()


@pytest.mark.parametrize("seed", range(8))
def test_step_of_random_sizes(cuda_device, seed):
    rng = np.random.default_rng(seed)
    n, T = int(rng.choice([1, 3, 9, 40])), int(rng.integers(1, 9))
    q = rng.integers(0, T + 1, n).tolist()
    q[0] = max(q[0], 1)
    G = int(rng.choice([1, 2, 3]))
    s = Step(cuda_device, q, T, G * int(rng.choice([1, 2, 4])), G, 64 * int(rng.choice([1, 1, 2, 3])), int(rng.choice([64, 128])),
             str(rng.choice(["f32", "bf16", "f16"])), W=int(rng.integers(1, 5)), gather=bool(rng.random() < 0.5),
             bias=bool(rng.random() < 0.5), seed=seed, gate=bool(rng.random() < 0.6), skip=bool(rng.random() < 0.6),
             strong=bool(rng.random() < 0.3))
    pool, conv = s.pool.clone(), s.conv_pool.clone()
    s.run()
    s.check(pool, conv)
    assert int(s.status) == 0


def test_step_padded_slots(cuda_device):
    """A sequence whose rewound slot is -1 is padding; a write slot of -1 skips that write."""
    s = Step(cuda_device, [3, 3, 3], 4, 2, 1, 64, 64, "f32", acc=[2, 1, 4], seed=32)
    s.idx[1, 0] = -1
    s.idx[2, 1] = -1
    s.go()


def test_step_bad_data_is_reported_and_skipped(cuda_device):
    def base():
        return Step(cuda_device, [2, 3, 2, 3], 4, 2, 1, 64, 64, "f32", acc=[1, 2, 3, 4], seed=33, gather=True)
    s = base()
    s.acc[1] = 5
    s.go(skipped=[1], flag=binding.GDN_FLAG_ACCEPTED)
    s = base()
    s.go(skipped=[1, 3], flag=binding.GDN_FLAG_QLEN, max_T=2)
    s = base()
    s.idx[2, 2] = s.pool.shape[0]
    s.go(skipped=[2], flag=binding.GDN_FLAG_SLOT_RANGE)
    s = base()
    s.idx[0, 1] = s.pool.shape[0]                                       # a write slot: only that write is skipped
    s.go(flag=binding.GDN_FLAG_SLOT_RANGE)
    s = base()
    s.conv_out[3] = s.conv_pool.shape[0]
    s.go(skipped=[3], flag=binding.GDN_FLAG_SLOT_RANGE)
    s = base()
    s.indx[3] = s.N
    s.go(skipped=[1], flag=binding.GDN_FLAG_TOKEN_ROW)


def test_step_after_prompt_equals_the_longer_prompt(cuda_device):
    """Convolution and scan over a prompt, then four tokens through the step: the rows that the prompt with
    those tokens in it gives (the step does not round its convolution to bf16, so within a bf16 step of the
    rows' terms; the raw conv slots are equal)."""
    H, G, P, S, W, n, k = 2, 1, 64, 64, 4, 150, 4
    s = Step(cuda_device, [k], k, H, G, P, S, "f32", acc=[1], seed=40)
    x = torch.randn(n + k, s.xbc.shape[1], generator=s.gen).bfloat16().to(cuda_device)
    dt = (torch.randn(n + k, H, generator=s.gen) * 0.5).bfloat16().to(cuda_device)
    z = torch.randn(n + k, H, P, generator=s.gen).bfloat16().to(cuda_device)
    conv_pool = torch.zeros(k + 2, W - 1 + k, x.shape[1], dtype=torch.bfloat16, device=cuda_device)
    pool = torch.zeros(k + 2, H, S, P, device=cuda_device)

    def prompt(m, slot):
        y = torch.empty(m, x.shape[1], dtype=torch.bfloat16, device=cuda_device)
        gdn.gdn_conv_prefill(x[:m], s.w, s.bias, conv_pool, _i32([-1], cuda_device), _i32([slot], cuda_device),
                             _i32([0, m], cuda_device), y)
        out = torch.empty(m, H, P, dtype=torch.bfloat16, device=cuda_device)
        gdn.gdn_ssm_prefill(y[:, :H * P].view(m, H, P), y[:, H * P:H * P + G * S].view(m, G, S),
                            y[:, H * P + G * S:].view(m, G, S), dt[:m], z[:m], s.A_log, s.dt_bias, s.D, pool,
                            _i32([-1], cuda_device), _i32([slot], cuda_device), _i32([0, m], cuda_device), out)
        return out
    whole = prompt(n + k, k + 1)
    prompt(n, 0)
    out = torch.empty(k, H, P, dtype=torch.bfloat16, device=cuda_device)
    gdn.gdn_ssm_decode(x[n:], s.w, s.bias, conv_pool, _i32([0], cuda_device), _i32([2], cuda_device), dt[n:], z[n:], s.A_log,
                       s.dt_bias, s.D, pool, _i32([[0, 1, 2, 3]], cuda_device), _i32([1], cuda_device),
                       _i32([0, k], cuda_device), out, G=G)
    rel = (out.double() - whole[n:].double()).norm() / whole[n:].double().norm()
    assert float(rel) <= 2.0 ** -7          # two bf16 results of rows that differ by half a step each way
    assert torch.equal(conv_pool[2, k - 1:k - 1 + W], x[n + k - W:])
