"""gdn_kv_write, gdn_kv_read and gdn_attn_decode against their definitions in
64 bits (tests/kv_ref.py).

What a write leaves and a read gives have to be equal to the definition, up to
the one rounding of a read row (half a step, checked as equality with torch's
rounding of the 64-bit value: codes times scale are exact in 64 bits and FP32
rounds them at most once more, to 24 bits of 11 + 8 significant ones: exact).

The attention's bound, elementwise, with A = sum_j p_j |v_j| (64 bits):
  2^-8 |o|                  the output's rounding to bf16, half a step
  A times, twice over (the weights' errors act on the sum and its divisor):
    D 2^-22 B + 2^-21 (1 + S)  a score's products, added up in FP32 (B: the largest sum of
                            |q k| scale; the tensor cores may cut instead of round, hence 2^-22 each),
                            and its rounding, its difference from the reference and the power of two
                            (S: the largest score in units of log2 e, two)
    w                       a weight's rounding: two bf16 parts 2^-16, fp16 2^-11
    (L / 8 + 64) 2^-22      FP32 sums over L positions in parts
  A 2^-19                   the gate's exponential and division, the division by the sum
  V 2^-30 L                 fp16 weights below 2^-14 have a step of 2^-24, half of it 2^-25, where the
                            largest is 2^6 at least; V: the largest |v| (of the values' unit: twice a scale times a code)
"""
from __future__ import annotations

import math
import random

import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from tests import kv_ref as ref

pytestmark = pytest.mark.gpu
KINDS = list(ref.TYPES)
# few query rows, a few dozen, and more than 64: there are two kernels and units of 8 to 64 rows (int8 caches, and pages that are no
# whole groups of 8 positions, run on the first with any number of rows)
BOTH = pytest.mark.parametrize("wide", [1, 7, 17])
SENTINEL = 0x7FBF               # a NaN bf16 pattern that no kernel writes


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _sentinel(shape, dev):
    return torch.full(shape, SENTINEL, dtype=torch.int16, device=dev).view(torch.bfloat16)


def _fill(cache, scales, table, lens, page, kind, g, loud=1.0):
    """Random rows at every position of every sequence; on the device, quantised as torch does."""
    k_cache, v_cache = cache
    G, D = k_cache.shape[2:]
    for i, n in enumerate(lens):
        if n == 0:
            continue
        x = torch.arange(n)
        pg = table[i].long()[x // page]
        ok = (pg >= 0) & (pg < k_cache.shape[0])
        pg, row = pg[ok].to(k_cache.device), (x[ok] % page).to(k_cache.device)
        for c, s in zip(cache, scales):
            v = torch.randn(len(pg), G, D, generator=g, device=c.device) * loud
            if s is None:
                c[pg, row] = v.to(c.dtype)
            elif kind == "int8":
                c[pg, row] = torch.randint(-127, 128, v.shape, generator=g, device=c.device, dtype=torch.int8)
                s[pg, row] = torch.rand(len(pg), G, generator=g, device=c.device) * 0.03 * loud + 1e-3
            else:
                c.view(torch.int8)[pg, row] = (v * 20).to(c.dtype).view(torch.int8)
                s[pg, row] = 2.0 ** torch.randint(-8, -2, (len(pg), G), generator=g, device=c.device).float() * loud


class Case:
    """A batch: tables, cache (NaN at every place that holds nothing), queries."""

    def __init__(self, dev, past, n, H, G, D, kind, page=16, layout="nhd", gate=False, gather=False, max_T=None, q_size=1.0, seed=0,
                 loud=1.0):
        self.dev, self.past, self.n, self.page, self.kind = dev, list(past), list(n), page, kind
        g = torch.Generator(device=dev).manual_seed(seed)
        self.table, pages = ref.tables(past, n, page, seed)
        self.k, self.v, self.ks, self.vs = ref.make_cache(pages, page, G, D, kind, layout, dev)
        _fill((self.k, self.v), (self.ks, self.vs), self.table, [p + m for p, m in zip(past, n)], page, kind, g, loud)
        self.cu = ref.offsets(n)
        N = int(self.cu[-1]) + (5 if gather else 0)
        self.rows = random.Random(seed).sample(range(N), int(self.cu[-1])) if gather else list(range(N))
        self.q = (torch.randn(N, H, D, generator=g, device=dev) * q_size).bfloat16()
        self.z = torch.randn(N, H, D, generator=g, device=dev).bfloat16() if gate else None
        self.out = _sentinel((N, H, D), dev)
        self.sti = _i32(self.rows, dev) if gather else None
        self.max_T = max_T or max(max(n), 1)
        self.status = _i32([0], dev)

    def kw(self, **over):
        kw = dict(max_T=self.max_T, k_scale=self.ks, v_scale=self.vs, z=self.z, spec_token_indx=self.sti, status=self.status)
        return {**kw, **over}

    def args(self):
        return (self.q, self.k, self.v, self.table.to(self.dev), _i32(self.past, self.dev), self.cu.to(self.dev), self.out)

    def run(self, **over):
        gdn.gdn_attn_decode(*self.args(), **self.kw(**over))
        torch.cuda.synchronize()
        return self.out

    def check(self, window=0, scale=None, skipped=(), some=None):
        """Every row against the definition; rows of nobody and of `skipped` sequences are as they were."""
        D = self.q.shape[2]
        scale = D ** -0.5 if scale is None else scale
        cpu = dict(k=self.k.cpu(), v=self.v.cpu(), ks=None if self.ks is None else self.ks.cpu(),
                   vs=None if self.vs is None else self.vs.cpu(), q=self.q.cpu(), z=None if self.z is None else self.z.cpu())
        out = self.out.cpu()
        written = torch.zeros(out.shape[0], dtype=torch.bool)
        w = 2.0 ** -16 if self.kind == "bf16" else 2.0 ** -11
        for i, (p, m) in enumerate(zip(self.past, self.n)):
            if i in skipped or m <= 0:
                continue
            for t in range(m):
                written[self.rows[int(self.cu[i]) + t]] = True
            if some is not None and i not in some:
                continue
            L = p + m
            x = torch.arange(L)
            pg = self.table[i].long()[x // self.page]
            has = (pg >= 0) & (pg < self.k.shape[0])
            pg, row = pg.clamp(0, self.k.shape[0] - 1), x % self.page
            k, v = ref.pick(cpu["k"], pg, row), ref.pick(cpu["v"], pg, row)
            if cpu["ks"] is not None:
                k, v = k * cpu["ks"][pg, row].double()[..., None], v * cpu["vs"][pg, row].double()[..., None]
            for t in range(m):
                r = self.rows[int(self.cu[i]) + t]
                seen = has & (x <= p + t)
                if window:
                    seen &= x > p + t - window
                want, A, B, S = ref.attend(cpu["q"][r], k, v, seen, scale, None if cpu["z"] is None else cpu["z"][r])
                got = out[r].double()
                if not bool(torch.isfinite(want).all()):
                    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))
                    fine = torch.isfinite(want)
                    got, want, A = got[fine], want[fine], A[fine]
                    if want.numel() == 0:
                        continue
                live = int(seen.sum())
                V = float(v[seen].abs().max()) if live else 0.0
                e = 2 * (D * 2.0 ** -22 * B + 2.0 ** -21 * (1 + 2 * S) + w + (live / 8 + 64) * 2.0 ** -22) + 2.0 ** -19
                bound = 2.0 ** -8 * want.abs() + e * A + (0 if self.kind == "bf16" else 2 * V * 2.0 ** -30 * live)
                bad = (got - want).abs() > bound
                assert not bool(bad.any()), (i, t, float(((got - want).abs() - bound).max()), float(want.abs().max()))
        left = out.view(torch.int16)[~written]
        assert bool((left == SENTINEL).all())


# ---- the attention ---------------------------------------------------------------------


LENS = [0, 1, 14, 15, 16, 17, 47, 62, 63, 64, 65, 126, 127, 128, 129, 200, 511, 1000]


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("kind", KINDS)
@BOTH
def test_single_tokens_of_every_length(cuda_device, kind, D, wide):
    c = Case(cuda_device, LENS, [1] * len(LENS), 8 * wide, 2, D, kind, seed=D)
    c.run()
    assert int(c.status) == 0
    c.check()


@pytest.mark.parametrize("H,G,T", [(1, 1, 1), (6, 2, 3), (16, 1, 1), (17, 1, 1), (8, 8, 8), (24, 4, 5), (32, 4, 8), (64, 1, 8), (5, 5, 2)])
@pytest.mark.parametrize("kind", KINDS)
def test_drafted_tokens_and_head_layouts(cuda_device, kind, H, G, T):
    past = [0, 3, 15, 16, 60, 63, 64, 100, 300, 777]
    n = [1 + (i * 3) % T for i in range(len(past))]
    n[4] = T
    c = Case(cuda_device, past, n, H, G, 128, kind, page=32, gate=True, gather=True, max_T=T, seed=H + T)
    c.run()
    assert int(c.status) == 0
    c.check()


@pytest.mark.parametrize("page", [1, 7, 8, 16, 40, 48, 64, 128, 256, 544])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "pair"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@BOTH
def test_page_sizes_and_layouts(cuda_device, kind, layout, page, wide):
    c = Case(cuda_device, [0, 40, 129, 700, 1200], [2, 1, 3, 2, 3], 6 * wide, 2, 64, kind, page=page, layout=layout, seed=page)
    c.run()
    c.check()


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 5000])
@pytest.mark.parametrize("kind", KINDS)
@BOTH
def test_windows(cuda_device, kind, window, wide):
    c = Case(cuda_device, [0, 5, 16, 99, 100, 640, 1500], [1, 4, 3, 4, 2, 4, 4], 8 * wide, 2, 128, kind, page=64 if wide > 1 else 16, seed=window)
    c.run(window=window)
    c.check(window=window)


@pytest.mark.parametrize("kind", KINDS)
@BOTH
def test_pages_that_are_none(cuda_device, kind, wide):
    """Pages that a window has left behind, a hole, and a sequence with no page at all: its rows are zero."""
    c = Case(cuda_device, [100, 400, 70, 33], [1, 3, 2, 1], 4 * wide, 2, 128, kind, seed=5)
    c.table[0, 0] = -1
    c.table[1, 3:9] = -7
    c.table[2, :] = -1
    c.run()
    assert int(c.status) == 0
    c.check()
    assert bool((c.out[4:6].float() == 0).all())


@pytest.mark.parametrize("scale", [0.0, 0.7])
def test_other_scales(cuda_device, scale):
    c = Case(cuda_device, [90, 600], [1, 4], 8, 2, 128, "bf16", seed=2)
    c.run(scale=scale)
    c.check(scale=scale)


def test_a_negative_scale_is_that_of_negated_queries(cuda_device):
    c = Case(cuda_device, [90, 600], [1, 4], 8, 2, 128, "e4m3", seed=2)
    got = c.run(scale=-0.2).clone()
    c.q = -c.q
    c.run(scale=0.2)
    assert torch.equal(got.view(torch.int16), c.out.view(torch.int16))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("order", ["rising", "falling", "loud"])
@BOTH
def test_references_that_move(cuda_device, kind, order, wide):
    """Scores that rise or fall by hundreds along a sequence, and large random ones."""
    dev = cuda_device
    c = Case(dev, [900, 2000], [1, 3], 8 * wide, 1, 64, kind, seed=9, q_size=1.0 if order != "loud" else 30.0)
    if order != "loud":
        u = torch.randn(64, generator=torch.Generator().manual_seed(1)).sign().to(dev)
        c.q = (u * 1.0 + 0.05 * c.q.float()).bfloat16()
        for i, (p, n) in enumerate(zip(c.past, c.n)):
            x = torch.arange(p + n)
            pg, row = c.table[i].long()[x // c.page].to(dev), (x % c.page).to(dev)
            size = torch.linspace(0.0, 40.0, len(x), device=dev)
            size = size if order == "rising" else size.flip(0)
            k = u * size[:, None, None] + 0.1 * torch.randn(len(x), 1, 64, device=dev, generator=torch.Generator(device=dev).manual_seed(2))
            if c.ks is None:
                c.k[pg, row] = k.to(c.k.dtype)
            else:
                s = k.abs().amax(-1).clamp(min=1e-6) / 100
                code = k / s[..., None]
                c.ks[pg, row] = s
                if kind == "int8":
                    c.k[pg, row] = code.round().to(torch.int8)
                else:
                    c.k.view(torch.int8)[pg, row] = code.to(c.k.dtype).view(torch.int8)
    c.run()
    c.check()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@BOTH
def test_scales_of_very_different_sizes(cuda_device, kind, wide):
    """Values' scales from 2^-40 to 2^40 in turn, zero among them; keys' scales that leave the scores small."""
    c = Case(cuda_device, [500, 80], [2, 1], 4 * wide, 1, 128, kind, seed=3)
    g = torch.Generator(device=cuda_device).manual_seed(4)
    live = ~torch.isnan(c.vs)
    c.vs[live] = 2.0 ** torch.randint(-40, 41, (int(live.sum()),), generator=g, device=cuda_device).float()
    c.vs[c.table[0, 2].item(), 3] = 0.0
    c.run()
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("heads", [4, 6, 8, 28])              # of one cache head, by four tokens: units of 16, 24, 32 and 64 rows
def test_a_token_that_is_no_number_spoils_those_that_see_it(cuda_device, kind, bad, heads):
    """The third of four drafted tokens has a value (16 bit) or a scale (8 bit) that is no number, and so has a row just outside
    another sequence's window: who does not see them is not touched."""
    for which in ("v", "k"):
        H = 2 * heads
        c = Case(cuda_device, [61, 200, 30], [4, 2, 1], H, 2, 64, kind, seed=11)
        cache, scale = (c.v, c.vs) if which == "v" else (c.k, c.ks)
        for i, x in ((0, 63), (1, 100)):
            pg, row = int(c.table[i, x // c.page]), x % c.page
            if scale is None:
                cache[pg, row, 1, 5] = bad
            else:
                scale[pg, row, 1] = math.nan
        window = 101                                 # position 100: of the second sequence's tokens 200 and 201 the first sees it
        c.run(window=window)
        out = c.out.double().cpu()
        first = [int(c.cu[i]) for i in range(3)]
        spoiled = torch.zeros(7, H, 64, dtype=torch.bool)
        cols = slice(None) if which == "k" or scale is not None else slice(5, 6)
        for r in (first[0] + 2, first[0] + 3, first[1]):
            spoiled[r, H // 2:, cols] = True
        if which == "v":
            assert torch.equal(~torch.isfinite(out), spoiled)
        else:                                        # an infinite score: NaN, or no weight where it is the negative one
            assert bool(torch.isfinite(out[~spoiled]).all())
            if math.isnan(bad) or scale is not None:
                assert bool(torch.isnan(out[spoiled]).all())
        if which == "v":                             # the rows and columns beside them are right
            _check_unspoiled(c, window, spoiled)


def _check_unspoiled(c, window, spoiled):
    out = c.out.double().cpu()
    k_cache, v_cache, q = c.k.cpu(), c.v.cpu(), c.q.cpu()
    for i, (p, n) in enumerate(zip(c.past, c.n)):
        for t in range(n):
            r = int(c.cu[i]) + t
            x = torch.arange(max(0, p + t - window + 1), p + t + 1)
            pg, row = c.table[i].long()[x // c.page], x % c.page
            k, v = ref.pick(k_cache, pg, row), ref.pick(v_cache, pg, row)
            if c.ks is not None:
                k, v = k * c.ks.cpu()[pg, row].double()[..., None], v * c.vs.cpu()[pg, row].double()[..., None]
            v = torch.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0)
            want, A, B, S = ref.attend(q[r], k, v, torch.ones(len(x), dtype=torch.bool), 64 ** -0.5)
            e = 2 * (64 * 2.0 ** -22 * B + 2.0 ** -21 * (1 + 2 * S) + 2.0 ** -11 + 96 * 2.0 ** -22) + 2.0 ** -19
            bound = 2.0 ** -8 * want.abs() + e * A + 2.0 ** -29 * len(x) * float(v.abs().max())
            assert bool((((out[r] - want).abs() <= bound) | spoiled[r]).all()), (i, t)


@BOTH
def test_queries_that_are_no_numbers_spoil_their_own_head(cuda_device, wide):
    for kind in KINDS:
        c = Case(cuda_device, [300, 20], [2, 1], 8 * wide, 2, 128, kind, seed=21)
        c.run()
        want = c.out.clone()
        c.q[1, 3, 7] = math.nan
        c.q[2, 0, 0] = math.inf
        c.run()
        hit = torch.zeros(3, 8 * wide, dtype=torch.bool, device=cuda_device)
        hit[1, 3] = hit[2, 0] = True
        assert bool(torch.isnan(c.out[hit].float()).all())
        assert torch.equal(c.out[~hit].view(torch.int16), want[~hit].view(torch.int16))


@pytest.mark.parametrize("kind,D,H,G", [("bf16", 128, 8, 1), ("e4m3", 128, 8, 1), ("int8", 256, 4, 2), ("f16", 64, 40, 1),
                                          ("bf16", 128, 40, 1), ("bf16", 256, 40, 1), ("e4m3", 192, 40, 1), ("e4m3", 256, 20, 1)])
def test_one_long_sequence_in_many_parts(cuda_device, kind, D, H, G):
    c = Case(cuda_device, [100003], [2], H, G, D, kind, page=64, seed=1, q_size=2.0)
    c.run()
    c.check()
    again = c.out.clone()
    call = gdn.prepare_attn_decode(*c.args(), **c.kw())
    for _ in range(20):
        c.out.view(torch.int16).fill_(SENTINEL)
        call()
        assert torch.equal(again.view(torch.int16), c.out.view(torch.int16))
    assert int(c.status) == 0


@pytest.mark.parametrize("batch", [127, 129, 257, 480, 481, 700, 1000])
@BOTH
def test_many_sequences(cuda_device, batch, wide):
    """More sequences than a CTA scans at a time, many of them without tokens."""
    rng = random.Random(batch)
    past = [rng.choice([0, 1, 30, 64, 100, 333]) for _ in range(batch)]
    n = [rng.choice([0, 0, 1, 2]) for _ in range(batch)]
    n[-1] = 2
    c = Case(cuda_device, past, n, 4 * wide, 2, 64, "bf16", seed=batch)
    c.run()
    assert int(c.status) == 0
    c.check()


@BOTH
def test_a_batch_without_tokens(cuda_device, wide):
    H = 6 * wide
    c = Case(cuda_device, [5, 9], [0, 0], H, 2, 64, "bf16")
    c.q, c.out = torch.randn(3, H, 64, device=cuda_device).bfloat16(), _sentinel((3, H, 64), cuda_device)
    c.run()
    assert int(c.status) == 0 and bool((c.out.view(torch.int16) == SENTINEL).all())


@BOTH
def test_strided_rows(cuda_device, wide):
    dev, H = cuda_device, 8 * wide
    W = H * 128
    c = Case(dev, [40, 300], [2, 3], H, 2, 128, "bf16", gate=True, seed=6)
    packed = torch.zeros(5, W * 2 + 64, device=dev, dtype=torch.bfloat16)
    packed[:, :W] = c.q.view(5, -1)
    packed[:, W:2 * W] = c.z.view(5, -1)
    c.q, c.z = packed[:, :W].view(5, H, 128), packed[:, W:2 * W].view(5, H, 128)
    wider = _sentinel((5, W + 8), dev)
    c.out = wider[:, :W].view(5, H, 128)
    table = torch.full((2, 40), -1, dtype=torch.int32, device=dev)
    table[:, :c.table.shape[1]] = c.table.to(dev)
    gdn.gdn_attn_decode(c.q, c.k, c.v, table[:, :c.table.shape[1]], _i32(c.past, dev), c.cu.to(dev), c.out, **c.kw())
    torch.cuda.synchronize()
    c.check()
    assert bool((wider[:, W:].contiguous().view(torch.int16) == SENTINEL).all())


FLAGS = [("page", 1), ("long", 1), ("negative", 1), ("q_len", 4), ("row", 8), ("offsets", 8)]


@pytest.mark.parametrize("what,flag", FLAGS)
@BOTH
def test_bad_data_skips_the_sequence(cuda_device, what, flag, wide):
    # (20 and 40 rows for a single token: the bound on the tokens is part of which kernel runs)
    c = Case(cuda_device, [40, 90, 200], [2, 2, 1], {1: 4, 7: 40, 17: 80}[wide], 2, 128, "bf16", gather=what == "row", seed=8)
    skipped = (1,)
    table, past, cu, sti = c.table.clone(), list(c.past), c.cu.clone(), c.sti
    if what == "page":
        table[1, 2] = c.k.shape[0]                   # a page outside counts as none: the sequence runs without it
        c.table[1, 2] = -1
        skipped = ()
    elif what == "long":
        past[1] = table.shape[1] * c.page - 1
    elif what == "negative":
        past[1] = -1
    elif what == "q_len":
        c.max_T = 1
        c.n, c.past = [2, 2, 1], c.past
        skipped = (0, 1)
    elif what == "row":
        sti = sti.clone()
        sti[3] = c.q.shape[0]
    elif what == "offsets":
        cu = torch.tensor([0, 2, 6, 5], dtype=torch.int32)     # the second ends behind the last
        skipped = (1, 2)
    gdn.gdn_attn_decode(c.q, c.k, c.v, table.to(cuda_device), _i32(past, cuda_device), cu.to(cuda_device), c.out,
                        **c.kw(spec_token_indx=sti))
    torch.cuda.synchronize()
    assert int(c.status) == flag
    c.check(skipped=skipped)


@BOTH
def test_rows_and_places_beyond_two_to_the_31_elements(cuda_device, wide):
    """Pages so far apart that the last lies beyond 2^31 elements, 8 and 16 bits."""
    dev = cuda_device
    for kind in ("bf16", "int8" if wide == 1 else "e4m3"):
        c = Case(dev, [70, 33], [1, 2], 4 * wide, 1, 64, kind, seed=2)
        pages = c.k.shape[0]
        apart = (2 ** 31 // max(int(c.table.max()), 1) // 64 + 1) * 64
        big = [torch.zeros(apart * (pages - 1) + c.page * 64, dtype=torch.int8 if c.ks is not None else c.k.dtype, device=dev).view(c.k.dtype)
               for _ in range(2)]
        views = [b.as_strided((pages, c.page, 1, 64), (apart, 64, 64, 1)) for b in big]
        for v, old in zip(views, (c.k, c.v)):
            (v.view(torch.int8) if c.ks is not None else v).copy_(old.view(torch.int8) if c.ks is not None else old)
        assert int(c.table.max()) * apart > 2 ** 31
        c.k, c.v = views
        c.run()
        c.k, c.v = ((v.view(torch.int8) if c.ks is not None else v).contiguous().view(v.dtype) for v in views)
        c.check()
        k = torch.randn(3, 1, 64, device=dev).bfloat16()
        gdn.gdn_kv_write(k, -k, *views, c.table.to(dev), _i32(c.past, dev), c.cu.to(dev), k_scale=c.ks, v_scale=c.vs)
        got = [torch.empty(3, 1, 64, device=dev) for _ in range(2)]
        gdn.gdn_kv_read(*views, c.table.to(dev), _i32(c.past, dev), c.cu.to(dev), *got, k_scale=c.ks, v_scale=c.vs)
        off = (got[0] - k.float()).abs()             # half a step of 8-bit codes (e4m3: of its 4 bits)
        assert bool((off <= k.float().abs().amax(-1, keepdim=True) * (2.0 ** -4 if kind == "e4m3" else 1 / 252)).all())
        assert torch.equal(got[1], -got[0])
        del big, views


@BOTH
def test_captured_on_two_streams_with_lengths_that_grow(cuda_device, wide):
    dev = cuda_device
    cases, graphs, lens = [], [], []
    for s in range(2):
        c = Case(dev, [900, 40, 3000], [4, 4, 4], 8 * wide, 2, 128, ("bf16", "e4m3")[s], seed=s)
        lens.append(_i32(c.past, dev))
        a = list(c.args())
        a[4] = lens[-1]
        call = gdn.prepare_attn_decode(*a, **c.kw())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            call()
        cases.append(c)
        graphs.append((graph, call))
    streams = [torch.cuda.Stream() for _ in range(2)]
    full = [list(c.past) for c in cases]
    for back in (2000, 1, 0):
        for c, l, f in zip(cases, lens, full):
            c.past = [max(0, p - back) for p in f]
            l.copy_(_i32(c.past, dev))
        torch.cuda.synchronize()
        for _ in range(3):
            for (graph, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for c in cases:
            c.check()


@BOTH
def test_a_given_workspace_holds_anything(cuda_device, wide):
    c = Case(cuda_device, [3000, 20], [2, 1], 8 * wide, 2, 128, "f16", seed=3)
    need = gdn.prepare_attn_decode(*c.args(), **c.kw())._bytes
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=cuda_device)
    with pytest.raises(ValueError, match="workspace"):
        c.run(workspace=ws[:-1])
    c.run(workspace=ws)
    c.check()
    other = torch.cuda.Stream()
    gdn.gdn_attn_decode(*c.args(), **c.kw(workspace=ws), stream=other)
    other.synchronize()
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [9, 16, 17, 24, 25, 31, 32, 33, 48])
def test_units_of_every_size_and_pages_that_sequences_share(cuda_device, kind, D, rows):
    c = Case(cuda_device, [0, 40, 700, 700, 2500], [1, 1, 1, 1, 1], rows, 1, D, kind, seed=rows)
    c.table[3, :40] = c.table[2, :40]                # a common prefix
    c.table[4, 7] = c.table[4, 6]                    # and a page twice
    for window in (0, 300):
        c.run(window=window)
        assert int(c.status) == 0
        c.check(window=window)


@pytest.mark.parametrize("seed", range(48))
def test_random_batches(cuda_device, seed):
    rng = random.Random(1000 + seed)
    T = rng.randint(1, 8)
    batch = rng.choice([1, 2, 3, 5, 9, 20])
    G = rng.choice([1, 2, 3, 8])
    kind = KINDS[seed % 4]
    past = [int(math.exp(rng.uniform(0, math.log(4000)))) - 1 for _ in range(batch)]
    n = [rng.randint(0 if batch > 1 else 1, T) for _ in range(batch)]
    window = rng.choice([0, 0, 1, 33, 500])
    c = Case(cuda_device, past, n, G * rng.choice([1, 2, 5, 8, 12, 20]), G, rng.choice([64, 128, 192, 256]), kind, page=rng.choice([1, 16, 24, 64, 100, 128]),
             layout=rng.choice(["nhd", "hnd", "pair"]), gate=rng.random() < 0.5, gather=rng.random() < 0.5, max_T=T, q_size=rng.choice([0.3, 1, 4]),
             seed=seed, loud=rng.choice([0.01, 1.0, 5.0]))
    c.run(window=window)
    assert int(c.status) == 0
    c.check(window=window)


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
def test_waits_that_run_out_end_the_call(cuda_device, kind):
    """With a bound of one poll every wait of the tensor-core kernel runs out: the call ends, says so, and the next one is right."""
    from gated_deltanet_linear_sm_gb300 import binding
    c = Case(cuda_device, [3000, 500, 77], [4, 1, 2], 32, 2, 128, kind, page=64, seed=4)
    binding.set_wait_limit(1)
    try:
        c.run()
    finally:
        binding.set_wait_limit(0)
    assert int(c.status) == binding.GDN_FLAG_TIMEOUT
    c.status.zero_()
    c.out.view(torch.int16).fill_(SENTINEL)
    c.run()
    assert int(c.status) == 0
    c.check()


# ---- the cache -----------------------------------------------------------------------------


def _written(k, kind, cache, scale, where, h):
    """Whether the row at `where`, head h, is what the definition makes of k [D] (float64)."""
    got = cache[where[0], where[1], h]
    if not ref.is_small(kind):
        return torch.equal(got.view(torch.int16), k.to(torch.float32).to(cache.dtype).view(torch.int16))
    code, s = ref.quantise(k, kind)
    sc = float(scale[where[0], where[1], h])
    return (math.isnan(sc) and math.isnan(s) or sc == s) and torch.equal(got.double(), code)


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_write_and_read_back(cuda_device, kind, D):
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(D)
    past, n, G, page = [0, 5, 31, 16, 200], [1, 40, 3, 0, 17], 3, 16
    table, pages = ref.tables(past, n, page, D)
    cache = ref.make_cache(pages, page, G, D, kind, "hnd" if D == 192 else "nhd", dev)
    before = [t.clone() for t in cache if t is not None]
    N = sum(n)
    size = 10.0 ** torch.linspace(-6, 6, N, device=dev)[:, None, None]
    k, v = ((torch.randn(N, G, D, generator=g, device=dev) * size).bfloat16() for _ in range(2))
    k[3, 1] = 0
    k[4, 0] = 1e-38                                  # below the least scale
    v[5, 2, 7] = math.inf
    k[6, 0, 0] = math.nan
    k[7, 0] = torch.arange(D, device=dev).bfloat16() * 0.5 - 30.0    # ties between codes
    k[7, 0, 0] = 127.0 if kind == "int8" else 448.0
    v[8, 0] = 3.0e38
    status = _i32([0], dev)
    cu = ref.offsets(n)
    args = (table.to(dev), _i32(past, dev), cu.to(dev))
    gdn.gdn_kv_write(k, v, cache[0], cache[1], *args, k_scale=cache[2], v_scale=cache[3], status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    ck, cv, cks, cvs = (None if t is None else t.cpu() for t in cache)
    kc, vc = k.double().cpu(), v.double().cpu()
    touched = set()
    for i in range(len(n)):
        for t in range(n[i]):
            where = ref.place(table, i, past[i] + t, page, pages)
            touched.add(where)
            for h in range(G):
                r = int(cu[i]) + t
                if ref.is_small(kind) or bool(torch.isfinite(kc[r, h]).all()):
                    assert _written(kc[r, h], kind, ck, cks, where, h), (i, t, h)
                if ref.is_small(kind) or bool(torch.isfinite(vc[r, h]).all()):
                    assert _written(vc[r, h], kind, cv, cvs, where, h), (i, t, h)
    for old, new in zip(before, [t for t in cache if t is not None]):      # nothing else was written
        o, m = (x.cpu().contiguous().view({1: torch.int8, 2: torch.int16, 4: torch.int32}[x.dtype.itemsize]) for x in (old, new))
        for p in range(pages):
            for r in range(page):
                if (p, r) not in touched:
                    assert torch.equal(o[p, r], m[p, r])
    for dt in (torch.bfloat16, torch.float16, torch.float32):
        rows = [torch.empty(N, G, D, device=dev, dtype=dt) for _ in range(2)]
        gdn.gdn_kv_read(cache[0], cache[1], *args, *rows, k_scale=cache[2], v_scale=cache[3], status=status)
        torch.cuda.synchronize()
        for got, c, s in zip(rows, (ck, cv), (cks, cvs)):
            want = torch.empty(N, G, D, dtype=torch.float64)
            for i in range(len(n)):
                for t in range(n[i]):
                    want[int(cu[i]) + t] = ref.held(c, s, ref.place(table, i, past[i] + t, page, pages))
            want = want.float().to(dt)               # (FP32 holds code times scale; or rounds it before the row's rounding)
            nan = torch.isnan(want)
            assert torch.equal(torch.isnan(got.cpu()), nan)
            a, b = got.cpu()[~nan], want[~nan]
            assert torch.equal(a, b)
    assert int(status) == 0


def test_write_a_prompt_then_the_rest_and_gathered_rows(cuda_device):
    """Prompts in two pieces, the second through a gather of strided rows: the cache is that of one write."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(1)
    n, G, D, page = [300, 7, 64], 4, 128, 48
    table, pages = ref.tables([0] * 3, n, page, 1)
    N = sum(n)
    k, v = (torch.randn(N, G, D, generator=g, device=dev).bfloat16() for _ in range(2))
    for kind in KINDS:
        one, two = (ref.make_cache(pages, page, G, D, kind, "nhd", dev) for _ in range(2))
        gdn.gdn_kv_write(k, v, one[0], one[1], table.to(dev), _i32([0] * 3, dev), ref.offsets(n).to(dev), k_scale=one[2], v_scale=one[3])
        head = [100, 7, 1]
        start = [0, 300, 307]
        first = torch.cat([torch.arange(s, s + h) for s, h in zip(start, head)]).to(dev)
        gdn.gdn_kv_write(k[first], v[first], two[0], two[1], table.to(dev), _i32([0] * 3, dev), ref.offsets(head).to(dev),
                         k_scale=two[2], v_scale=two[3])
        rest = torch.cat([torch.arange(s + h, s + m) for s, h, m in zip(start, head, n)]).to(dev)
        wide = torch.zeros(N, 2 * G * D + 8, device=dev, dtype=torch.bfloat16)
        perm = torch.randperm(N, generator=g, device=dev)
        wide[perm, :G * D], wide[perm, G * D:2 * G * D] = k.view(N, -1), v.view(N, -1)
        kk, vv = wide[:, :G * D].view(N, G, D), wide[:, G * D:2 * G * D].view(N, G, D)
        gdn.gdn_kv_write(kk, vv, two[0], two[1], table.to(dev), _i32(head, dev), ref.offsets([m - h for m, h in zip(n, head)]).to(dev),
                         k_scale=two[2], v_scale=two[3], spec_token_indx=perm[rest].int())
        for a, b in zip(one, two):
            if a is not None:
                assert torch.equal(a.contiguous().view(torch.int8), b.contiguous().view(torch.int8))


@pytest.mark.parametrize("batch", [255, 256, 300, 1000])
def test_write_rows_of_many_sequences(cuda_device, batch):
    dev = cuda_device
    rng = random.Random(batch)
    past, n = [rng.randint(0, 40) for _ in range(batch)], [rng.choice([0, 1, 1, 3]) for _ in range(batch)]
    n[0], n[-1] = 0, 0
    table, pages = ref.tables(past, n, 16, batch)
    N, G, D = sum(n), 2, 64
    k = torch.arange(N, device=dev).float()[:, None, None].expand(N, G, D).bfloat16().contiguous()
    cache = ref.make_cache(pages, 16, G, D, "f16", "pair", dev)
    gdn.gdn_kv_write(k, -k, cache[0], cache[1], table.to(dev), _i32(past, dev), ref.offsets(n).to(dev))
    rows = [_sentinel((N + 3, G, D), dev) for _ in range(2)]
    gdn.gdn_kv_read(cache[0], cache[1], table.to(dev), _i32(past, dev), ref.offsets(n).to(dev), *rows)
    assert torch.equal(rows[0][:N], k) and torch.equal(rows[1][:N], -k)
    assert bool((rows[0][N:].view(torch.int16) == SENTINEL).all())


@pytest.mark.parametrize("kind", KINDS)
def test_captured_reads_and_writes_beside_each_other(cuda_device, kind):
    """A graph that moves rows from one part of a sequence to another sequence, replayed as both places move, beside another
    graph's on another stream."""
    dev, page, G, D, N = cuda_device, 16, 2, 128, 70
    g = torch.Generator(device=dev).manual_seed(6)
    jobs = []
    for j in range(2):
        table, pages = ref.tables([700, 700], [100, 100], page, j)
        cache = ref.make_cache(pages, page, G, D, kind, "nhd", dev)
        _fill(cache[:2], cache[2:], table, [800, 800], page, kind, g)
        rows = [torch.zeros(N, G, D, device=dev, dtype=torch.bfloat16) for _ in range(2)]
        begin, to, cu = _i32([0], dev), _i32([0], dev), _i32([0, N], dev)
        tables = [table[i:i + 1].to(dev).contiguous() for i in range(2)]
        scales = dict(k_scale=cache[2], v_scale=cache[3])
        calls = [gdn.prepare_kv_read(cache[0], cache[1], tables[0], begin, cu, *rows, **scales),
                 gdn.prepare_kv_write(*rows, cache[0], cache[1], tables[1], to, cu, **scales)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            for call in calls:
                call()
        jobs.append((cache, table, rows, begin, to, graph, torch.cuda.Stream(), calls))
    for a, b in ((0, 0), (31, 555), (729, 3)):
        for cache, table, rows, begin, to, graph, stream, _ in jobs:
            begin.fill_(a)
            to.fill_(b)
        torch.cuda.synchronize()
        for job in jobs:
            with torch.cuda.stream(job[6]):
                job[5].replay()
        torch.cuda.synchronize()
        for cache, table, rows, *_ in jobs:
            for c, s, r in zip(cache[:2], cache[2:], rows):
                c, s = c.cpu(), None if s is None else s.cpu()
                x = torch.arange(N) + a
                want = ref.pick(c, table[0].long()[x // page], x % page)
                if s is not None:
                    want = want * s[table[0].long()[x // page], x % page].double()[..., None]
                assert torch.equal(r.cpu(), want.float().bfloat16())
                for t in (0, 33, N - 1):
                    where = ref.place(table, 1, b + t, page, c.shape[0])
                    assert all(_written(r[t, h].double().cpu(), kind, c, s, where, h) for h in range(G))


@pytest.mark.parametrize("what,flag", [("page", 1), ("long", 1), ("negative", 1), ("row", 8), ("offsets", 8), ("none", 0)])
def test_bad_data_of_a_write_and_a_read(cuda_device, what, flag):
    dev = cuda_device
    past, n, G, D, page = [4, 10, 30], [3, 20, 2], 2, 64, 16
    table, pages = ref.tables(past, n, page, 3)
    k = torch.randn(25, G, D, device=dev).bfloat16()
    cu, lens, tab = ref.offsets(n), list(past), table.clone()
    lost = set(range(3, 23))                         # rows of the second sequence
    sti = None
    if what in ("page", "none"):
        tab[1, 1] = pages if what == "page" else -1
        lost = {3 + t for t in range(20) if (10 + t) // page == 1}
    elif what == "long":
        lens[1] = tab.shape[1] * page - 19
    elif what == "negative":
        lens[1] = -1
    elif what == "row":
        sti = torch.arange(25, dtype=torch.int32)
        sti[5] = 25
        lost = {5}
    else:
        cu = torch.tensor([0, 3, 23, 26], dtype=torch.int32)      # the last one ends behind the rows
        lost = {23, 24}
    cache = ref.make_cache(pages, page, G, D, "bf16", "nhd", dev)
    status = _i32([0], dev)
    gdn.gdn_kv_write(k, k, cache[0], cache[1], tab.to(dev), _i32(lens, dev), cu.to(dev), spec_token_indx=None if sti is None else sti.to(dev),
                     status=status)
    torch.cuda.synchronize()
    assert int(status) == flag
    full = sum(int(torch.isfinite(cache[0][p, r]).all()) for p in range(pages) for r in range(page))
    assert full == 25 - len(lost)
    if what == "row":
        return
    rows = [_sentinel((25, G, D), dev) for _ in range(2)]
    status.zero_()
    gdn.gdn_kv_read(cache[0], cache[1], tab.to(dev), _i32(lens, dev), cu.to(dev), *rows, status=status)
    torch.cuda.synchronize()
    assert int(status) == flag
    for r in range(25):
        if r in lost:
            assert bool((rows[0][r].view(torch.int16) == SENTINEL).all())
        else:
            assert torch.equal(rows[0][r], k[r])


# ---- the calls together -----------------------------------------------------------------------


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_speculative_loop_over_the_cache(cuda_device, kind):
    """Captured: the step's rows into the cache, attention over it, the verification, the lengths moved on.  The cache ends with the
    kept tokens alone, and every step's attention is that of a dense softmax over them and the step's own."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(7)
    B, T, H, G, D, V, page, steps = 3, 4, 8, 2, 128, 200, 16, 5
    cols = 8
    table = torch.randperm(B * cols, generator=g, device=dev).int().view(B, cols)
    k_cache, v_cache, ks, vs = ref.make_cache(B * cols, page, G, D, kind, "nhd", dev)
    N = B * T
    q, z = (torch.zeros(N, H, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    k, v = (torch.zeros(N, G, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    out = torch.zeros_like(q)
    q_lens, lens, accepted = (torch.zeros(B, dtype=torch.int32, device=dev) for _ in range(3))
    accepted += 1
    slots = torch.zeros(B, T, dtype=torch.int32, device=dev)
    cu, indx, idx, acc = (torch.zeros(s, dtype=torch.int32, device=dev) for s in (B + 1, N, (B, T), B))
    target = torch.zeros(N, V, device=dev)
    tokens, u, us = torch.zeros(B, T - 1, dtype=torch.int32, device=dev), torch.zeros(B, T - 1, device=dev), torch.zeros(B, device=dev)
    out_tokens, status = torch.zeros(B, T, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    calls = [
        gdn.prepare_step_tables(q_lens, slots, cu, indx, idx, acc, accepted=accepted, status=status),
        gdn.prepare_kv_write(k, v, k_cache, v_cache, table, lens, cu, k_scale=ks, v_scale=vs, spec_token_indx=indx, status=status),
        gdn.prepare_attn_decode(q, k_cache, v_cache, table, lens, cu, out, max_T=T, k_scale=ks, v_scale=vs, z=z, spec_token_indx=indx,
                                status=status),
        gdn.prepare_verify_drafts(target, tokens, u, us, cu, out_tokens, accepted, spec_token_indx=indx, status=status),
    ]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        for c in calls:
            c()
        lens += accepted * (q_lens > 0)
    assert lens.tolist() == [0] * B
    kept = [[] for _ in range(B)]                    # (k, v) rows, float64, as the cache holds them
    for step in range(steps):
        n = [1 + (i + step) % T for i in range(B)]
        if step == 2:
            n[1] = 0
        q_lens.copy_(_i32(n, dev))
        for t in (q, z, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device=dev))
        target.copy_(torch.softmax(3 * torch.randn(N, V, generator=g, device=dev), -1))
        first = ref.offsets(n).tolist()
        for i in range(B):
            for t in range(n[i] - 1):
                tokens[i, t] = int(target[first[i] + t].argmax())
        u.uniform_(generator=g)
        us.uniform_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        assert int(status) == 0
        count = accepted.tolist()
        for i in range(B):
            rows = []
            for t in range(n[i]):
                r = first[i] + t
                kv = []
                for x in (k, v):
                    x = x[r].double().cpu()
                    if kind == "e4m3":
                        x = torch.stack([torch.mul(*ref.quantise(x[h], kind)) for h in range(G)])
                    kv.append(x)
                rows.append(kv)
                K, W = (torch.stack([a[j] for a in kept[i] + rows]) for j in range(2))
                want, A, _, _ = ref.attend(q[r].cpu(), K, W, torch.ones(len(K), dtype=torch.bool), D ** -0.5, z[r].cpu())
                # (weights 2^-11, scores of a few units in FP32: below 2^-10 of A in all; the output's half step)
                assert bool(((out[r].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * A).all())
            kept[i] += rows[:count[i]] if n[i] else []
        assert lens.tolist() == [len(x) for x in kept]
    for i in range(B):
        for x, (kk, vv) in enumerate(kept[i]):
            where = ref.place(table.cpu(), i, x, page, B * cols)
            assert torch.equal(ref.held(k_cache.cpu(), None if ks is None else ks.cpu(), where), kk)
            assert torch.equal(ref.held(v_cache.cpu(), None if vs is None else vs.cpu(), where), vv)
