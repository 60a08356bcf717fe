"""gdn_attn_decode where sizes differ by many powers of two: values' scales that
a row does not see or hardly weighs, loud elements of q, scores of any finite
size, weights far below the largest.  Against the definition in 64 bits.

The bound, elementwise, with p_j the softmax's weights and A = sum_j p_j |v_j|:
  2^-8 |o|                  the output's rounding to bf16, half a step
  sum_j p_j d_j (|v_j| + A) an error d_j of score j acts on the sum and on its divisor:
      D 2^-22 B_j               products of the head dim added up in FP32 (B_j = sum |q k| scale)
      2^-21 (1 + |s_j| + |s|)   its rounding and its difference from the reference (s: the row's largest score)
      2^-31 Q K_j               q's elements below 2^-24 of its largest, Q; K_j = sum |k| scale
  2 A (w + (L / 8 + 64) 2^-22)  a weight's rounding: w = 2^-16 for two bf16 parts, 2^-11 for fp16; FP32 sums over L
                            positions in parts
  1.25 2^-31 T C            weights times scales have a step of 2^-22 at most (half of it is off, and 2^-25 before that) where
                            the row's largest, T = max p_j |scale_j|, is 2^8, or 2^-24 where it is 2^6; C = sum_j |code_j|
  A 2^-19                   the gate's exponential and division, the division by the sum
"""
from __future__ import annotations

import math

import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from tests import kv_ref as ref
from tests.test_gpu_kv import BOTH, KINDS, Case

pytestmark = pytest.mark.gpu
SMALL = ["e4m3", "int8"]


def _places(c, i):
    """Pages and rows of all positions of sequence i."""
    x = torch.arange(c.past[i] + c.n[i])
    return c.table[i].long()[x // c.page].to(c.dev), (x % c.page).to(c.dev)


def _bits(t):
    return t.view(torch.int8) if t.dtype.itemsize == 1 else t


def _put(c, which, i, x, value):
    """Row(s) at position(s) x of sequence i become `value` (codes of an 8-bit cache)."""
    pg, row = _places(c, i)
    cache = {"k": c.k, "v": c.v}[which]
    _bits(cache)[pg[x], row[x]] = _bits(value.to(cache.dtype))


def check(c, window=0, scale=None):
    D = c.q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    w = 2.0 ** -16 if c.kind == "bf16" else 2.0 ** -11
    G = c.k.shape[2]
    worst = 0.0
    for i, (p, m) in enumerate(zip(c.past, c.n)):
        pg, row = (t.cpu() for t in _places(c, i))
        k, code = ref.pick(c.k.cpu(), pg, row), ref.pick(c.v.cpu(), pg, row)
        f = torch.ones(k.shape[:2], dtype=torch.float64)
        if c.ks is not None:
            k, f = k * c.ks.cpu()[pg, row].double()[..., None], c.vs.cpu()[pg, row].double()
        for t in range(m):
            r = c.rows[int(c.cu[i]) + t]
            x = torch.arange(p + m)
            seen = (x <= p + t) & (x > p + t - window if window else x >= 0)
            kk, cc, ff = k[seen], code[seen], f[seen]
            q = c.q[r].double().cpu().view(G, -1, D)
            s = torch.einsum("grd,lgd->grl", q, kk) * scale
            B = torch.einsum("grd,lgd->grl", q.abs(), kk.abs()) * scale
            K = kk.abs().sum(-1).t()[:, None] * scale
            d = D * 2.0 ** -22 * B + 2.0 ** -21 * (1 + s.abs() + s.amax(-1, keepdim=True).abs()) + 2.0 ** -31 * q.abs().amax(-1, keepdim=True) * K
            pr = torch.softmax(s, -1)
            v = cc * ff[..., None]
            want, A = torch.einsum("grl,lgd->grd", pr, v), torch.einsum("grl,lgd->grd", pr, v.abs())
            bound = torch.einsum("grl,lgd->grd", pr * d, v.abs()) + A * ((pr * d).sum(-1, keepdim=True) + 2 * w + (len(kk) / 8 + 64) * 2.0 ** -21)
            if c.kind != "bf16":
                top = (pr * ff.abs().t()[:, None]).amax(-1, keepdim=True)
                bound = bound + 1.25 * 2.0 ** -31 * top * cc.abs().sum(0)[:, None]
            gate = torch.sigmoid(c.z[r].double().cpu()).view(want.shape) if c.z is not None else 1.0
            want, bound = want * gate, (bound + 2.0 ** -19 * A) * gate
            bound = bound + 2.0 ** -8 * want.abs() + 2.0 ** -133
            off = (c.out[r].double().cpu().view(want.shape) - want).abs() / bound
            assert bool((off <= 1).all()), (i, t, float(off.nan_to_num(math.inf).max()))
            worst = max(worst, float(off.max()))
    return worst


def _even_scales(c, size=2.0 ** -5):
    """Values' scales within a factor of two, wherever there is one."""
    live = ~torch.isnan(c.vs)
    g = torch.Generator(device=c.dev).manual_seed(3)
    c.vs[live] = size * (1 + torch.rand(int(live.sum()), generator=g, device=c.dev))


# ---- values' scales that a row does not see, or hardly weighs ------------------------------------


@pytest.mark.parametrize("kind", SMALL)
@pytest.mark.parametrize("log2", [20, 32, 60, 120])
@BOTH
def test_a_huge_value_that_a_row_does_not_see(cuda_device, kind, log2, wide):
    """The last drafted token's value, one just below a window, and one that the window leaves to the first token alone."""
    window = 101
    c = Case(cuda_device, [61, 200, 300, 0], [4, 3, 2, 2], 8 * wide, 2, 128, kind, page=16, seed=log2)
    _even_scales(c)
    for i, x in ((0, 64), (1, 98), (2, 200), (3, 1)):
        pg, row = _places(c, i)
        c.vs[pg[x], row[x]] *= 2.0 ** log2
    c.run(window=window)
    assert int(c.status) == 0
    check(c, window)


def _along(c, size):
    """Scores `size` [positions] (natural units) for every row: q of ones, equal elements in a key."""
    D = c.q.shape[2]
    c.q.fill_(1.0)
    for i in range(len(c.n)):
        pg, row = _places(c, i)
        k = size[:len(pg)].to(c.dev)[:, None].expand(-1, c.k.shape[2]) / D ** 0.5
        if c.ks is None:
            c.k[pg, row] = k[..., None].expand(-1, -1, D).to(c.k.dtype)
        else:
            _bits(c.k)[pg, row] = _bits((k.sign() * 64)[..., None].expand(-1, -1, D).to(c.k.dtype))
            c.ks[pg, row] = (k.abs() / 64).float()


@pytest.mark.parametrize("kind", SMALL)
@pytest.mark.parametrize("order", ["first", "middle", "rising"])
@BOTH
def test_huge_values_of_no_weight(cuda_device, kind, order, wide):
    """Values 2^40 times the others under weights of e^-60, and values 2^60 times the others from where scores have risen by hundreds."""
    L = 700
    c = Case(cuda_device, [L - 1, 90], [1, 2], 8 * wide, 2, 128, kind, page=16, seed=1)
    _even_scales(c)
    size = torch.zeros(L + 1)
    if order == "rising":
        size = torch.linspace(0, 400, L + 1)
    else:
        size[5 if order == "first" else 77] = -60.0
    _along(c, size)
    for i in range(2):
        pg, row = _places(c, i)
        for x in [5] if order == "first" else [77] if order == "middle" else range(0, 16):
            c.vs[pg[x], row[x]] *= 2.0 ** (60 if order == "rising" else 40)
    c.run()
    check(c)


@pytest.mark.parametrize("kind", SMALL)
@pytest.mark.parametrize("size", [2.0 ** -70, 2.0 ** -30, 2.0 ** 30, 2.0 ** 100])
@BOTH
def test_values_of_any_size(cuda_device, kind, size, wide):
    c = Case(cuda_device, [300, 4000], [2, 1], 8 * wide, 2, 128, kind, page=16, seed=2)
    _even_scales(c, size)
    c.run()
    check(c)


@pytest.mark.parametrize("kind", SMALL)
@BOTH
def test_rows_of_zeros_before_values(cuda_device, kind, wide):
    """Zeros have the least scale, 2^-100; values of ordinary and of large scales follow, with less weight and with more."""
    for rise in (0.0, 30.0, -30.0):
        c = Case(cuda_device, [900], [2], 8 * wide, 2, 128, kind, page=16, seed=4)
        _even_scales(c)
        _along(c, torch.cat([torch.zeros(300), torch.full((602,), rise)]))
        pg, row = _places(c, 0)
        _bits(c.v)[pg[:300], row[:300]] = 0
        c.vs[pg[:300], row[:300]] = 2.0 ** -100
        c.vs[pg[600:], row[600:]] *= 2.0 ** 20
        c.run()
        check(c)


# ---- weights far below the largest ---------------------------------------------------------------------


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("L,share", [(8192, 0.9), (8192, 0.98), (100003, 0.9)])
@BOTH
def test_many_small_weights_beside_a_large_one(cuda_device, kind, L, share, wide):
    """One position with a value of zeros takes most of the weight; all others share the rest, their values of one sign."""
    c = Case(cuda_device, [L - 1], [1], 8 * wide, 2, 128, kind, page=64, seed=5)
    if c.vs is not None:
        c.vs[~torch.isnan(c.vs)] = 2.0 ** -5
    size = torch.zeros(L)
    size[20] = math.log(share / (1 - share) * (L - 1))
    _along(c, size)
    pg, row = _places(c, 0)
    live = _bits(c.v)[pg, row]
    _bits(c.v)[pg, row] = live.abs() if c.vs is None else live & 0x7F if kind == "e4m3" else live.abs()
    _bits(c.v)[pg[20], row[20]] = 0
    c.run()
    check(c)


# ---- q ---------------------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("log2", [7, 11, 16, 22])
@BOTH
def test_a_loud_element_of_q(cuda_device, kind, log2, wide):
    """One element of each query is 2^7 to 2^22 times the others, where the keys have nothing."""
    c = Case(cuda_device, [61, 500], [2, 3], 8 * wide, 2, 128, kind, page=16, seed=log2)
    c.q[..., 3] = 2.0 ** log2 * 1.5
    for i in range(2):
        pg, row = _places(c, i)
        _bits(c.k)[pg, row, :, 3] = 0
    c.run()
    check(c)


# ---- scores --------------------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("score", [-1e34, -3e31, -1e9, 1e9, 1e34])
@BOTH
def test_scores_of_any_size(cuda_device, kind, score, wide):
    """Equal scores, far below or above zero: the output is the mean of the values, whatever their scales."""
    D = 128
    for factor in (1.0, 2.0 ** 20):
        c = Case(cuda_device, [0, 40, 300], [1, 3, 1], 8 * wide, 2, D, kind, page=16, seed=6)
        if c.vs is not None:
            _even_scales(c, factor * 2.0 ** -5)
        size = 32768.0
        c.q.fill_(score / size / D ** 0.5)
        for i in range(3):
            pg, row = _places(c, i)
            if c.ks is None:
                c.k[pg, row] = size
            else:
                _bits(c.k)[pg, row] = _bits(torch.full((1,), 64.0, device=c.dev).to(c.k.dtype))
                c.ks[pg, row] = size / 64
        c.run()
        for i, (p, n) in enumerate(zip(c.past, c.n)):
            pg, row = (t.cpu() for t in _places(c, i))
            v = ref.pick(c.v.cpu(), pg, row)
            if c.vs is not None:
                v = v * c.vs.cpu()[pg, row].double()[..., None]
            for t in range(n):
                want, A = v[:p + t + 1].mean(0), v[:p + t + 1].abs().mean(0)
                got = c.out[int(c.cu[i]) + t].double().cpu().view(2, -1, D)
                # (a weight's rounding twice over; FP32 sums; the output's half step)
                assert bool(((got - want[:, None]).abs() <= 2.0 ** -8 * want.abs()[:, None] + 2.0 ** -9 * A[:, None]).all()), (i, t)


# ---- what is no number, where its weight is 0 in FP32 ----------------------------------------------------


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("x", [0, 21, 700, 2000])
@BOTH
def test_a_value_that_is_no_number_at_scores_far_below(cuda_device, kind, bad, x, wide):
    """Scores rise by 900 along the sequence; whoever sees the value is spoiled, whichever warp or CTA took it."""
    L = 6000
    c = Case(cuda_device, [L, 300], [1, 2], 8 * wide, 2, 128, kind, page=16, seed=8)
    _along(c, torch.linspace(0, 900, L + 2))
    clean = c.run().double().cpu()
    pg, row = _places(c, 0)
    if c.vs is None:
        c.v[pg[x], row[x], 1, 5] = bad
    else:
        c.vs[pg[x], row[x], 1] = bad
    spoiled = torch.zeros(3, 8 * wide, 128, dtype=torch.bool)
    spoiled[0, 4 * wide:, slice(5, 6) if c.vs is None else slice(None)] = True
    out = c.run().double().cpu()
    if c.vs is not None and math.isinf(bad):         # (an infinite scale times a code of 0 is NaN, times others an infinity)
        assert not bool(torch.isfinite(out[spoiled]).any())
    assert torch.equal(~torch.isfinite(out), spoiled)
    assert torch.equal(out[~spoiled], clean[~spoiled])


# ---- values up to the largest ------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@BOTH
def test_values_up_to_the_largest(cuda_device, kind, wide):
    """Rows of values up to 3e38 through gdn_kv_write, attended to alone, a few and many of them."""
    dev, H, G, D, page = cuda_device, 8 * wide, 2, 128, 16
    past, n = [0, 2, 700], [1, 2, 1]
    c = Case(dev, past, n, H, G, D, kind, page=page, seed=9)
    g = torch.Generator(device=dev).manual_seed(1)
    full = [p + m for p, m in zip(past, n)]
    N = sum(full)
    k = torch.randn(N, G, D, generator=g, device=dev).bfloat16()
    v = ((torch.rand(N, G, D, generator=g, device=dev) * 0.5 + 0.45) * 3e38).bfloat16()
    v[..., ::3] = -v[..., ::3]
    gdn.gdn_kv_write(k, v, c.k, c.v, c.table.to(dev), torch.zeros(3, dtype=torch.int32, device=dev), ref.offsets(full).to(dev),
                     k_scale=c.ks, v_scale=c.vs)
    c.run()
    check(c)


# ---- the gate ------------------------------------------------------------------------------------------------


@BOTH
def test_gates_far_below_zero(cuda_device, wide):
    """Large values through a gate of e^-60 to e^-100 (an output that is a number as long as bf16 has one)."""
    c = Case(cuda_device, [3, 900], [2, 1], 8 * wide, 2, 128, "bf16", page=16, seed=10, gate=True)
    for i in range(2):
        pg, row = _places(c, i)
        c.v[pg, row] = (c.v[pg, row].float() * 1e30).bfloat16()
    c.z[:] = torch.linspace(-100, -60, 128, device=c.dev).bfloat16()
    c.run()
    check(c)


@pytest.mark.parametrize("kind", KINDS)
@BOTH
def test_scores_beside_which_a_reference_is_rounded(cuda_device, kind, wide):
    """A single position: its value, whatever the score's size (2^20 to 2^36 in steps of a third of a power)."""
    D = 128
    c = Case(cuda_device, [0], [1], 8 * wide, 2, D, kind, page=16, seed=6)
    if c.vs is not None:
        _even_scales(c)
    pg, row = _places(c, 0)
    if c.ks is None:
        c.k[pg, row] = 32768.0
    else:
        _bits(c.k)[pg, row] = _bits(torch.full((1,), 64.0, device=c.dev).to(c.k.dtype))
        c.ks[pg, row] = 512.0
    v = ref.pick(c.v.cpu(), pg.cpu(), row.cpu())[0]
    if c.vs is not None:
        v = v * c.vs.cpu()[pg.cpu(), row.cpu()].double()[0][:, None]
    for log2 in range(60, 109):
        for sign in (1, -1):
            c.q.fill_(sign * 2.0 ** (log2 / 3) / 32768.0 / D ** 0.5)
            got = c.run()[0].double().cpu().view(2, -1, D)
            assert bool(((got - v[:, None]).abs() <= (2.0 ** -8 + 2.0 ** -11) * v.abs()[:, None]).all()), (log2, sign)
