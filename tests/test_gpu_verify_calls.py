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


def _units(p):
    """Probabilities as whole multiples of 2^-52; a row's sums stay far below 2^64."""
    x = np.asarray(p, np.float64)
    return np.rint(np.where(np.isnan(x), 0.0, np.clip(x, 0.0, 1.0)) * 2.0 ** 52).astype(np.uint64)


def _draw(left, u):
    """The lowest entry whose cumulative sum is above u times the sum; -1 for sums of 0 and of 16 or more."""
    total = int(left.sum())
    if total == 0 or total >= 16 * 2 ** 52:
        return -1
    return int(np.searchsorted(np.cumsum(left), np.uint64(int(float(u) * total)), side="right"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V,n", [(4096, 1), (4099, 1), (40000, 200)])
def test_the_limit_of_16_is_on_what_is_left(cuda_device, dtype, draft, V, n):
    """Rows of scores after a refused draft, on both sides of the limit: a row may sum to more where the
    remainder does not."""
    d, step = V // 2, V // 64
    ones = np.array([k * step for k in range(60) if k * step != d])

    def row(entries, at_d):
        p = np.zeros(V)
        p[ones[:int(entries)]] = 1.0
        if entries % 1:
            p[ones[int(entries)]] = entries % 1
        p[d] = at_d
        return p
    if draft:
        # (p, q) with q(d) = 1 and p(d) = 0.5, refused by u = 0.75: r sums to the difference of the ones
        pairs = [(row(20, 0.5), row(10, 1)), (row(26, 0.5), row(10, 1)), (row(25.75, 0.5), row(10, 1)), (row(40, 0.5), row(24, 1)),
                 (row(20, 0.5), row(30, 1)),                            # nothing left: p itself, 20.5
                 (row(15, 0.5), row(30, 1)),                            # p itself, 15.5
                 (row(15.5, 0.5), row(30, 1))]                          # p itself, 16
    else:
        # r is p without the draft
        pairs = [(row(15.75, 0.5), None), (row(16, 0.5), None), (row(15, 0.5), None), (row(17, 0.5), None)]
    target = np.stack([p for p, _ in pairs])
    want, u = [], []
    for k, (p, q) in enumerate(pairs):
        left = _units(p)
        if draft:
            left = np.where(left > _units(q), left - np.minimum(left, _units(q)), np.uint64(0))
            if left.sum() == 0:
                left = _units(p)
        else:
            left[d] = 0
        u.append(np.float32(0.0625 + 0.125 * (k % 7)))
        want.append(_draw(left, u[-1]))
    assert -1 in want and max(want) >= 0
    B = len(pairs) * n
    pick = np.tile(np.arange(len(pairs)), n)
    # every sequence: row k and a row behind its draft that is not reached; the rows are shared
    rows = torch.from_numpy(np.concatenate([target, np.full((1, V), 1.0 / V)])).to(DT[dtype]).to(cuda_device)
    indx = np.stack([pick, np.full(B, len(pairs))], 1).reshape(-1)
    q = torch.from_numpy(np.stack([q for _, q in pairs])).to(DT[dtype]).to(cuda_device)[_i32(pick, cuda_device).long()][:, None] \
        if draft else None
    out, acc = (torch.full(s, -77, dtype=torch.int32, device=cuda_device) for s in ((B, 2), (B,)))
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    gdn.gdn_verify_drafts(rows, torch.full((B, 1), d, dtype=torch.int32, device=cuda_device),
                          torch.full((B, 1), 0.75, device=cuda_device), torch.tensor(np.array(u)[pick], device=cuda_device),
                          _i32(np.arange(B + 1) * 2, cuda_device), out, acc, draft_probs=q,
                          spec_token_indx=_i32(indx, cuda_device), status=status)
    torch.cuda.synchronize()
    assert (acc == 1).all() and (out[:, 1] == -1).all()
    assert out[:, 0].tolist() == [want[k] for k in pick]
    assert int(status) == binding.GDN_FLAG_NO_TOKEN


@pytest.mark.parametrize("dtype,draft", [("f32", True), ("f32", False), ("bf16", True), ("bf16", False), ("f16", False)])
def test_rows_that_are_folded_more_than_once(cuda_device, dtype, draft):
    """A vocabulary above 131072 with one CTA a sequence: a lane adds up more than 256 entries of its piece.
    The rows are shared, the sampling numbers reach every part of them."""
    V, B, T = 151936, 400, 2
    g = torch.Generator(device=cuda_device).manual_seed(30)
    assert 2 * B > 2 * torch.cuda.get_device_properties(cuda_device).multi_processor_count
    P = torch.softmax(torch.randn(3, V, generator=g, device=cuda_device), -1).to(DT[dtype])
    Q = torch.softmax(torch.randn(2, V, generator=g, device=cuda_device), -1).to(DT[dtype]) if draft else None
    d = P[:2].float().argmin(-1).int()                                  # drafts that the target hardly ever takes
    if draft:
        Q[torch.arange(2), d.long()] = 1.0
    pick = np.arange(B) % 2
    u = (np.arange(B) + 0.5) / B
    lefts = []
    for k in range(2):
        left = _units(_host(P)[k])
        if draft:
            q = _units(_host(Q)[k])
            left = np.where(left > q, left - np.minimum(left, q), np.uint64(0))
        else:
            left[int(d[k])] = 0
        lefts.append(left)
    want = [_draw(lefts[k], np.float32(x)) for k, x in zip(pick, u)]
    rows = _i32(np.stack([pick, np.full(B, 2)], 1).reshape(-1), cuda_device)
    out, acc = (torch.full(s, -77, dtype=torch.int32, device=cuda_device) for s in ((B, T), (B,)))
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    sel = _i32(pick, cuda_device).long()
    gdn.gdn_verify_drafts(P, d[sel][:, None].contiguous(), torch.full((B, 1), 0.9999, device=cuda_device),
                          torch.tensor(u, dtype=torch.float32, device=cuda_device), _i32(np.arange(B + 1) * 2, cuda_device), out, acc,
                          draft_probs=None if Q is None else Q[sel][:, None].contiguous(), spec_token_indx=rows, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and (acc == 1).all()
    assert out[:, 0].tolist() == want
