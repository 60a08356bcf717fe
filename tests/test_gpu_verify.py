"""gdn_verify_drafts and gdn_step_tables against their definitions (whole
numbers: every value has to be equal)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from gated_deltanet_linear_sm_gb300 import binding
from tests import ops_ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _i32(v, dev):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)


def _host(t):
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


class Batch:
    """Random inputs of a verification: distributions of sharpness `sharp`,
    drafts near the target's (so that some are kept and some are not)."""

    def __init__(self, dev, q_lens, T, V, dtype, draft=True, seed=0, gather=False, sharp=3.0, near=0.7, offset=0):
        g = torch.Generator().manual_seed(seed)
        B = len(q_lens)
        self.T, self.V = T, V
        cu = np.concatenate([[0], np.cumsum(np.maximum(q_lens, 0))])
        n = int(cu[-1])
        self.N = n + (7 if gather else 0)
        logits = torch.randn(max(self.N, 1), V, generator=g) * sharp
        # rows start `offset` elements behind an aligned address
        room = torch.zeros(max(self.N, 1) * V + offset, dtype=DT[dtype], device=dev)
        self.target = room[offset:].view(max(self.N, 1), V)
        self.target.copy_(torch.softmax(logits, -1))
        self.indx = torch.randperm(self.N, generator=g)[:n].int() if gather else None
        rows = self.indx.tolist() if gather else list(range(n))
        self.rows = [rows[cu[i]:cu[i + 1]] for i in range(B)]
        k = max(T - 1, 1)
        self.tokens = torch.zeros(B, k, dtype=torch.int32)
        self.draft = torch.zeros(B, k, V, device=dev, dtype=DT[dtype]) if draft else None
        for i, r in enumerate(self.rows):
            for t in range(len(r) - 1):
                close = logits[r[t]] + near * torch.randn(V, generator=g)
                q = torch.softmax(close, -1)
                self.tokens[i, t] = int(torch.multinomial(q, 1, generator=g)) if draft else int(logits[r[t]].argmax())
                if draft:
                    self.draft[i, t] = q.to(self.draft)
        self.tokens = self.tokens.to(dev)
        self.accept_u = torch.rand(B, k, generator=g).to(dev)
        self.sample_u = torch.rand(B, generator=g).to(dev)
        self.cu = _i32(cu, dev)
        self.indx = self.indx.to(dev) if gather else None
        self.out = torch.full((B, T), -77, dtype=torch.int32, device=dev)
        self.acc = torch.full((B,), -77, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def run(self, **kw):
        gdn.gdn_verify_drafts(self.target, self.tokens, self.accept_u, self.sample_u, self.cu, self.out, self.acc,
                              draft_probs=self.draft, spec_token_indx=self.indx, status=self.status, **kw)

    def check(self, flag=0):
        torch.cuda.synchronize()
        want, acc, empty = ops_ref.verify(_host(self.target), None if self.draft is None else _host(self.draft),
                                          _host(self.tokens), _host(self.accept_u), _host(self.sample_u), self.rows, self.T)
        assert self.acc.cpu().tolist() == [-77 if v < 0 else v for v in acc.tolist()]
        assert self.out.cpu().tolist() == want.tolist()
        assert int(self.status) == flag | (binding.GDN_FLAG_NO_TOKEN if empty else 0)
        return want, acc


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,T,lens", [
    (1, 2, [2, 1]), (2, 3, [3, 3, 0, 1]), (7, 1, [1, 1, 0]), (1000, 4, [4, 1, 2, 0, 3, 4]), (4099, 5, [5, 3]),
    (32000, 3, [3]), (50021, 9, [9, 2, 5]), (300, 32, [32, 31, 17, 1]),
])
@pytest.mark.parametrize("draft", [True, False])
def test_against_definition(cuda_device, dtype, V, T, lens, draft):
    b = Batch(cuda_device, lens, T, V, dtype, draft=draft, seed=V + T)
    b.run()
    b.check()


@pytest.mark.parametrize("dtype,offset", [("f32", 1), ("f32", 3), ("bf16", 1), ("bf16", 5), ("f16", 7)])
def test_rows_at_any_element(cuda_device, dtype, offset):
    """Rows that start off a 16-byte boundary, with an odd row length; the drafter's rows sit at other offsets."""
    b = Batch(cuda_device, [3, 4, 1], 4, 10007, dtype, seed=offset, offset=offset)
    b.run()
    b.check()


@pytest.mark.parametrize("seed", range(8))
def test_random_sizes(cuda_device, seed):
    rng = np.random.default_rng(seed)
    n, T = int(rng.choice([1, 2, 9, 80])), int(rng.integers(1, 9))
    q = rng.integers(0, T + 1, n).tolist()
    q[0] = max(q[0], 1)
    V = int(np.exp(rng.uniform(0, np.log(9000 if n > 9 else 60000))))
    b = Batch(cuda_device, q, T, V, str(rng.choice(["f32", "bf16", "f16"])), draft=bool(rng.random() < 0.6), seed=seed,
              gather=bool(rng.random() < 0.5), sharp=float(rng.choice([0.5, 3, 8])), near=float(rng.choice([0.1, 0.7, 2])),
              offset=int(rng.choice([0, 0, 1, 3, 5])))
    b.run()
    b.check()


def test_gathered_rows_and_strides(cuda_device):
    """Rows through spec_token_indx; the target's rows and the draft tables inside wider tensors; the
    drafter's rows stacked step by step."""
    b = Batch(cuda_device, [3, 1, 4, 2], 4, 501, "f32", gather=True, seed=3)
    wide = torch.full((b.target.shape[0], 600), float("nan"), device=cuda_device)
    wide[:, 50:551] = b.target
    b.target = wide[:, 50:551]
    tok = torch.full((4, 9), 10 ** 6, dtype=torch.int32, device=cuda_device)
    tok[:, 2:5] = b.tokens
    b.tokens = tok[:, 2:5]
    u = torch.full((4, 9), float("nan"), device=cuda_device)
    u[:, 2:5] = b.accept_u
    b.accept_u = u[:, 2:5]
    b.draft = b.draft.transpose(0, 1).contiguous().transpose(0, 1)     # [T-1, B, V] underneath
    b.run()
    b.check()


def test_all_kept_and_none_kept(cuda_device):
    b = Batch(cuda_device, [5, 5], 5, 777, "f32", seed=1)
    b.accept_u[0] = 0.0
    b.accept_u[1] = 1.0
    b.draft[1, 0] = 0.0
    b.draft[1, 0, b.tokens[1, 0].long()] = 1.0                          # the drafter was certain of a token
    b.run()
    want, acc = b.check()
    assert acc.tolist() == [5, 1]
    assert want[1, 0] != int(b.tokens[1, 0])                            # and it cannot be drawn again


@pytest.mark.parametrize("u", [0.0, 1.0, float(np.nextafter(np.float32(1), np.float32(0))), 1e-30, -0.5, 7.0, float("nan")])
def test_ends_of_the_sampling_number(cuda_device, u):
    b = Batch(cuda_device, [2, 1, 3], 3, 2049, "f32", seed=5)
    b.sample_u[:] = u
    b.run()
    want, _ = b.check()
    assert ((want < 2049) & (want >= -1)).all()


def test_probabilities_outside_their_range(cuda_device):
    """NaN and negative entries count as 0, entries above 1 as 1."""
    b = Batch(cuda_device, [3, 1, 2], 3, 900, "f32", seed=6)
    b.target[:, ::7] = float("nan")
    b.target[:, 1::11] = -float("inf")
    b.target[:, 5] = float("inf")
    b.target[:, 6] = 3.0
    b.draft[:, :, ::13] = float("nan")
    b.draft[:, :, 6] = 9.0
    b.run()
    b.check()


def test_rows_that_leave_nothing(cuda_device):
    """p below q everywhere: the token comes from p; p of zeros: no token, and a flag."""
    b = Batch(cuda_device, [2, 2, 1], 2, 640, "f32", seed=7)
    b.target[0] = b.draft[0, 0] * 0.5
    b.accept_u[0, 0] = 0.9
    b.run()
    want, acc = b.check()
    assert acc[0] == 1 and want[0, 0] >= 0
    b.target[b.rows[2][0]] = 0.0
    b.run()
    want, acc = b.check()
    assert want[2, 0] == -1 and acc[2] == 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,n", [(4096, 1), (50000, 1), (50000, 700)])
def test_rows_of_scores_are_refused(cuda_device, dtype, V, n):
    """Rows that sum to 16 or more, up to a 1 in every entry (more than 64 bits hold): no token and a flag,
    whatever the number of CTAs; a row of just under 16 has one."""
    target = torch.ones(n, V, dtype=DT[dtype], device=cuda_device)
    target[0] = 0
    target[0, ::V // 16] = 0.96875                                      # 16 or 17 entries: 15.5 or 16.47
    target[0, 16 * (V // 16):] = 0                                      # 16
    out = torch.full((n, 1), -77, dtype=torch.int32, device=cuda_device)
    acc = torch.full((n,), -77, dtype=torch.int32, device=cuda_device)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    gdn.gdn_verify_drafts(target, None, None, torch.full((n,), 0.97, device=cuda_device), _i32(np.arange(n + 1), cuda_device),
                          out, acc, status=status)
    assert out[0, 0] == 15 * (V // 16) and (out[1:] == -1).all() and (acc == 1).all()
    assert int(status) == (binding.GDN_FLAG_NO_TOKEN if n > 1 else 0)
    target[0, 1] = 0.5
    gdn.gdn_verify_drafts(target, None, None, torch.full((n,), 0.97, device=cuda_device), _i32(np.arange(n + 1), cuda_device),
                          out, acc, status=status)
    assert (out == -1).all() and int(status) == binding.GDN_FLAG_NO_TOKEN
    target[0] = 1
    status.zero_()
    gdn.gdn_verify_drafts(target, None, None, torch.full((n,), 0.97, device=cuda_device), _i32(np.arange(n + 1), cuda_device),
                          out, acc, status=status)
    assert (out == -1).all() and int(status) == binding.GDN_FLAG_NO_TOKEN


@pytest.mark.parametrize("draft", [True, False])
def test_drafts_that_are_no_token(cuda_device, draft):
    """A draft outside the vocabulary ends the drafts and is replaced from p alone."""
    b = Batch(cuda_device, [4, 4, 4], 4, 333, "bf16", draft=draft, seed=8)
    b.accept_u[:] = 0.0
    b.tokens[0, 0] = -1
    b.tokens[1, 1] = 333
    b.tokens[2, 2] = 2 ** 31 - 1
    b.run()
    _, acc = b.check()
    assert acc.tolist() == [1, 2, 3]


def test_bad_data_is_reported_and_skipped(cuda_device):
    b = Batch(cuda_device, [2, 2, 2, 2], 2, 128, "f32", seed=9)
    good = [list(r) for r in b.rows]
    b.cu = _i32([0, 2, 5, 6, 8], cuda_device)                           # the second has 3 rows, beyond T = 2
    b.rows = [good[0], None, [5], [6, 7]]
    b.run()
    b.check(flag=binding.GDN_FLAG_QLEN)
    b.acc.fill_(-77)
    b.cu = _i32([-1, 1, 2, 4, 3], cuda_device)                          # before the rows; behind the last offset
    b.status.zero_()
    b.rows = [None, [1], None, None]
    b.run()
    b.check(flag=binding.GDN_FLAG_TOKEN_ROW)
    b.cu = _i32([0, 2, 4, 6, 8], cuda_device)
    b.indx = _i32([0, 1, 2, 8, 4, 5, -1, 7], cuda_device)               # rows outside the target's
    b.acc.fill_(-77)
    b.status.zero_()
    b.rows = [[0, 1], None, [4, 5], None]
    b.run()
    b.check(flag=binding.GDN_FLAG_TOKEN_ROW)


def test_the_split_of_a_row_does_not_matter(cuda_device):
    """One sequence alone (eight CTAs), among 40 and among 700 (one CTA): the same tokens."""
    one = Batch(cuda_device, [4], 4, 40000, "f32", seed=10)
    one.run()
    _, acc = one.check()
    for n in (40, 700):
        out = torch.empty(n, 4, dtype=torch.int32, device=cuda_device)
        got = torch.empty(n, dtype=torch.int32, device=cuda_device)
        gdn.gdn_verify_drafts(one.target, one.tokens.expand(n, 3).contiguous(), one.accept_u.expand(n, 3).contiguous(),
                              one.sample_u.expand(n).contiguous(), _i32(np.arange(n + 1) * 4, cuda_device), out, got,
                              draft_probs=one.draft.expand(n, 3, 40000).contiguous(),
                              spec_token_indx=_i32(list(range(4)) * n, cuda_device))
        assert (got == one.acc).all() and (out == one.out).all()


def test_tokens_follow_the_target(cuda_device):
    """Whatever the drafter proposes, a first token has the target's
    distribution: 20000 verifications over 6 tokens, each count within 5
    standard deviations of n p (fixed random numbers)."""
    n, V = 20000, 6
    g = torch.Generator().manual_seed(12)
    p = torch.tensor([0.05, 0.4, 0.1, 0.25, 0.15, 0.05])
    q = torch.tensor([0.3, 0.1, 0.3, 0.1, 0.1, 0.1])
    tok = torch.multinomial(q, n, replacement=True, generator=g).int().view(n, 1)
    out = torch.empty(n, 2, dtype=torch.int32, device=cuda_device)
    acc = torch.empty(n, dtype=torch.int32, device=cuda_device)
    gdn.gdn_verify_drafts(p.expand(2 * n, V).contiguous().to(cuda_device), tok.to(cuda_device),
                          torch.rand(n, 1, generator=g).to(cuda_device), torch.rand(n, generator=g).to(cuda_device),
                          _i32(np.arange(n + 1) * 2, cuda_device), out, acc,
                          draft_probs=q.expand(n, 1, V).contiguous().to(cuda_device))
    count = np.bincount(out[:, 0].cpu().numpy(), minlength=V)
    want = n * p.numpy()
    assert (np.abs(count - want) <= 5 * np.sqrt(want * (1 - p.numpy()))).all(), count


def test_captured_and_on_a_side_stream(cuda_device):
    b = Batch(cuda_device, [4, 2, 1], 4, 9001, "f32", seed=13)
    call = gdn.prepare_verify_drafts(b.target, b.tokens, b.accept_u, b.sample_u, b.cu, b.out, b.acc, draft_probs=b.draft,
                                     status=b.status)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    b.out.fill_(-5)
    graph.replay()
    b.check()
    b.sample_u.uniform_(generator=torch.Generator(device=cuda_device).manual_seed(1))
    torch.cuda.synchronize()
    graph.replay()
    b.check()
    b.out.fill_(-5)
    torch.cuda.synchronize()
    b.run(stream=side)
    b.check()


# ---- gdn_step_tables -----------------------------------------------------------


def _tables(dev, q, S, R, num_tokens=None, spec=None, request=None, conv=True, seed=0):
    rng = np.random.default_rng(seed)
    B = len(q)
    slots = rng.permutation(R * S).reshape(R, S)
    accepted = rng.integers(0, S + 1, R)
    pair = rng.permutation(2 * R).reshape(R, 2)
    turn = rng.integers(0, 2, R)
    n = int(np.maximum(q, 0).sum()) if num_tokens is None else num_tokens
    t = dict(cu_seqlens=B + 1, row_starts=B + 1, token_indx=n + 5 if num_tokens is None else n, num_accepted=B,
             conv_in=B, conv_out=B)
    t = {k: torch.full((v,), -9, dtype=torch.int32, device=dev) for k, v in t.items()}
    t["state_indices"] = torch.full((B, S), -9, dtype=torch.int32, device=dev)
    d = {k: (None if v is None else _i32(v, dev)) for k, v in
         dict(q=q, slots=slots, accepted=accepted, spec=spec, request=request, pair=pair, turn=turn).items()}
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    extra = dict(conv_table=d["pair"], conv_turn=d["turn"], conv_in=t["conv_in"], conv_out=t["conv_out"]) if conv else {}
    gdn.gdn_step_tables(d["q"], d["slots"], t["cu_seqlens"], t["token_indx"], t["state_indices"], t["num_accepted"],
                        accepted=d["accepted"], spec=d["spec"], request=d["request"], row_starts=t["row_starts"],
                        status=status, **extra)
    torch.cuda.synchronize()
    want, flags = ops_ref.tables(q, slots, accepted, t["token_indx"].shape[0], spec, request,
                                 pair if conv else None, turn if conv else None)
    assert int(status) == flags
    w = len(want["token_indx"])
    got = t["token_indx"].cpu().tolist()
    assert got[:w] == want["token_indx"] and got[w:] == [-9] * (len(got) - w)
    for k in ("cu_seqlens", "row_starts", "state_indices", "num_accepted"):
        assert t[k].cpu().tolist() == want[k], k
    if conv:
        assert t["conv_in"].cpu().tolist() == want["conv_in"] and t["conv_out"].cpu().tolist() == want["conv_out"]
        assert d["turn"].cpu().tolist() == want["conv_turn"].tolist()
    return flags


@pytest.mark.parametrize("B,S", [(1, 1), (1, 8), (5, 3), (63, 4), (64, 4), (65, 5), (130, 8), (1000, 2), (4097, 8)])
@pytest.mark.parametrize("mixed", [False, True])
def test_tables_against_definition(cuda_device, B, S, mixed):
    rng = np.random.default_rng(B + S)
    spec = (rng.random(B) < 0.6).astype(np.int32) if mixed else None
    q = rng.integers(0, S + 1, B)
    if mixed:
        q = np.where(spec == 1, q, rng.integers(0, 40, B))
        q[rng.integers(0, B)] = 2500 if spec.min() == 0 and B > 1 else q[0]     # one long prompt
        q = np.where((spec == 1) & (q > S), S, q)
    request = rng.permutation(B + 3)[:B] if mixed else None
    assert _tables(cuda_device, q, S, B + 3, spec=spec, request=request, conv=mixed, seed=B) == 0


def test_tables_of_padded_and_bad_requests(cuda_device):
    q = np.array([2, 0, 3, -4, 1, 9, 2, 1])
    request = np.array([4, 1, -1, 2, 8, 0, 3, 7])                       # row 8 of 8 does not exist; -1 is padding
    flags = _tables(cuda_device, q, 3, 8, request=request)
    assert flags == binding.GDN_FLAG_SLOT_RANGE | binding.GDN_FLAG_QLEN


def test_tables_that_do_not_fit_give_an_empty_step(cuda_device):
    assert _tables(cuda_device, np.array([2, 3, 4]), 4, 3, num_tokens=8) == binding.GDN_FLAG_TOKEN_ROW
    assert _tables(cuda_device, np.array([2, 3, 4]), 4, 3, num_tokens=9) == 0
    big = np.full(300, 2 ** 31 - 1)
    assert _tables(cuda_device, big, 4, 300, num_tokens=50, spec=np.zeros(300, np.int32)) == binding.GDN_FLAG_TOKEN_ROW


def test_tables_of_no_request(cuda_device):
    e = torch.empty(0, dtype=torch.int32, device=cuda_device)
    cu = torch.full((1,), -9, dtype=torch.int32, device=cuda_device)
    gdn.gdn_step_tables(e, torch.zeros(4, 2, dtype=torch.int32, device=cuda_device), cu, e, e.view(0, 2), e,
                        accepted=torch.zeros(4, dtype=torch.int32, device=cuda_device))
    assert cu.cpu().tolist() == [0]
