"""The calls of a speculative serving loop together, as a captured graph that
never returns to the host: tables -> gated-delta step and state-space step ->
verification -> the next step's tables.  At the end every request's states and
conv inputs are those of its kept tokens alone, run one at a time."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn

pytestmark = pytest.mark.gpu


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def test_the_loop_keeps_the_states_of_the_kept_tokens(cuda_device):
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(3)
    B, T, V, steps, W = 5, 4, 500, 6, 4
    spec = [1, 1, 0, 1, 1]                       # the third request is not speculative: its rows lie in between
    H_k, H_v = 1, 8                              # gated-delta layer
    H, G, P, S = 4, 2, 64, 64                    # state-space layer
    D = H * P + 2 * G * S
    N = B * T + 3
    kw = dict(generator=g, device=dev)
    bf = torch.bfloat16

    def new(*shape, dtype=torch.int32, fill=0):
        return torch.full(shape, fill, dtype=dtype, device=dev)
    # static buffers of the graph
    q_lens, cu, starts, indx = new(B), new(B + 1), new(B + 1), new(N)
    idx, acc, accepted = new(B, T), new(B), new(B, fill=1)
    cin, cout, turn = new(B), new(B), new(B)
    slots = torch.randperm(B * T, **kw).int().view(B, T)
    conv_table = torch.randperm(2 * B, **kw).int().view(B, 2)
    spec_t = _i32(spec, dev)
    q, k = (torch.zeros(N, H_k, 128, dtype=bf, device=dev) for _ in range(2))
    v, z = (torch.zeros(N, H_v, 128, dtype=bf, device=dev) for _ in range(2))
    a, b = (torch.zeros(N, H_v, dtype=bf, device=dev) for _ in range(2))
    xbc, dt, sz = torch.zeros(N, D, dtype=bf, device=dev), torch.zeros(N, H, dtype=bf, device=dev), torch.zeros(N, H, P, dtype=bf, device=dev)
    rows = [q, k, v, z, a, b, xbc, dt, sz]
    A_log, sA = torch.rand(H_v, **kw), torch.rand(H, **kw)
    bias, sbias = torch.randn(H_v, **kw).to(bf), torch.randn(H, **kw).to(bf)
    norm_w, sD = torch.randn(128, **kw).to(bf), torch.randn(H, **kw)
    conv_w, conv_b = (torch.randn(D, W, **kw) * 0.5).to(bf), (torch.randn(D, **kw) * 0.2).to(bf)
    pool, spool = torch.randn(B * T, H_v, 128, 128, **kw) * 0.1, torch.randn(B * T, H, S, P, **kw) * 0.1
    conv_pool = torch.randn(2 * B, W - 1 + T, D, **kw).to(bf)
    out, sout = torch.zeros(N, H_v, 128, dtype=bf, device=dev), torch.zeros(N, H, P, dtype=bf, device=dev)
    target, draft = torch.zeros(N, V, device=dev), torch.zeros(B, T - 1, V, device=dev)
    tokens, u, us = new(B, T - 1), torch.zeros(B, T - 1, device=dev), torch.zeros(B, device=dev)
    out_tokens, status = new(B, T), new(1)
    # the kept tokens alone: one slot a request, single-token steps
    ref, sref = pool[slots[:, 0].long()].clone(), spool[slots[:, 0].long()].clone()
    ref_conv = torch.zeros(2 * B, W, D, dtype=bf, device=dev)
    ref_conv[:B] = conv_pool[conv_table[:, 0].long(), :W]
    # a fresh slot holds its history behind row 0: num_accepted = 1 reads rows 1 .. W-1
    calls = [
        gdn.prepare_step_tables(q_lens, slots, cu, indx, idx, acc, accepted=accepted, spec=spec_t, row_starts=starts,
                                conv_table=conv_table, conv_turn=turn, conv_in=cin, conv_out=cout, status=status),
        gdn.prepare(q, k, v, a, b, z, A_log, bias, norm_w, pool, idx, acc, cu, out, spec_token_indx=indx, max_T=T, status=status),
        gdn.prepare_ssm_decode(xbc, conv_w, conv_b, conv_pool, cin, cout, dt, sz, sA, sbias, sD, spool, idx, acc, cu, sout, G=G,
                               spec_token_indx=indx, max_T=T, status=status),
        gdn.prepare_verify_drafts(target, tokens, u, us, cu, out_tokens, accepted, draft_probs=draft, spec_token_indx=indx,
                                  status=status),
    ]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        for c in calls:
            c()
    assert accepted.tolist() == [1] * B                                  # capturing ran nothing
    turns = [0] * B
    for step in range(steps):
        lens = [1 + (i + step) % T for i in range(B)]
        if step == 2:
            lens[1] = 0                                                  # a request that sits a step out
        q_lens.copy_(_i32(lens, dev))
        for t in rows:
            t.copy_(torch.randn(t.shape, **kw))
        logits = torch.randn(N, V, **kw)
        target.copy_(torch.softmax(logits, -1))
        first = [sum(lens[:i]) for i in range(B)]
        for i in range(B):
            for t in range(lens[i] - 1):
                draft[i, t] = torch.softmax(logits[first[i] + t] + 0.4 * torch.randn(V, **kw), -1)
                tokens[i, t] = int(torch.multinomial(draft[i, t], 1, generator=g))
        u.uniform_(generator=g)
        us.uniform_(generator=g)
        was = accepted.tolist()
        graph.replay()
        torch.cuda.synchronize()
        assert int(status) == 0
        now = accepted.tolist()
        for i in range(B):
            if not spec[i] or lens[i] == 0:                              # nothing of it ran
                assert now[i] == was[i] and out_tokens[i].tolist() == [-1] * T
                continue
            turns[i] ^= 1
            assert 1 <= now[i] <= lens[i] and (out_tokens[i] >= 0).sum() == now[i]
            one = _i32([0, 1], dev)
            for t in range(now[i]):
                r = slice(first[i] + t, first[i] + t + 1)
                slot = _i32([[i]], dev)
                o = torch.empty(1, H_v, 128, dtype=bf, device=dev)
                gdn.gdn_spec_decode(q[r], k[r], v[r], a[r], b[r], z[r], A_log, bias, norm_w, ref, slot, _i32([1], dev), one, o)
                so = torch.empty(1, H, P, dtype=bf, device=dev)
                gdn.gdn_ssm_decode(xbc[r], conv_w, conv_b, ref_conv, _i32([i], dev), _i32([B + i], dev), dt[r], sz[r], sA, sbias,
                                   sD, sref, slot, _i32([1], dev), one, so, G=G)
                # the new slot's rows are the history and the token; shift them to where a fresh slot holds its history
                ref_conv[i, 1:] = ref_conv[B + i, 1:W].clone()
                # equal up to FP32 rounding order between the layouts: 2^-8 in a bf16 output, twice
                for got, want in ((out[r], o), (sout[r], so)):
                    assert float((got.double() - want.double()).norm()) <= 2.0 ** -7 * float(want.double().norm())
    for i in range(B):
        if not spec[i]:
            continue
        last = int(slots[i, max(int(accepted[i]) - 1, 0)])
        # FP32 states after at most 24 tokens: 24 x 8 roundings of 2^-24
        for got, want in ((pool[last], ref[i]), (spool[last], sref[i])):
            assert float((got.double() - want.double()).norm()) <= 192 * 2.0 ** -24 * float(want.double().norm())
        held = conv_pool[int(conv_table[i, turns[i]])]
        n = int(accepted[i])
        assert torch.equal(held[n:n + W - 1], ref_conv[i, 1:W])
