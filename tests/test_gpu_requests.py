"""Batches whose sequences are requests in some other order: where the
verification's counts go, and the loop of tables, step and verification over
batches that are permuted parts of the requests."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from gated_deltanet_linear_sm_gb300 import binding
from tests.test_gpu_verify import Batch, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,draft,dtype", [(700, True, "f32"), (40000, False, "bf16"), (9, True, "f16")])
def test_counts_go_to_the_requests(cuda_device, V, draft, dtype):
    b = Batch(cuda_device, [3, 1, 0, 4, 2, 4], 4, V, dtype, draft=draft, seed=V)
    b.run()
    _, acc = b.check()                                                  # in batch order, against the definition
    want_tokens = b.out.clone()
    request = [7, 0, 4, 2, -1, 5]                                       # the third has no rows, the fifth is nobody's
    counts = torch.arange(100, 109, dtype=torch.int32, device=cuda_device)
    want = counts.tolist()
    for i in (0, 1, 3, 5):
        want[request[i]] = int(acc[i])
    b.out.fill_(-77)
    b.acc = counts
    b.run(request=_i32(request, cuda_device))
    torch.cuda.synchronize()
    assert torch.equal(b.out, want_tokens) and counts.tolist() == want and int(b.status) == 0


def test_request_out_of_range_is_reported(cuda_device):
    b = Batch(cuda_device, [3, 0, 2, 1], 3, 500, "f32", seed=4)
    b.run()
    torch.cuda.synchronize()
    want_tokens, acc = b.out.clone(), b.acc.tolist()
    counts = torch.full((6,), -9, dtype=torch.int32, device=cuda_device)
    b.acc = counts
    b.run(request=_i32([2, 6, 6, 1], cuda_device))                      # the second has no rows: nothing of it is looked at
    torch.cuda.synchronize()
    assert int(b.status) == binding.GDN_FLAG_SLOT_RANGE
    assert torch.equal(b.out, want_tokens) and counts.tolist() == [-9, acc[3], acc[0], -9, -9, -9]
    b.status.zero_()
    b.run(request=_i32([2, 2 ** 31 - 1, -2 ** 31, 1], cuda_device))
    torch.cuda.synchronize()
    assert int(b.status) == 0 and counts.tolist() == [-9, acc[3], acc[0], -9, -9, -9]


def test_loop_over_permuted_parts_of_the_requests(cuda_device):
    """A captured step of tables, state-space step and verification over batches of four of seven requests
    (or three and a padded entry), another choice in another order each time: every request's state is that
    of its kept tokens alone."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(5)
    R, B, T, V, W, steps = 7, 4, 4, 300, 4, 8
    H, G, P, S = 2, 1, 64, 64
    D, N, bf = H * P + 2 * G * S, B * T, torch.bfloat16
    kw = dict(generator=g, device=dev)

    def new(*shape, dtype=torch.int32, fill=0):
        return torch.full(shape, fill, dtype=dtype, device=dev)
    q_lens, request, cu, indx = new(B), new(B), new(B + 1), new(N)
    idx, acc, accepted = new(B, T), new(B), new(R, fill=1)
    cin, cout, turn = new(B), new(B), new(R)
    slots = torch.randperm(R * T, **kw).int().view(R, T)
    conv_table = torch.randperm(2 * R, **kw).int().view(R, 2)
    xbc, dt, z = new(N, D, dtype=bf), new(N, H, dtype=bf), new(N, H, P, dtype=bf)
    A_log, bias, skip = torch.rand(H, **kw), torch.randn(H, **kw).to(bf), torch.randn(H, **kw)
    conv_w, conv_b = (torch.randn(D, W, **kw) * 0.5).to(bf), (torch.randn(D, **kw) * 0.2).to(bf)
    pool, conv_pool = torch.randn(R * T, H, S, P, **kw) * 0.1, torch.randn(2 * R, W - 1 + T, D, **kw).to(bf)
    out, target, draft = new(N, H, P, dtype=bf), torch.zeros(N, V, device=dev), torch.zeros(B, T - 1, V, device=dev)
    tokens, u, us = new(B, T - 1), torch.zeros(B, T - 1, device=dev), torch.zeros(B, device=dev)
    out_tokens, status = new(B, T), new(1)
    ref, ref_conv = pool[slots[:, 0].long()].clone(), torch.zeros(2 * R, W, D, dtype=bf, device=dev)
    ref_conv[:R] = conv_pool[conv_table[:, 0].long(), :W]
    calls = [
        gdn.prepare_step_tables(q_lens, slots, cu, indx, idx, acc, accepted=accepted, request=request, conv_table=conv_table,
                                conv_turn=turn, conv_in=cin, conv_out=cout, status=status),
        gdn.prepare_ssm_decode(xbc, conv_w, conv_b, conv_pool, cin, cout, dt, z, A_log, bias, skip, pool, idx, acc, cu, out, G=G,
                               spec_token_indx=indx, max_T=T, status=status),
        gdn.prepare_verify_drafts(target, tokens, u, us, cu, out_tokens, accepted, draft_probs=draft, spec_token_indx=indx,
                                  request=request, status=status),
    ]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        for c in calls:
            c()
    rng = np.random.default_rng(6)
    for step in range(steps):
        who = rng.permutation(R)[:B].tolist()
        lens = rng.integers(1, T + 1, B).tolist()
        if step % 3 == 2:
            who[step % B], lens[step % B] = -1, 0
        request.copy_(_i32(who, dev))
        q_lens.copy_(_i32(lens, dev))
        for t in (xbc, dt, z):
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
        assert all(now[r] == was[r] for r in range(R) if r not in who)
        for i, r in enumerate(who):
            if r < 0:
                assert out_tokens[i].tolist() == [-1] * T
                continue
            assert 1 <= now[r] <= lens[i] and (out_tokens[i] >= 0).sum() == now[r]
            for t in range(now[r]):
                row = slice(first[i] + t, first[i] + t + 1)
                o = torch.empty(1, H, P, dtype=bf, device=dev)
                gdn.gdn_ssm_decode(xbc[row], conv_w, conv_b, ref_conv, _i32([r], dev), _i32([R + r], dev), dt[row], z[row], A_log,
                                   bias, skip, ref, _i32([[r]], dev), _i32([1], dev), _i32([0, 1], dev), o, G=G)
                ref_conv[r, 1:] = ref_conv[R + r, 1:W].clone()
                # two bf16 outputs of FP32 sums in another order: half a step each
                assert float((out[row].double() - o.double()).norm()) <= 2.0 ** -7 * float(o.double().norm())
    for r in range(R):
        last = int(slots[r, max(int(accepted[r]) - 1, 0)])
        # FP32 states after at most steps x T tokens of 8 roundings each
        tol = steps * T * 8 * 2.0 ** -24
        assert float((pool[last].double() - ref[r].double()).norm()) <= tol * float(ref[r].double().norm())
