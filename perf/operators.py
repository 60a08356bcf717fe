"""The operators around a recurrent-state layer's step, as measured cases.

Five calls that a serving loop with speculative decoding makes beside
gdn_spec_decode: the verification of drafted tokens (gdn_verify_drafts), the
next step's tables (gdn_step_tables), the short causal convolution over prompts
(gdn_conv_prefill), and the selective state-space layer over prompts
(gdn_ssm_prefill) and over single or drafted tokens (gdn_ssm_decode).

listed() and draw() give cases, prepare() their inputs on the GPU, run() one
pass: in elementary torch operations, or with ``own`` through this package.
exact() is each operator's definition in 64 bits, token by token.
"""
import math
import random

import torch
import torch.nn.functional as F

own = False

W = 4                       # taps of the short convolution
FIX = float(2 ** 52)        # probabilities are counted in units of 2^-52
STATE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---- cases -------------------------------------------------------------------


def listed():
    return [
        # verification: one request with four drafts (an interactive session), an ordinary speculative batch with the
        # drafter's distributions, and a large batch whose drafts came without distributions (n-gram or greedy drafts)
        dict(name="verify b1 t5 v32000", op="verify", batch=1, T=5, vocab=32000, dtype="f32", draft=True, ragged=False),
        dict(name="verify b32 t8 v151936", op="verify", batch=32, T=8, vocab=151936, dtype="f32", draft=True, ragged=True),
        dict(name="verify b256 t4 v128256 bf16", op="verify", batch=256, T=4, vocab=128256, dtype="bf16", draft=False, ragged=True),
        # tables: the mixed batch of 48 speculative requests among 80 others, and a large engine's step
        dict(name="tables b128 mixed", op="tables", batch=128, S=4, spec_share=0.375, other_max=1),
        dict(name="tables b4096 with prompts", op="tables", batch=4096, S=8, spec_share=0.9, other_max=200),
        # convolution: four prompts of the gated-delta layer's channels, and ragged prompts of a wide state-space layer
        dict(name="conv 4x1024 d2560", op="conv", seqs=4, tokens=4096, ragged=False, channels=2560),
        dict(name="conv 9 ragged d4352", op="conv", seqs=9, tokens=16211, ragged=True, channels=4352),
        # scan: a short prompt, an ordinary prefill batch, and one long prompt of a wide layer
        dict(name="scan 1x100", op="scan", seqs=1, tokens=100, ragged=False, H=16, G=1, P=64, N=128, state="bf16", gate=True),
        dict(name="scan 6 ragged h32", op="scan", seqs=6, tokens=5003, ragged=True, H=32, G=2, P=64, N=64, state="f16", gate=False),
        dict(name="scan 1x16384 h64", op="scan", seqs=1, tokens=16384, ragged=False, H=64, G=8, P=64, N=128, state="f32", gate=True),
        # step: one token for each of two requests, and four drafted tokens for each of 64
        dict(name="step b2 t1 h32", op="step", batch=2, T=1, H=32, G=1, P=64, N=128, state="bf16", gate=True, ragged=False),
        dict(name="step b64 t4 h64", op="step", batch=64, T=4, H=64, G=8, P=64, N=128, state="f32", gate=True, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["verify", "tables", "conv", "scan", "step"])
    if op == "verify":
        return dict(op=op, batch=_log(rng, 1, 200), T=rng.randint(1, 9), vocab=_log(rng, 1000, 160000),
                    dtype=rng.choice(["f32", "bf16", "f16"]), draft=rng.random() < 0.6, ragged=rng.random() < 0.6)
    if op == "tables":
        return dict(op=op, batch=_log(rng, 1, 4000), S=rng.randint(1, 8), spec_share=round(rng.uniform(0.1, 1.0), 2),
                    other_max=_log(rng, 1, 200))
    if op == "conv":
        seqs = _log(rng, 1, 40)
        return dict(op=op, seqs=seqs, tokens=_log(rng, max(seqs, 40), 16000), ragged=rng.random() < 0.7,
                    channels=4 * _log(rng, 40, 1080))
    H = rng.choice([8, 16, 24, 32, 48, 64])
    layer = dict(H=H, G=rng.choice([1, 2, 4, 8]), P=rng.choice([64, 64, 128]) if H <= 32 else 64, N=rng.choice([64, 128]),
                 state=rng.choice(["f32", "bf16", "f16"]), gate=rng.random() < 0.7)
    if op == "scan":
        seqs = _log(rng, 1, 24)
        return dict(op=op, seqs=seqs, tokens=_log(rng, max(seqs, 20), 12000), ragged=rng.random() < 0.7, **layer)
    T = rng.randint(1, 8)
    most = 224 * 64 * 64 * 128 // ((T + 1) * H * layer["P"] * layer["N"])        # states read and written
    return dict(op=op, batch=_log(rng, 1, min(most, 300)), T=T, ragged=rng.random() < 0.7, **layer)


# ---- inputs ------------------------------------------------------------------


def _lengths(total, parts, ragged, seed):
    """`parts` lengths of at least one that add up to `total`."""
    if not ragged:
        return [total // parts + (1 if i < total % parts else 0) for i in range(parts)]
    rng = random.Random(seed)
    cuts = [rng.random() ** 2 + 1e-3 for _ in range(parts)]
    lens = [1 + int((total - parts) * c / sum(cuts)) for c in cuts]
    lens[-1] += total - sum(lens)
    return lens


def _rows(case):
    """The rows of each request in a step, the speculative ones first: the same numbers for every seed."""
    B = case["batch"]
    rng = random.Random(B)
    if case["op"] == "tables":
        spec = max(1, round(case["spec_share"] * B))
        return [rng.randint(1, case["S"]) for _ in range(spec)], [rng.randint(1, case["other_max"]) for _ in range(B - spec)]
    return [rng.randint(1, case["T"]) if case["ragged"] else case["T"] for _ in range(B)]


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"] = case["op"]
    if own:
        s["call"] = _call(s)        # marshalled once, as a serving loop keeps it
    return s


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"verify": _prepare_verify, "tables": _prepare_tables, "conv": _prepare_conv, "scan": _prepare_scan,
            "step": _prepare_step}[case["op"]](case, seed, g)


def _prepare_verify(case, seed, g):
    B, T, V = case["batch"], case["T"], case["vocab"]
    q_lens = _rows(case)
    random.Random(seed).shuffle(q_lens)
    cu = _offsets(q_lens)
    dt = STATE[case["dtype"]]
    kw = dict(generator=g, device="cuda")
    rows = sum(q_lens)
    target = torch.empty(rows, V, device="cuda", dtype=dt)
    draft = torch.empty(B, max(T - 1, 1), V, device="cuda", dtype=dt) if case["draft"] else None
    tokens = torch.randint(0, V, (B, max(T - 1, 1)), dtype=torch.int32, **kw)
    for i in range(B):              # drafts come from a distribution near the target's
        n = q_lens[i]
        logits = torch.randn(n, V, **kw) * 3
        target[cu[i]:cu[i + 1]] = torch.softmax(logits, -1).to(dt)
        if n > 1:
            near = logits[:-1] + 0.5 * torch.randn(n - 1, V, **kw)
            noise = -torch.log(-torch.log(torch.rand(n - 1, V, **kw).clamp(1e-9, 1 - 1e-6)))
            tokens[i, :n - 1] = (near + (noise if case["draft"] else 0)).argmax(-1).int()
            if draft is not None:
                draft[i, :n - 1] = torch.softmax(near, -1).to(dt)
        if draft is not None and n <= T - 1:
            draft[i, n - 1:] = 0
        elif draft is not None and T == 1:
            draft[i] = 0
    return dict(target=target, draft=draft, tokens=tokens, accept_u=torch.rand(B, max(T - 1, 1), **kw),
                sample_u=torch.rand(B, **kw), cu=_i32(cu), T=T,
                out=torch.empty(B, T, dtype=torch.int32, device="cuda"),
                accepted=torch.empty(B, dtype=torch.int32, device="cuda"))


def _prepare_tables(case, seed, g):
    B, S = case["batch"], case["S"]
    mine, others = _rows(case)
    pairs = [(1, n) for n in mine] + [(0, n) for n in others]
    random.Random(seed).shuffle(pairs)
    spec, q = [f for f, _ in pairs], [n for _, n in pairs]
    R = B + 16
    e = dict(dtype=torch.int32, device="cuda")
    perm = torch.randperm(R * S, generator=g, device="cuda").int()
    conv = torch.randperm(R * 2, generator=g, device="cuda").int()
    return dict(q_lens=_i32(q), spec=_i32(spec), request=torch.randperm(R, generator=g, device="cuda")[:B].int(),
                slots=perm.view(R, S), accepted=torch.randint(1, S + 1, (R,), generator=g, **e),
                conv_table=conv.view(R, 2), conv_turn=torch.randint(0, 2, (R,), generator=g, **e),
                cu=torch.empty(B + 1, **e), starts=torch.empty(B + 1, **e), indx=torch.zeros(sum(q), **e),
                idx=torch.empty(B, S, **e), acc=torch.empty(B, **e), conv_in=torch.empty(B, **e), conv_out=torch.empty(B, **e))


def _prepare_conv(case, seed, g):
    lens = _lengths(case["tokens"], case["seqs"], case["ragged"], seed)
    B, D, Ntok = len(lens), case["channels"], case["tokens"]
    kw = dict(generator=g, device="cuda")
    rng = random.Random(seed + 1)
    return dict(x=torch.randn(Ntok, D, **kw).bfloat16(), w=(torch.randn(D, W, **kw) * 0.5).bfloat16(),
                bias=(torch.randn(D, **kw) * 0.1).bfloat16(), pool=torch.randn(2 * B, W + 3, D, **kw).bfloat16(),
                conv_in=_i32([i if rng.random() < 0.5 else -1 for i in range(B)]), conv_out=_i32([B + i for i in range(B)]),
                cu=_i32(_offsets(lens)), y=torch.empty(Ntok, D, device="cuda", dtype=torch.bfloat16))


def _layer(case, Ntok, g):
    """A state-space layer's parameters and rows: step sizes between about 0.001 and 0.2, decay rates 1 to 16 a unit step."""
    H, P = case["H"], case["P"]
    kw = dict(generator=g, device="cuda")
    rate = torch.exp(torch.empty(H, device="cuda").uniform_(math.log(1e-3), math.log(0.1), generator=g))
    return dict(dt=(torch.randn(Ntok, H, **kw) * 0.5).bfloat16(), dt_bias=torch.log(torch.expm1(rate)).bfloat16(),
                A_log=torch.log(torch.empty(H, device="cuda").uniform_(1, 16, generator=g)),
                D=torch.randn(H, **kw) * 0.5 + 1, z=torch.randn(Ntok, H, P, **kw).bfloat16() if case["gate"] else None,
                out=torch.empty(Ntok, H, P, device="cuda", dtype=torch.bfloat16))


def _prepare_scan(case, seed, g):
    lens = _lengths(case["tokens"], case["seqs"], case["ragged"], seed)
    B, Ntok, H, G, P, N = len(lens), case["tokens"], case["H"], case["G"], case["P"], case["N"]
    kw = dict(generator=g, device="cuda")
    rng = random.Random(seed + 1)
    packed = F.silu(torch.randn(Ntok, H * P + 2 * G * N, **kw)).bfloat16()      # the convolution's rows, channels x | B | C
    return dict(x=packed[:, :H * P].view(Ntok, H, P), B=packed[:, H * P:H * P + G * N].view(Ntok, G, N),
                C=packed[:, H * P + G * N:].view(Ntok, G, N), **_layer(case, Ntok, g),
                pool=(torch.randn(2 * B, H, N, P, **kw) * 0.1).to(STATE[case["state"]]),
                read=_i32([i if rng.random() < 0.5 else -1 for i in range(B)]), write=_i32([B + i for i in range(B)]),
                cu=_i32(_offsets(lens)), lens=lens)


def _prepare_step(case, seed, g):
    B, T, H, G, P, N = case["batch"], case["T"], case["H"], case["G"], case["P"], case["N"]
    D = H * P + 2 * G * N
    rng = random.Random(seed)
    lens = _rows(case)
    rng.shuffle(lens)
    Ntok = sum(lens)
    kw = dict(generator=g, device="cuda")
    return dict(xbc=torch.randn(Ntok, D, **kw).bfloat16(), w=(torch.randn(D, W, **kw) * 0.5).bfloat16(),
                bias=(torch.randn(D, **kw) * 0.1).bfloat16(), conv_pool=torch.randn(2 * B, W - 1 + T, D, **kw).bfloat16(),
                conv_in=_i32(list(range(B))), conv_out=_i32([B + i for i in range(B)]), **_layer(case, Ntok, g),
                pool=(torch.randn(B * T, H, N, P, **kw) * 0.1).to(STATE[case["state"]]),
                idx=torch.randperm(B * T, generator=g, device="cuda").int().view(B, T),
                acc=_i32([rng.randint(0, T) for _ in range(B)]), cu=_i32(_offsets(lens)), T=T, G=G)


# ---- one pass ----------------------------------------------------------------


def run(s):
    if own:
        s["call"]()
    else:
        {"verify": _verify, "tables": _tables, "conv": _conv, "scan": _scan, "step": _step}[s["op"]](s)
    return _outputs(s)


def _outputs(s):
    return {"verify": lambda: {"tokens": s["out"], "accepted": s["accepted"]},
            "tables": lambda: {k: s[k] for k in ("cu", "starts", "indx", "idx", "acc", "conv_in", "conv_out", "conv_turn")},
            "conv": lambda: {"y": s["y"], "pool": s["pool"]},
            "scan": lambda: {"out": s["out"], "pool": s["pool"]},
            "step": lambda: {"out": s["out"], "pool": s["pool"], "conv_pool": s["conv_pool"]}}[s["op"]]()


def _call(s):
    import gated_deltanet_linear_sm_gb300 as gdn
    if s["op"] == "verify":
        return gdn.prepare_verify_drafts(s["target"], s["tokens"], s["accept_u"], s["sample_u"], s["cu"], s["out"], s["accepted"],
                                         draft_probs=s["draft"])
    if s["op"] == "tables":
        return gdn.prepare_step_tables(s["q_lens"], s["slots"], s["cu"], s["indx"], s["idx"], s["acc"], spec=s["spec"],
                                       request=s["request"], accepted=s["accepted"], row_starts=s["starts"],
                                       conv_table=s["conv_table"], conv_turn=s["conv_turn"], conv_in=s["conv_in"],
                                       conv_out=s["conv_out"])
    if s["op"] == "conv":
        return gdn.prepare_conv_prefill(s["x"], s["w"], s["bias"], s["pool"], s["conv_in"], s["conv_out"], s["cu"], s["y"])
    if s["op"] == "scan":
        return gdn.prepare_ssm_prefill(s["x"], s["B"], s["C"], s["dt"], s["z"], s["A_log"], s["dt_bias"], s["D"], s["pool"],
                                       s["read"], s["write"], s["cu"], s["out"])
    return gdn.prepare_ssm_decode(s["xbc"], s["w"], s["bias"], s["conv_pool"], s["conv_in"], s["conv_out"], s["dt"], s["z"],
                                  s["A_log"], s["dt_bias"], s["D"], s["pool"], s["idx"], s["acc"], s["cu"], s["out"], G=s["G"])


# ---- the plain forms ---------------------------------------------------------


def _fixed(p):
    return (p.double().nan_to_num(0).clamp(0, 1) * FIX).round().long()


def _verify(s):
    target, tokens, cu, T = s["target"], s["tokens"][:, :s["T"] - 1].long(), s["cu"].long(), s["T"]
    B, V = tokens.shape[0], target.shape[1]
    drafts = cu[1:] - cu[:-1] - 1                                                # per request
    t = torch.arange(T, device="cuda")
    rows = (cu[:-1, None] + t).clamp(max=target.shape[0] - 1)
    p = target[rows[:, :-1], tokens].double()
    i = torch.arange(B, device="cuda")
    q = s["draft"][i[:, None], t[:-1], tokens].double() if s["draft"] is not None else torch.ones_like(p)
    ok = (s["accept_u"][:, :T - 1].double() * q < p) & (t[:-1] < drafts[:, None])
    a = ok.long().cumprod(1).sum(1)
    rejected = a < drafts
    P = _fixed(target[rows[i, a]])
    if T == 1:
        Q = torch.zeros_like(P)
    elif s["draft"] is not None:
        Q = _fixed(s["draft"][i, a.clamp(max=T - 2)])
    else:
        Q = (torch.arange(V, device="cuda") == tokens[i, a.clamp(max=T - 2)][:, None]) * int(FIX)
    rest = (P - Q * rejected[:, None]).clamp(min=0)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, P)
    total = rest.sum(1)
    level = torch.minimum((s["sample_u"].double() * total.double()).floor().long(), total - 1)
    new = (rest.cumsum(1) <= level[:, None]).sum(1)
    new = torch.where(total > 0, new, -1)
    drafted = F.pad(tokens, (0, 1))
    s["out"].copy_(torch.where(t < a[:, None], drafted, torch.where(t == a[:, None], new[:, None], -1)))
    s["accepted"].copy_(a + 1)


def _tables(s):
    q, spec, req = s["q_lens"].long(), s["spec"] > 0, s["request"].long()
    zero = q.new_zeros(1)
    starts = torch.cat([zero, q.cumsum(0)])
    cu = torch.cat([zero, (q * spec).cumsum(0)])
    row = torch.arange(s["indx"].shape[0], device="cuda")
    i = torch.searchsorted(starts, row, right=True) - 1                          # the request of each row
    off = row - starts[i]
    place = torch.where(spec[i], cu[i] + off, cu[-1] + starts[i] - cu[i] + off)
    s["indx"][place] = row.int()
    s["cu"].copy_(cu)
    s["starts"].copy_(starts)
    s["idx"].copy_(torch.where(spec[:, None], s["slots"][req], -1))
    s["acc"].copy_(torch.where(spec, s["accepted"][req], 0))
    turn = s["conv_turn"][req].long()
    pair = s["conv_table"][req]
    s["conv_in"].copy_(torch.where(spec, pair.gather(1, turn[:, None])[:, 0], -1))
    s["conv_out"].copy_(torch.where(spec, pair.gather(1, 1 - turn[:, None])[:, 0], -1))
    s["conv_turn"][req] = torch.where(spec, 1 - turn, turn).int()


def _silu(x):
    return x / (1 + torch.exp(-x))


def _conv(s):
    x, cu = s["x"].float(), s["cu"].long()
    B, D = s["conv_in"].shape[0], x.shape[1]
    past = s["pool"][s["conv_in"].long().clamp(min=0), 1:W].float() * (s["conv_in"] >= 0)[:, None, None]
    # rows in time order, each request's history in front of its own
    row = torch.arange(x.shape[0], device="cuda")
    i = torch.searchsorted(cu, row, right=True) - 1
    ext = x.new_empty(x.shape[0] + B * (W - 1), D)
    at = row + (i + 1) * (W - 1)
    ext[at] = x
    ext[(cu[:-1] + torch.arange(B, device="cuda") * (W - 1))[:, None] + torch.arange(W - 1, device="cuda")] = past
    w = s["w"].float()
    y = s["bias"].float() + sum(ext[at - (W - 1) + k] * w[:, k] for k in range(W))
    s["y"].copy_(_silu(y))
    end = cu[1:] + torch.arange(1, B + 1, device="cuda") * (W - 1)
    s["pool"][s["conv_out"].long(), :W] = ext[end[:, None] - W + torch.arange(W, device="cuda")].bfloat16()


def _decay(dt, dt_bias, A_log):
    """Step sizes, and log-decays in 64 bits (they are summed over whole prompts)."""
    x = dt.float() + dt_bias.float()
    step = torch.where(x > 20, x, torch.log1p(torch.exp(x)))
    return step, -torch.exp(A_log.double()) * step.double()


def _scan(s, chunk=64):
    H, P = s["x"].shape[1:]
    G, N = s["B"].shape[1:]
    lens, cu = s["lens"], _offsets(s["lens"])
    start = [c for i, n in enumerate(lens) for c in range(cu[i], cu[i] + n, chunk)]
    seq = [i for i, n in enumerate(lens) for c in range(0, n, chunk)]
    NC = len(start)
    of = torch.tensor(seq, device="cuda")
    rows = torch.tensor(start, device="cuda")[:, None] + torch.arange(chunk, device="cuda")
    live = rows < s["cu"].long()[of + 1][:, None]                                # rows of another prompt do not count
    rows = rows.clamp(max=s["x"].shape[0] - 1)
    m = live[..., None, None].float()
    x, Bm, Cm = s["x"][rows].float() * m, s["B"][rows].float() * m, s["C"][rows].float() * m      # [NC, Q, ...]
    Bm, Cm = (v.repeat_interleave(H // G, 2) for v in (Bm, Cm))
    step, la = _decay(s["dt"], s["dt_bias"], s["A_log"])
    step, la = step[rows] * m[..., 0], la[rows] * m[..., 0]
    run_ = la.cumsum(1).transpose(1, 2)                                          # [NC, H, Q]
    low = torch.ones(chunk, chunk, device="cuda", dtype=torch.bool).tril()
    inside = torch.exp((run_[..., :, None] - run_[..., None, :]).masked_fill(~low, -math.inf)).float()
    xs = (x * step[..., None]).permute(0, 2, 1, 3)                               # [NC, H, Q, P]
    Bh, Ch = Bm.permute(0, 2, 1, 3), Cm.permute(0, 2, 1, 3)                      # [NC, H, Q, N]
    y = ((Ch @ Bh.transpose(2, 3)) * inside) @ xs
    left = torch.exp(run_[..., -1:] - run_).float()
    add = (Bh * left[..., None]).transpose(2, 3) @ xs                            # [NC, H, N, P]
    # the state before each chunk, from every earlier chunk of its prompt
    total = run_[..., -1].transpose(0, 1)                                        # [H, NC]
    c = torch.arange(NC, device="cuda")
    upto = total.cumsum(1)
    before = upto - total
    same = (of[:, None] == of) & (c[:, None] > c)
    carry = torch.exp((before[:, :, None] - upto[:, None, :]).masked_fill(~same, -math.inf)).float()
    S0 = s["pool"][s["read"].long().clamp(min=0)].float() * (s["read"] >= 0)[:, None, None, None]
    first = torch.tensor([seq.index(i) for i in range(len(lens))], device="cuda")
    since = torch.exp(before - before[:, first[of]]).float().transpose(0, 1)
    S = (carry @ add.transpose(0, 1).reshape(H, NC, N * P)).view(H, NC, N, P).transpose(0, 1)
    S = S + since[..., None, None] * S0[of]
    y = y + torch.exp(run_).float()[..., None] * (Ch @ S) + s["D"][:, None, None] * x.permute(0, 2, 1, 3)
    y = y.permute(0, 2, 1, 3)[live]
    s["out"].copy_(y * _silu(s["z"].float()) if s["z"] is not None else y)
    end = torch.cat([first[1:], first.new_tensor([NC])]) - 1
    s["pool"][s["write"].long()] = (torch.exp(run_[end][..., -1]).float()[..., None, None] * S[end] + add[end]).to(s["pool"].dtype)


def _step(s):
    H, N, P = s["pool"].shape[1:]
    G, T = s["G"], s["T"]
    cu, idx = s["cu"].long(), s["idx"].long()
    B = idx.shape[0]
    n = cu[1:] - cu[:-1]
    t = torch.arange(T, device="cuda")
    live = t < n[:, None]
    rows = (cu[:-1, None] + t).clamp(max=s["xbc"].shape[0] - 1)                  # [B, T]
    i = torch.arange(B, device="cuda")[:, None]
    back = s["acc"].long().clamp(min=1)[:, None] + torch.arange(W - 1, device="cuda")
    past = s["conv_pool"][s["conv_in"].long()[:, None], back]
    ext = torch.cat([past, s["xbc"][rows]], 1)                                   # [B, W-1+T, D]
    w = s["w"].float()
    u = _silu(s["bias"].float() + sum(ext[:, k:k + T].float() * w[:, k] for k in range(W)))
    keep = torch.arange(W - 1 + T, device="cuda") < (W - 1 + n)[:, None]
    new = s["conv_out"].long()
    s["conv_pool"][new] = torch.where(keep[..., None], ext, s["conv_pool"][new])
    x = u[..., :H * P].view(B, T, H, P)
    Bm = u[..., H * P:H * P + G * N].view(B, T, G, N).repeat_interleave(H // G, 2)
    Cm = u[..., H * P + G * N:].view(B, T, G, N).repeat_interleave(H // G, 2)
    step, la = _decay(s["dt"], s["dt_bias"], s["A_log"])
    run_ = la[rows].cumsum(1)                                                    # [B, T, H]
    low = torch.ones(T, T, device="cuda", dtype=torch.bool).tril()
    inside = torch.exp((run_[:, :, None] - run_[:, None, :]).masked_fill(~low[..., None], -math.inf)).float()    # [B, t, s, H]
    S0 = s["pool"][idx.gather(1, (s["acc"].long() - 1).clamp(min=0)[:, None])[:, 0]].float()
    xs = x * step[rows][..., None]
    weight = (inside[..., None] * Bm[:, None]).permute(0, 3, 1, 4, 2)            # [B, H, t, N, s]
    S = (weight.reshape(B, H, T * N, T) @ xs.permute(0, 2, 1, 3)).view(B, H, T, N, P).transpose(1, 2)
    S = S + torch.exp(run_).float()[..., None, None] * S0[:, None]
    y = (Cm[..., None, :] @ S)[..., 0, :] + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"][rows].float())
    s["out"][rows[live]] = y[live].bfloat16()
    s["pool"][idx[live]] = S[live].to(s["pool"].dtype)


# ---- what a pass cannot do without ---------------------------------------------


def work(case):
    op = case["op"]
    if op == "verify":
        size = 4 if case["dtype"] == "f32" else 2
        B, T, V = case["batch"], case["T"], case["vocab"]
        # one target row a request, and the drafter's row where a draft was refused (each is accepted with about 0.81)
        rows = B + sum(1 - 0.81 ** (n - 1) for n in _rows(case)) * case["draft"]
        return {"bytes": rows * V * size + B * T * 24, "flops": 2 * rows * V}
    if op == "tables":
        B, S = case["batch"], case["S"]
        rows = sum(map(sum, _rows(case)))
        return {"bytes": 4 * (B * (14 + 2 * S) + rows), "flops": 4 * B}
    if op == "conv":
        Ntok, D, B = case["tokens"], case["channels"], case["seqs"]
        return {"bytes": 2 * D * (2 * Ntok + 5 + B * (W + W)), "flops": Ntok * D * (2 * W + 5)}
    H, G, P, N = case["H"], case["G"], case["P"], case["N"]
    size = 4 if case["state"] == "f32" else 2
    tile = H * N * P
    if op == "scan":
        Ntok, B = case["tokens"], case["seqs"]
        rows = Ntok * 2 * (H * P * (3 if case["gate"] else 2) + 2 * G * N + H)
        # the token recurrence: the decay, the update and the readout of every state element
        return {"bytes": rows + 1.5 * B * tile * size, "flops": 5 * Ntok * tile}
    B, T = case["batch"], case["T"]
    Ntok = sum(_rows(case))
    D = H * P + 2 * G * N
    rows = Ntok * 2 * (H * P * (2 if case["gate"] else 1) + D + H) + B * 2 * D * (W - 1) + (B * (W - 1) + Ntok) * 2 * D + 10 * D
    return {"bytes": rows + (B + Ntok) * tile * size, "flops": 5 * Ntok * tile + Ntok * D * (2 * W + 5)}


# ---- the definitions in 64 bits --------------------------------------------------


def exact(case, seed):
    s = _inputs(case, seed)
    return {"verify": _exact_verify, "tables": _exact_tables, "conv": _exact_conv, "scan": _exact_scan,
            "step": _exact_step}[case["op"]](s)


def _exact_verify(s):
    cu, T = s["cu"].tolist(), s["T"]
    out, accepted = [], []
    for i in range(len(cu) - 1):
        n, a = cu[i + 1] - cu[i], 0
        while a < n - 1:
            d = int(s["tokens"][i, a])
            q = float(s["draft"][i, a, d]) if s["draft"] is not None else 1.0
            if not float(s["accept_u"][i, a]) * q < float(s["target"][cu[i] + a, d]):
                break
            a += 1
        r = s["target"][cu[i] + a].double()
        if a < n - 1:
            less = torch.zeros_like(r)
            if s["draft"] is not None:
                less = s["draft"][i, a].double()
            else:
                less[int(s["tokens"][i, a])] = 1
            r = (r - less).clamp(min=0) if float((r - less).clamp(min=0).sum()) > 0 else r
        cdf = r.cumsum(0)
        new = int(torch.searchsorted(cdf, s["sample_u"][i].double().view(1) * cdf[-1], right=True).clamp(max=r.numel() - 1))
        row = s["tokens"][i, :a].tolist() + [new]
        out.append(row + [-1] * (T - len(row)))
        accepted.append(a + 1)
    return {"tokens": _i32(out), "accepted": _i32(accepted)}


def _exact_tables(s):
    q, spec, req, S = s["q_lens"].tolist(), s["spec"].tolist(), s["request"].tolist(), s["slots"].shape[1]
    slots, accepted, pair, turn = s["slots"].tolist(), s["accepted"].tolist(), s["conv_table"].tolist(), s["conv_turn"].tolist()
    cu, starts, mine, rest, idx, acc, cin, cout = [0], [0], [], [], [], [], [], []
    for i, r in enumerate(req):
        rows = list(range(starts[-1], starts[-1] + q[i]))
        (mine if spec[i] else rest).extend(rows)
        starts.append(starts[-1] + q[i])
        cu.append(len(mine))
        idx.append(slots[r] if spec[i] else [-1] * S)
        acc.append(accepted[r] if spec[i] else 0)
        cin.append(pair[r][turn[r]] if spec[i] else -1)
        cout.append(pair[r][1 - turn[r]] if spec[i] else -1)
        turn[r] ^= spec[i]
    return {k: _i32(v) for k, v in dict(cu=cu, starts=starts, indx=mine + rest, idx=idx, acc=acc, conv_in=cin, conv_out=cout,
                                        conv_turn=turn).items()}


def _exact_conv(s):
    cu, x, w, pool = s["cu"].tolist(), s["x"].double(), s["w"].double(), s["pool"].double()
    cin, cout, parts = s["conv_in"].tolist(), s["conv_out"].tolist(), []
    for i in range(len(cin)):
        old = s["pool"][cin[i], :W].double() if cin[i] >= 0 else x.new_zeros(W, x.shape[1])
        ext = torch.cat([old, x[cu[i]:cu[i + 1]]])
        y = s["bias"].double() + (ext[1:].unfold(0, W, 1) * w).sum(-1)
        parts.append(y * torch.sigmoid(y))
        pool[cout[i], :W] = ext[-W:]
    return {"y": torch.cat(parts), "pool": pool}


def _exact_scan(s):
    cu, H, G = s["cu"].tolist(), s["x"].shape[1], s["B"].shape[1]
    out, pool = torch.zeros_like(s["out"], dtype=torch.float64), s["pool"].double()
    dt = F.softplus(s["dt"].double() + s["dt_bias"].double())
    keep = torch.exp(-torch.exp(s["A_log"].double()) * dt)
    read, write = s["read"].tolist(), s["write"].tolist()
    # all prompts advance together, token by token
    lens = [cu[i + 1] - cu[i] for i in range(len(read))]
    order = sorted(range(len(read)), key=lambda i: -lens[i])
    base = torch.tensor([cu[i] for i in order], device="cuda")
    S = torch.stack([s["pool"][read[i]].double() if read[i] >= 0 else torch.zeros_like(pool[0]) for i in order])
    live = len(order)
    for t in range(lens[order[0]]):
        while lens[order[live - 1]] <= t:
            live -= 1
        r = base[:live] + t
        x, Bt, Ct = s["x"][r].double(), s["B"][r].double(), s["C"][r].double()
        Bt, Ct = (v[:, :, None].expand(-1, -1, H // G, -1).reshape(live, H, -1) for v in (Bt, Ct))
        now = S[:live]
        now.mul_(keep[r][..., None, None]).addcmul_(Bt[..., None], (dt[r][..., None] * x)[..., None, :])
        out[r] = torch.einsum("bhn,bhnp->bhp", Ct, now) + s["D"].double()[:, None] * x
    if s["z"] is not None:
        z = s["z"].double()
        out *= z * torch.sigmoid(z)
    for k, i in enumerate(order):
        pool[write[i]] = S[k]
    return {"out": out, "pool": pool}


def _exact_step(s):
    cu, acc, idx, G = s["cu"].tolist(), s["acc"].tolist(), s["idx"].tolist(), s["G"]
    H, N, P = s["pool"].shape[1:]
    out, pool, conv = torch.zeros_like(s["out"], dtype=torch.float64), s["pool"].double(), s["conv_pool"].double()
    dt = F.softplus(s["dt"].double() + s["dt_bias"].double())
    keep = torch.exp(-torch.exp(s["A_log"].double()) * dt)
    w, cin, cout = s["w"].double(), s["conv_in"].tolist(), s["conv_out"].tolist()
    for i in range(len(acc)):
        a, n = max(acc[i], 1), cu[i + 1] - cu[i]
        ext = torch.cat([s["conv_pool"][cin[i], a:a + W - 1], s["xbc"][cu[i]:cu[i + 1]]]).double()
        conv[cout[i], :W - 1 + n] = ext
        u = s["bias"].double() + (ext.unfold(0, W, 1) * w).sum(-1)
        u = u * torch.sigmoid(u)
        S = s["pool"][idx[i][a - 1]].double()
        for t in range(n):
            r = cu[i] + t
            x = u[t, :H * P].view(H, P)
            Bt, Ct = (v.view(G, 1, N).expand(G, H // G, N).reshape(H, N) for v in (u[t, H * P:H * P + G * N], u[t, H * P + G * N:]))
            S = S * keep[r][:, None, None] + Bt[..., None] * (dt[r][:, None] * x)[:, None]
            out[r] = (Ct[..., None] * S).sum(1) + s["D"].double()[:, None] * x
            pool[idx[i][t]] = S
    if s["z"] is not None:
        z = s["z"].double()
        out *= z * torch.sigmoid(z)
    return {"out": out, "pool": pool, "conv_pool": conv}
