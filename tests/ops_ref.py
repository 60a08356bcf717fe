"""Plain 64-bit forms of the calls around the step, from their definitions in
include/gdnspec.h: loops over sequences and tokens, NumPy arrays on the host.
Test infrastructure; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np

UNIT = 2.0 ** 52


def fixed(p):
    """Probabilities as whole multiples of 2^-52 (Python integers)."""
    x = np.asarray(p, dtype=np.float64)
    x = np.where(np.isnan(x), 0.0, np.clip(x, 0.0, 1.0))
    return [int(v) for v in np.rint(x * UNIT)]


def _clamp01(p):
    return 0.0 if math.isnan(p) else min(max(p, 0.0), 1.0)


def verify(target, draft, tokens, accept_u, sample_u, rows, T):
    """rows: the target row of each position, per sequence (None: bad data).
    Returns (out_tokens, num_accepted (-1: left alone), whether a row gave no token)."""
    V = target.shape[1]
    out, accepted, empty = [], [], False
    for i, r in enumerate(rows):
        if not r:
            out.append([-1] * T)
            accepted.append(-1)
            continue
        n, a = len(r) - 1, 0
        while a < n:
            d = int(tokens[i, a])
            if not 0 <= d < V:
                break
            q = _clamp01(float(draft[i, a, d])) if draft is not None else 1.0
            if not float(accept_u[i, a]) * q < _clamp01(float(target[r[a], d])):
                break
            a += 1
        P = fixed(target[r[a]])
        left = P
        if a < n and 0 <= int(tokens[i, a]) < V:
            d = int(tokens[i, a])
            if draft is not None:
                left = [max(x - y, 0) for x, y in zip(P, fixed(draft[i, a]))]
            else:
                left = [0 if v == d else x for v, x in enumerate(P)]
            if sum(left) == 0:
                left = P
        total = sum(left)
        if total == 0:
            new, empty = -1, True
        else:
            x = float(sample_u[i]) * float(total)
            x = 0.0 if math.isnan(x) else max(x, 0.0)
            level = total - 1 if x >= float(total) else min(int(x), total - 1)
            new, run = 0, left[0]
            while run <= level:
                new += 1
                run += left[new]
        out.append([int(t) for t in tokens[i, :a]] + [new] + [-1] * (T - 1 - a))
        accepted.append(a + 1)
    return np.array(out, np.int32).reshape(len(rows), T), np.array(accepted, np.int32), empty


def tables(q_lens, slot_table, accepted, num_tokens, spec=None, request=None, conv_table=None, conv_turn=None):
    """Returns a dict of the tables (token_indx: only its written entries) and the flag bits."""
    R, S = slot_table.shape
    B = len(q_lens)
    flags = 0
    q = [max(int(v), 0) for v in q_lens]
    req = [int(v) for v in (request if request is not None else range(B))]
    mine = []
    for i in range(B):
        if req[i] >= R:
            flags |= 1
            req[i] = -1
        m = (spec is None or spec[i] != 0) and req[i] >= 0
        if m and q[i] > S:
            flags |= 4
            m = False
        mine.append(m)
    if sum(q) > num_tokens:
        flags |= 8
        q, mine = [0] * B, [False] * B
    cu, starts, first, rest = [0], [0], [], []
    idx, acc, cin, cout = [], [], [], []
    turn = None if conv_turn is None else np.array(conv_turn)
    for i in range(B):
        rows = range(starts[-1], starts[-1] + q[i])
        (first if mine[i] else rest).extend(rows)
        starts.append(starts[-1] + q[i])
        cu.append(len(first))
        r = req[i]
        idx.append([int(v) for v in slot_table[r]] if mine[i] else [-1] * S)
        acc.append(int(accepted[r]) if mine[i] else 0)
        if conv_table is not None:
            c = int(turn[r]) & 1 if mine[i] else 0
            cin.append(int(conv_table[r, c]) if mine[i] else -1)
            cout.append(int(conv_table[r, 1 - c]) if mine[i] else -1)
            if mine[i] and q[i] > 0:
                turn[r] = 1 - c
    return dict(cu_seqlens=cu, row_starts=starts, token_indx=first + rest, state_indices=idx, num_accepted=acc,
                conv_in=cin, conv_out=cout, conv_turn=turn), flags


def silu(x):
    with np.errstate(over="ignore", invalid="ignore"):
        return x / (1.0 + np.exp(-x))


def conv_rows(ext, w, bias):
    """silu(bias + taps) for every row of `ext` from row W-1 on, and the sum of
    the absolute terms in front of the silu."""
    W = w.shape[1]
    n = ext.shape[0] - (W - 1)
    a = np.zeros((n, ext.shape[1])) + (0.0 if bias is None else bias)
    m = np.abs(a)
    for k in range(W):
        a = a + ext[k:k + n] * w[:, k]
        m = m + np.abs(ext[k:k + n] * w[:, k])
    return silu(a), m


def layer_step(S, M, a, d, B, C, x, D, zgate):
    """One token for all heads: S, M [H, N, P] (the state, and the sum of the
    absolute values of what makes it up); B, C [H, N]; x [H, P].  Returns the
    new S, M, the output [H, P] and the sum of absolute values behind it."""
    add = B[:, :, None] * (d[:, None] * x)[:, None, :]
    S = S * a[:, None, None] + add
    M = M * a[:, None, None] + np.abs(add)
    y = np.einsum("hn,hnp->hp", C, S) + D[:, None] * x
    my = np.einsum("hn,hnp->hp", np.abs(C), M) + np.abs(D[:, None] * x)
    return S, M, y * zgate, my * np.abs(zgate)


def softplus(x):
    return np.where(x > 20.0, x, np.log1p(np.exp(np.minimum(x, 20.0))))
