"""The key-value cache beside the recurrent layers, as measured cases.

A hybrid model's full attention layers need, in the same serving loop as
gdn_spec_decode: the step's (or the prompts') keys and values written into a
paged cache, quantised where it has 8 bits (gdn_kv_write), cached rows read back
(gdn_kv_read), and the attention of a step's one to eight tokens over the cache
(gdn_attn_decode).

listed() and draw() give cases, prepare() their inputs on the GPU, run() one
pass: in elementary torch operations, or with ``own`` through this package.
exact() is each operator's definition in 64 bits, sequence by sequence.
"""
import math
import random

import torch

own = False

CACHE = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LEAST = 2.0 ** -100         # the least scale of an 8-bit row


# ---- cases -------------------------------------------------------------------
# H query heads over G key-value heads of D elements; `page` positions a page;
# `keys` is the longest context of the batch, `ragged` spreads the others below it


def listed():
    return [
        # write: one new token of each of 32 sequences, and the next rows of nine ragged prompts into an 8-bit cache,
        # read back for the prompt's own attention
        dict(name="write b32 t1 bf16", op="write", seqs=32, rows=32, ragged=False, keys=2000, G=8, D=128, page=16, cache="bf16"),
        dict(name="write 9 prompts e4m3", op="write", seqs=9, rows=16211, ragged=True, keys=1000, G=8, D=128, page=64, cache="e4m3"),
        # read: a short shared prefix, and the cached prefixes of six conversations
        dict(name="read 2x300 int8", op="read", seqs=2, rows=600, ragged=False, keys=400, G=2, D=256, page=16, cache="int8"),
        dict(name="read 6 ragged e4m3", op="read", seqs=6, rows=120007, ragged=True, keys=64000, G=8, D=128, page=64, cache="e4m3"),
        # attention: an interactive session's token; an ordinary batch; many short sequences of a model without shared heads
        dict(name="attend b1 t1 777 d256", op="attend", batch=1, T=1, keys=777, ragged=False, H=16, G=2, D=256, page=16,
             cache="bf16", window=0, gate=True),
        dict(name="attend b32 t1 4096", op="attend", batch=32, T=1, keys=4096, ragged=True, H=32, G=8, D=128, page=16,
             cache="bf16", window=0, gate=False),
        dict(name="attend b256 t1 500 g8 d64", op="attend", batch=256, T=1, keys=500, ragged=True, H=8, G=8, D=64, page=32,
             cache="f16", window=0, gate=False),
        # a few very long contexts in 8 bits
        dict(name="attend b4 t1 131072 e4m3", op="attend", batch=4, T=1, keys=131072, ragged=False, H=32, G=8, D=128, page=64,
             cache="e4m3", window=0, gate=False),
        # drafted tokens: three with a sliding window, four over long ragged contexts, eight in a large 8-bit batch, and
        # eight of two long documents
        dict(name="attend b64 t3 w1024 int8", op="attend", batch=64, T=3, keys=8000, ragged=True, H=24, G=4, D=128, page=48,
             cache="int8", window=1024, gate=False),
        dict(name="attend b16 t4 16384 d256", op="attend", batch=16, T=4, keys=16384, ragged=True, H=16, G=2, D=256, page=544,
             cache="bf16", window=0, gate=True),
        dict(name="attend b32 t8 8192 e4m3", op="attend", batch=32, T=8, keys=8192, ragged=False, H=32, G=4, D=128, page=64,
             cache="e4m3", window=0, gate=False),
        dict(name="attend b2 t8 65535 d256", op="attend", batch=2, T=8, keys=65535, ragged=False, H=16, G=2, D=256, page=128,
             cache="bf16", window=0, gate=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    R, G = rng.choice([1, 2, 3, 4, 6, 8, 16]), rng.choice([1, 2, 4, 8])
    common = dict(op=op, G=G, D=rng.choice([64, 128, 128, 192, 256]), page=rng.choice([16, 16, 32, 48, 64, 128, 544, 7]),
                  cache=rng.choice(["bf16", "f16", "e4m3", "int8"]))
    if op != "attend":
        seqs = _log(rng, 1, 200)
        wide = G * common["D"]
        return dict(seqs=seqs, rows=_log(rng, seqs, max(seqs, min(2 ** 26 // wide, 100000))), ragged=rng.random() < 0.7,
                    keys=_log(rng, 1, max(1, min(2 ** 27 // (wide * seqs), 20000))), **common)
    T = rng.choice([1, 1, 2, 3, 4, 5, 6, 7, 8])
    batch = _log(rng, 1, 256)
    size = 2 if common["cache"] in ("bf16", "f16") else 1
    # no more bytes and products than the largest listed
    most = min(2 ** 30 // (batch * G * common["D"] * 2 * size), 2 ** 35 // (batch * T * R * G * common["D"] * 4), 131072)
    return dict(batch=batch, T=T, keys=_log(rng, 1, max(most, 16)), ragged=rng.random() < 0.7, H=R * G,
                window=rng.choice([0, 0, 0, 100, 1024]), gate=rng.random() < 0.4, **common)


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


def _sizes(case):
    """Rows of this call and cached positions of each sequence: the same numbers for every seed."""
    rng = random.Random(case["keys"])
    if case["op"] == "attend":
        B, T, most = case["batch"], case["T"], case["keys"]
        rows = [rng.randint(1, T) if case["ragged"] and i else T for i in range(B)]
        # positions before the step: with the step's own, `keys` at most
        past = [max(0, (rng.randint(most // 4, most) if case["ragged"] and i else most) - rows[i]) for i in range(B)]
        return rows, past
    rows = _lengths(case["rows"], case["seqs"], case["ragged"], case["rows"])
    return rows, [rng.randint(0, case["keys"]) for _ in rows]


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _quantise(x, dtype):
    """Values a scale apart and scales of rows (the last axis)."""
    most = x.abs().amax(-1, keepdim=True)
    if dtype == torch.float8_e4m3fn:
        m, e = torch.frexp(most.clamp(min=LEAST))                                # most = m 2^e, 448 = 0.875 2^9
        scale = torch.ldexp(torch.ones_like(most), e - 9 + (m > 0.875).int()).clamp(min=LEAST)
        return (x / scale).to(dtype), scale[..., 0]
    # up to the next value of eight significant bits
    scale = (((most / 127).view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32).clamp(min=LEAST)
    return torch.round(x / scale).to(dtype), scale[..., 0]


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        s["call"] = _call(s)        # marshalled once, as a serving loop keeps it
    return s


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kw = dict(generator=g, device="cuda")
    G, D, page, dtype = case["G"], case["D"], case["page"], CACHE[case["cache"]]
    rows, past = _sizes(case)
    order = list(range(len(rows)))
    random.Random(seed).shuffle(order)
    rows, past = [rows[i] for i in order], [past[i] for i in order]
    cu, B, N = _offsets(rows), len(rows), sum(rows)
    need = [-(-(p + n) // page) for p, n in zip(past, rows)]
    pages = sum(need) + 3
    perm = torch.randperm(pages, **kw).int()
    cols = torch.arange(max(need), device="cuda")
    first, count = _i32(_offsets(need)[:-1]).long(), _i32(need).long()
    at = (first[:, None] + cols).clamp(max=pages - 1)
    table = torch.where(cols < count[:, None], perm[at], -1).int()
    s = dict(case=case, table=table, past=_i32(past), cu=_i32(cu), page=page, k_scale=None, v_scale=None,
             lens=_i32([p + n for p, n in zip(past, rows)]), longest=max(p + n for p, n in zip(past, rows)))
    for name in ("k", "v"):
        # keys and values with the channels that stand out in such caches
        loud = 1 + 3 * (torch.rand(G, D, **kw) < 0.02).float()
        cache = torch.empty(pages, page, G, D, device="cuda", dtype=dtype)
        scale = torch.empty(pages, page, G, device="cuda") if dtype.itemsize == 1 else None
        for a in range(0, pages, 1 + 2 ** 27 // (page * G * D)):
            b = min(pages, a + 1 + 2 ** 27 // (page * G * D))
            x = (torch.randn(b - a, page, G, D, **kw) * loud).bfloat16()
            if scale is None:
                cache[a:b] = x.to(dtype)
            else:
                cache[a:b], scale[a:b] = _quantise(x.float(), dtype)
        s[name + "_cache"], s[name + "_scale"] = cache, scale
        if case["op"] == "write":
            s[name] = (torch.randn(N, G, D, **kw) * loud).bfloat16()
        if case["op"] != "attend":
            s[name + "_out"] = torch.empty(N, G, D, device="cuda", dtype=torch.bfloat16)
    if case["op"] == "read":                                                    # positions from the middle of each sequence
        s["begin"] = _i32([p // 2 for p in past])
    if case["op"] == "attend":
        H = case["H"]
        s.update(q=(torch.randn(N, H, D, **kw) * 1.5).bfloat16(), T=case["T"], window=case["window"],
                 z=torch.randn(N, H, D, **kw).bfloat16() if case["gate"] else None,
                 out=torch.empty(N, H, D, device="cuda", dtype=torch.bfloat16))
    return s


# ---- one pass ----------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        for call in s["call"]:
            call()
    elif op == "attend":
        _attend(s)
    else:
        if op == "write":
            _write(s)
        if op == "read" or s["k_scale"] is not None:
            _read(s)
    if op == "attend":
        return {"out": s["out"]}
    if op == "read":
        return {"k": s["k_out"], "v": s["v_out"]}
    if s["k_scale"] is None:
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {"k": s["k_out"], "v": s["v_out"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _call(s):
    import gated_deltanet_linear_sm_gb300 as gdn
    op = s["case"]["op"]
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op == "attend":
        return [gdn.prepare_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["past"], s["cu"], s["out"], max_T=s["T"],
                                        z=s["z"], window=s["window"], **scales)]
    calls = []
    if op == "write":
        calls.append(gdn.prepare_kv_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["past"], s["cu"], **scales))
    if op == "read" or s["k_scale"] is not None:
        calls.append(gdn.prepare_kv_read(s["k_cache"], s["v_cache"], s["table"], s["begin"] if op == "read" else s["past"], s["cu"],
                                         s["k_out"], s["v_out"], **scales))
    return calls


# ---- the plain forms ---------------------------------------------------------


def _places(s, begin):
    """Page and place in it of each row of the call, from its sequence's position `begin` on."""
    cu = s["cu"].long()
    row = torch.arange(s["k_out"].shape[0], device="cuda")
    i = torch.searchsorted(cu, row, right=True) - 1
    pos = begin.long()[i] + row - cu[i]
    return s["table"].long()[i, pos // s["page"]], pos % s["page"]


def _write(s):
    page, at = _places(s, s["past"])
    if s["k_scale"] is None:
        s["k_cache"][page, at] = s["k"].to(s["k_cache"].dtype)
        s["v_cache"][page, at] = s["v"].to(s["v_cache"].dtype)
    else:
        for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
            code, scale[page, at] = _quantise(x.float(), cache.dtype)
            cache.view(torch.int8)[page, at] = code.view(torch.int8)


def _read(s):
    page, at = _places(s, s["begin"] if "begin" in s else s["past"])
    s["k_out"].copy_(_values(s, "k", page, at))
    s["v_out"].copy_(_values(s, "v", page, at))


def _values(s, name, page, at):
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    if scale is None:
        return cache[page, at].float()
    return cache.view(torch.int8)[page, at].view(cache.dtype).float() * scale[page, at][..., None]


def _attend(s):
    q, T = s["q"].float(), s["T"]
    cu, past = s["cu"].long(), s["past"].long()
    B, (N, H, D), G = past.shape[0], q.shape, s["k_cache"].shape[2]
    R = H // G
    t = torch.arange(T, device="cuda")
    live = t < (cu[1:] - cu[:-1])[:, None]                                       # [B, T]
    rows = (cu[:-1, None] + t).clamp(max=N - 1)
    pos = past[:, None] + t
    low = (pos - s["window"] + 1).clamp(min=0) if s["window"] else torch.zeros_like(pos)
    # only the positions that some row of the batch sees
    first = low.amin(1)
    width = min(s["longest"], s["window"] + T - 1) if s["window"] else s["longest"]
    x = first[:, None] + torch.arange(width, device="cuda")                      # [B, L]
    seen = (x[:, None] <= pos[..., None]) & (x[:, None] >= low[..., None])       # [B, T, L]
    x = torch.minimum(x, s["lens"].long()[:, None] - 1)
    page = s["table"].long().gather(1, x // s["page"])
    k = _values(s, "k", page, x % s["page"])                                     # [B, L, G, D]
    qs = q[rows].view(B, T, G, R, D).permute(0, 2, 1, 3, 4).reshape(B, G, T * R, D) * D ** -0.5
    score = qs @ k.permute(0, 2, 3, 1)
    del k
    score = score.view(B, G, T, R, -1).masked_fill(~seen[:, None, :, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(B, G, T * R, -1)
    o = p @ _values(s, "v", page, x % s["page"]).permute(0, 2, 1, 3)
    o = o.view(B, G, T, R, D).permute(0, 2, 1, 3, 4).reshape(B, T, H, D)
    if s["z"] is not None:
        o = o / (1 + torch.exp(-s["z"].float()[rows]))
    s["out"][rows[live]] = o[live].bfloat16()


# ---- what a pass cannot do without ---------------------------------------------


def work(case):
    rows, past = _sizes(case)
    N, G, D = sum(rows), case["G"], case["D"]
    cached = 2 * G * (D * CACHE[case["cache"]].itemsize + (4 if case["cache"] in ("e4m3", "int8") else 0))    # a position
    if case["op"] != "attend":
        quantised = case["cache"] in ("e4m3", "int8")
        passes = 2 if case["op"] == "write" and quantised else 1
        tables = 4 * (len(rows) * 2 + sum(-(-n // case["page"]) for n in rows))
        return {"bytes": passes * (N * (cached + 2 * G * D * 2) + tables), "flops": N * 2 * G * D * 2 * passes}
    H, w = case["H"], case["window"]
    keys = sum(min(p + n, w + n - 1) if w else p + n for p, n in zip(past, rows))
    pairs = sum(min(p + t + 1, w) if w else p + t + 1 for p, n in zip(past, rows) for t in range(n))
    tables = 4 * (len(rows) * 2 + keys // case["page"])
    return {"bytes": keys * cached + N * H * D * 2 * (3 if case["gate"] else 2) + tables, "flops": 4 * pairs * H * D}


# ---- the definitions in 64 bits --------------------------------------------------


def exact(case, seed):
    s = _inputs(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)


def _span(s, i, a, b):
    """Where positions a .. b-1 of sequence i are, as flat rows of the cache."""
    x = torch.arange(a, b, device="cuda")
    return s["table"][i].long()[x // s["page"]] * s["page"] + x % s["page"]


def _held(s, name, at):
    cache = s[name + "_cache"]
    v = cache.flatten(0, 1).view(torch.int8 if cache.dtype.itemsize == 1 else torch.int16)[at].view(cache.dtype).double()
    return v if s[name + "_scale"] is None else v * s[name + "_scale"].flatten(0, 1)[at].double()[..., None]


def _nearest_e4m3(v):
    """Multiples of a step: 2^-9 below 2^-6, an eighth of the power of two below the value from there."""
    step = torch.exp2(torch.frexp(v)[1].clamp(min=-5).double() - 4)
    return torch.round(v / step) * step


def _exact_write(s):
    cu, past = s["cu"].tolist(), s["past"].tolist()
    at = torch.cat([_span(s, i, past[i], past[i] + cu[i + 1] - cu[i]) for i in range(len(past))])
    got = {}
    for name in ("k", "v"):
        x = s[name].double()
        if s[name + "_scale"] is None:
            pool = s[name + "_cache"].double()
            pool.flatten(0, 1)[at] = x
            got[name + "_cache"] = pool
            continue
        most = x.abs().amax(-1, keepdim=True)
        if s["case"]["cache"] == "e4m3":
            m, e = torch.frexp(most.clamp(min=LEAST) / 448)                      # itself where it is a power of two, m = 1/2
            scale = torch.exp2((e - (m == 0.5).int()).double()).clamp(min=LEAST)
            held = _nearest_e4m3(x / scale) * scale
        else:
            m, e = torch.frexp(most / 127)
            scale = (torch.ceil(m * 256) * torch.exp2(e.double() - 8)).clamp(min=LEAST)
            held = torch.round(x / scale) * scale
        scales = s[name + "_scale"].double()
        scales.flatten(0, 1)[at] = scale[..., 0]
        got.update({name: held, name + "_scale": scales})
    return got


def _exact_read(s):
    cu, begin = s["cu"].tolist(), s["begin"].tolist()
    at = torch.cat([_span(s, i, begin[i], begin[i] + cu[i + 1] - cu[i]) for i in range(len(begin))])
    return {"k": _held(s, "k", at), "v": _held(s, "v", at)}


def _exact_attend(s):
    cu, past, w = s["cu"].tolist(), s["past"].tolist(), s["window"]
    H, D = s["q"].shape[1:]
    G = s["k_cache"].shape[2]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i in range(len(past)):
        n = cu[i + 1] - cu[i]
        a = max(0, past[i] - w + 1) if w else 0
        at = _span(s, i, a, past[i] + n)
        k, v = _held(s, "k", at), _held(s, "v", at)                              # [L, G, D]
        q = s["q"][cu[i]:cu[i + 1]].double().view(n, G, H // G, D)
        score = torch.einsum("tgrd,lgd->tgrl", q, k) / math.sqrt(D)
        x, pos = torch.arange(a, past[i] + n, device="cuda"), past[i] + torch.arange(n, device="cuda")[:, None]
        hidden = (x > pos) | ((x <= pos - w) if w else (x < 0))
        p = torch.softmax(score.masked_fill(hidden[:, None, None], -math.inf), -1)
        out[cu[i]:cu[i + 1]] = torch.einsum("tgrl,lgd->tgrd", p, v).reshape(n, H, D)
    if s["z"] is not None:
        out *= torch.sigmoid(s["z"].double())
    return {"out": out}
