"""The key-value cache's calls without a GPU: the struct's layout, what the C entry
points refuse before anything is launched, what the binding refuses before the
library is reached, and the 64-bit references against closed forms."""
from __future__ import annotations

import ctypes
import math
import os
import subprocess

import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from gated_deltanet_linear_sm_gb300 import kv
from tests import kv_ref as ref
from tests.test_ops_cpu import A, BAD_SHAPE, MISALIGNED, NULL, ROOT, UNSUPPORTED, _set, lib, no_library  # noqa: F401

BF16, F16, E4M3, I8 = 1, 2, 3, 4
BASE = dict(batch=2, num_tokens=6, H_q=8, H_kv=2, D=128, page_size=16, table_cols=4, max_T=3, num_pages=10)


def test_struct_layout_matches_c(tmp_path):
    mirror = kv.gdn_kv_dims
    fields = [f for f, _ in mirror._fields_]
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdnspec.h"\nint main(void){\n'
                   '  printf("%zu\\n", sizeof(gdn_kv_dims));\n'
                   + "".join(f'  printf("%zu\\n", offsetof(gdn_kv_dims, {f}));\n' for f in fields) + "  return 0;\n}\n")
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    vals = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert vals == [ctypes.sizeof(mirror)] + [getattr(mirror, f).offset for f in fields]


def _dims(over):
    d = kv.gdn_kv_dims()
    for k, v in {**BASE, **over}.items():
        setattr(d, k, v)
    return d


def _call(lib, which, dims={}, kind=E4M3, row=BF16, scale=0.1, ws=A, ws_bytes=1 << 40, **ptrs):  # noqa: F811
    names = {"write": ["k", "v", "kc", "vc", "ks", "vs", "table", "lens", "cu", "sti"],
             "read": ["kc", "vc", "ks", "vs", "table", "lens", "cu", "k", "v"],
             "attn": ["q", "kc", "vc", "ks", "vs", "table", "lens", "cu", "sti", "z", "out"]}[which]
    p = [({n: A for n in names} | ptrs)[n] for n in names]
    d = ctypes.byref(_dims(dims))
    if which == "write":
        return lib.gdn_kv_write(*p, d, kind, None, None)
    if which == "read":
        return lib.gdn_kv_read(*p, d, kind, row, None, None)
    return lib.gdn_attn_decode(*p, ws, ws_bytes, d, scale, kind, None, None)


CALLS = ["write", "read", "attn"]


@pytest.mark.parametrize("which", CALLS)
@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), BAD_SHAPE), (dict(num_tokens=-1), BAD_SHAPE), (dict(batch=2 ** 20 + 1), BAD_SHAPE), (dict(num_tokens=2 ** 30 + 1), BAD_SHAPE),
    (dict(H_kv=0), BAD_SHAPE), (dict(H_kv=4097, H_q=4097), BAD_SHAPE), (dict(D=0), BAD_SHAPE), (dict(D=96), UNSUPPORTED),
    (dict(D=512), UNSUPPORTED), (dict(page_size=0), BAD_SHAPE), (dict(table_cols=0), BAD_SHAPE), (dict(num_pages=0), BAD_SHAPE),
    (dict(reserved=1), BAD_SHAPE), (dict(page_stride=-16), BAD_SHAPE), (dict(scale_token_stride=-1), BAD_SHAPE), (dict(table_stride=-1), BAD_SHAPE),
    (dict(page_size=2 ** 16, table_cols=2 ** 15), BAD_SHAPE), (dict(page_size=2 ** 31 - 1), BAD_SHAPE),
    (dict(page_stride=2 ** 20 + 8), MISALIGNED), (dict(token_stride=264), MISALIGNED), (dict(head_stride=136), MISALIGNED)])
def test_sizes_that_every_call_refuses(lib, which, over, code):  # noqa: F811
    assert _call(lib, which, over) == code


@pytest.mark.parametrize("which", CALLS)
def test_types_that_are_refused(lib, which):  # noqa: F811
    for kind in (0, 5, -1):
        assert _call(lib, which, kind=kind) == UNSUPPORTED
    if which == "read":
        for row in (E4M3, I8, 7):
            assert _call(lib, which, row=row) == UNSUPPORTED


def test_no_other_call_takes_the_cache_types(lib):  # noqa: F811
    from gated_deltanet_linear_sm_gb300 import binding, ops
    from tests.test_boundary_cpu import _call as spec_call
    from tests.test_boundary_cpu import _dims as spec_dims
    for t in (E4M3, I8):
        assert spec_call(lib, spec_dims(), state_dtype=t) == UNSUPPORTED
        P = [A] * 14
        assert lib.gdn_prefill(*P, ctypes.byref(spec_dims()), 0.1, 1e-5, t, None, None) == UNSUPPORTED
        assert lib.gdn_prefill_chunked(*P, ctypes.byref(spec_dims()), 0.1, 1e-5, t, None, None) == UNSUPPORTED
        d = _set(ops.gdn_verify_dims(), dict(batch=2, num_tokens=6, vocab=100, max_T=3), {})
        assert lib.gdn_verify_drafts(A, A, A, A, A, A, None, A, A, ctypes.byref(d), t, None, None) == UNSUPPORTED
        s = _set(ops.gdn_ssm_dims(), dict(batch=2, num_tokens=4, H=4, G=2, P=64, N=64, spec_stride=2, max_T=2, num_slots=4), {})
        c = _set(binding.gdn_conv_dims(), dict(width=4, state_len=5, num_conv_slots=3), {})
        assert lib.gdn_ssm_prefill(*[A] * 14, 1 << 40, ctypes.byref(s), t, None, None) == UNSUPPORTED
        assert lib.gdn_ssm_decode(*[A] * 6, ctypes.byref(c), *[A] * 11, ctypes.byref(s), t, None, None) == UNSUPPORTED


@pytest.mark.parametrize("which,need", [("write", ["k", "v", "kc", "vc", "ks", "vs", "table", "lens", "cu"]),
                                        ("read", ["k", "v", "kc", "vc", "ks", "vs", "table", "cu"]),
                                        ("attn", ["q", "kc", "vc", "ks", "vs", "table", "lens", "cu", "out"])])
def test_pointers(lib, which, need):  # noqa: F811
    for n in need:
        assert _call(lib, which, **{n: None}) == NULL, n
        assert _call(lib, which, **{n: A + (2 if n in ("ks", "vs", "table", "lens", "cu") else 8)}) == MISALIGNED, n
    assert _call(lib, which, dict(batch=0), **{n: None for n in need}) == 0
    assert _call(lib, which, dict(num_tokens=0), **{n: None for n in need}) == 0
    for over in (dict(k_stride=260), dict(v_stride=260)) if which != "attn" else (dict(q_stride=1028), dict(out_stride=1028), dict(z_stride=4)):
        assert _call(lib, which, over) == MISALIGNED
    if which == "attn":
        assert _call(lib, which, ws=None) == NULL
        assert _call(lib, which, ws=A + 8) == MISALIGNED
        need_bytes = lib.gdn_attn_decode_workspace(ctypes.byref(_dims({})), E4M3)
        assert need_bytes > 0 and _call(lib, which, ws_bytes=need_bytes - 1) == BAD_SHAPE
    with_none = {"write": lib.gdn_kv_write, "read": lib.gdn_kv_read}.get(which)
    if which == "write":
        assert with_none(*[A] * 10, None, E4M3, None, None) == NULL
    if which == "read":
        assert with_none(*[A] * 9, None, E4M3, BF16, None, None) == NULL


@pytest.mark.parametrize("over", [dict(H_q=0), dict(H_q=7), dict(H_q=4098), dict(max_T=0), dict(max_T=9), dict(window=-1), dict(q_stride=-8),
                                  dict(batch=2 ** 20, table_cols=2 ** 26, H_q=4096)])
def test_attention_sizes(lib, over):  # noqa: F811
    assert _call(lib, "attn", over) == BAD_SHAPE
    assert lib.gdn_attn_decode_workspace(ctypes.byref(_dims(over)), E4M3) == -1


def test_attention_scale_and_workspace(lib):  # noqa: F811
    for scale in (math.nan, math.inf):
        assert _call(lib, "attn", scale=scale) == BAD_SHAPE
    assert lib.gdn_attn_decode_workspace(ctypes.byref(_dims({})), 0) == -1
    assert lib.gdn_attn_decode_workspace(ctypes.byref(_dims(dict(batch=0))), BF16) == 0
    assert lib.gdn_attn_decode_workspace(None, BF16) == -1


# ---- the binding -------------------------------------------------------------------


def _b(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _i(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


CACHE = dict(k_cache=_b(5, 16, 2, 64), v_cache=_b(5, 16, 2, 64), page_table=_i(3, 4), cu_seqlens=_i(4))
BAD_CACHE = dict(k_cache=_b(5, 16, 128), v_cache=_b(5, 16, 2, 128), page_table=_i(2, 4), cu_seqlens=_i(4, 1))
CALLS_OF = {
    gdn.gdn_kv_write: (dict(k=_b(9, 2, 64), v=_b(9, 2, 64), kv_lens=_i(3), **CACHE),
                       dict(k=_b(9, 3, 64), v=_b(8, 2, 64), kv_lens=_i(4), **BAD_CACHE)),
    gdn.gdn_kv_read: (dict(k=_b(9, 2, 64), v=_b(9, 2, 64), kv_begin=_i(3), **CACHE),
                      dict(k=_b(9, 2, 128), v=_b(9, 1, 64), kv_begin=_i(2), **BAD_CACHE)),
    gdn.gdn_attn_decode: (dict(q=_b(9, 8, 64), out=_b(9, 8, 64), z=_b(9, 8, 64), kv_lens=_i(3), max_T=2, **CACHE),
                          dict(q=_b(9, 7, 64), out=_b(9, 4, 64), z=_b(9, 8, 128), kv_lens=_i(4), **BAD_CACHE)),
}


@pytest.mark.parametrize("call", CALLS_OF, ids=lambda c: c.__name__)
def test_sizes_are_refused_before_the_library(no_library, call):  # noqa: F811
    d, bad = CALLS_OF[call]
    for k, v in bad.items():
        with pytest.raises(ValueError, match="expected"):
            call(**{**d, k: v})
    for over in (dict(k_scale=torch.zeros(5, 16, 2)), dict(v_scale=torch.zeros(5, 16, 2)), dict(page_table=_i(3, 0)),
                 dict(k_cache=_b(0, 16, 2, 64), v_cache=_b(0, 16, 2, 64))):
        with pytest.raises(ValueError, match="expected"):
            call(**{**d, **over})
    small = dict(k_cache=d["k_cache"].to(torch.int8), v_cache=d["v_cache"].to(torch.int8))
    for scales in (dict(), dict(k_scale=torch.zeros(5, 16, 2)), dict(k_scale=torch.zeros(5, 16, 2), v_scale=torch.zeros(5, 16))):
        with pytest.raises(ValueError, match="expected"):
            call(**{**d, **small, **scales})
    with pytest.raises(TypeError, match="k_cache"):
        call(**{**d, "k_cache": d["k_cache"].float()})
    with pytest.raises(ValueError, match="CUDA"):
        call(**d)


def test_head_dims_that_are_refused(no_library):  # noqa: F811
    d, _ = CALLS_OF[gdn.gdn_kv_write]
    wide = {k: _b(*v.shape[:-1], 96) for k, v in d.items() if v.dtype == torch.bfloat16}
    with pytest.raises(ValueError, match="head dim"):
        gdn.gdn_kv_write(**{**d, **wide})


def test_sizes_beyond_32_bits(no_library):  # noqa: F811
    big = 2 ** 31
    d, _ = CALLS_OF[gdn.gdn_attn_decode]
    for k in ("max_T", "window"):
        with pytest.raises(ValueError, match=k):
            gdn.gdn_attn_decode(**{**d, k: big})
    rows = torch.empty(1, dtype=torch.bfloat16).expand(big, 8, 64)
    with pytest.raises(ValueError, match="rows"):
        gdn.gdn_attn_decode(**{**d, "q": rows, "out": rows, "z": rows})
    rows = torch.empty(1, dtype=torch.bfloat16).expand(big, 2, 64)
    d, _ = CALLS_OF[gdn.gdn_kv_write]
    with pytest.raises(ValueError, match="rows"):
        gdn.gdn_kv_write(**{**d, "k": rows, "v": rows})


def test_cache_strides():
    k = _b(5, 16, 2, 64)
    assert kv._strides(k, k, "k", 3) == [2048, 128, 64]
    h = _b(5, 2, 16, 64).transpose(1, 2)
    assert kv._strides(h, h, "k", 3) == [2048, 64, 1024]
    both = _b(5, 2, 16, 2, 64)
    assert kv._strides(both[:, 0], both[:, 1], "k", 3) == [4096, 128, 64]
    one = _b(5, 16, 1, 64)
    assert kv._strides(one, one, "k", 3)[:2] == [1024, 64]
    assert all(s % 16 == 0 and s > 0 for s in kv._strides(one, one, "k", 3))
    with pytest.raises(ValueError, match="same strides"):
        kv._strides(k, h, "k", 3)
    with pytest.raises(ValueError, match="overlap"):
        t = _b(1, 16, 2, 64).expand(5, 16, 2, 64)
        kv._strides(t, t, "k", 3)
    with pytest.raises(ValueError, match="overlap"):
        t = _b(100000).as_strided((5, 16, 2, 64), (1024, 64, 64, 1))
        kv._strides(t, t, "k", 3)


# ---- the references ------------------------------------------------------------------


def test_reference_quantisation():
    """Half a step at most off; the scales are what the header says; e4m3 as torch rounds it."""
    g = torch.Generator().manual_seed(0)
    for size in (1e-3, 1.0, 300.0):
        x = (torch.randn(256, generator=g) * size).bfloat16().double()
        a = float(x.abs().max())
        code, s = ref.quantise(x, "int8")
        assert a / 127 <= s < a / 127 * (1 + 2.0 ** -7) and float((code * s - x).abs().max()) <= s / 2 and float(code.abs().max()) <= 127
        code, s = ref.quantise(x, "e4m3")
        assert math.log2(s) == int(math.log2(s)) and a <= 448 * s < 2 * a
        assert torch.equal(code, (x / s).float().to(torch.float8_e4m3fn).double())
        assert bool(((code * s - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10 * s, dtype=torch.float64))).all())
    assert ref.quantise(torch.zeros(4, dtype=torch.float64), "int8")[1] == ref.LEAST
    assert ref.quantise(torch.zeros(4, dtype=torch.float64), "e4m3")[1] == ref.LEAST
    assert math.isnan(ref.quantise(torch.tensor([1.0, math.inf], dtype=torch.float64), "int8")[1])


def test_reference_attention_of_equal_keys_is_the_mean():
    v = torch.arange(12, dtype=torch.float64).view(3, 2, 2)
    q, k = torch.ones(4, 2), torch.ones(3, 2, 2, dtype=torch.float64)
    out, A, B, S = ref.attend(q, k, v, torch.tensor([True, False, True]), 0.5)
    assert torch.equal(out, torch.tensor([[4.0, 5], [4, 5], [6, 7], [6, 7]], dtype=torch.float64)) and torch.equal(A, out)
    assert B == 1.0 and S == 1.0
    assert float(ref.attend(q, k, v, torch.zeros(3, dtype=torch.bool), 0.5)[0].abs().max()) == 0
