"""The calls around the step without a GPU: struct layouts, what the C entry
points refuse before anything is launched, what the binding refuses before the
library is reached, and the 64-bit references against closed forms."""
from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from gated_deltanet_linear_sm_gb300 import binding, ops
from gated_deltanet_linear_sm_gb300 import build as gbuild
from tests import ops_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, BAD_SHAPE, UNSUPPORTED, MISALIGNED = 1, 2, 3, 4
A = 0x1000          # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load_library()


@pytest.mark.parametrize("struct", ["gdn_verify_dims", "gdn_tables_dims", "gdn_ssm_dims"])
def test_struct_layout_matches_c(tmp_path, struct):
    mirror = getattr(ops, struct)
    fields = [f for f, _ in mirror._fields_]
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdnspec.h"\nint main(void){\n'
                   f'  printf("%zu\\n", sizeof({struct}));\n'
                   + "".join(f'  printf("%zu\\n", offsetof({struct}, {f}));\n' for f in fields) + "  return 0;\n}\n")
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    vals = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(mirror)
    for f, off in zip(fields, vals[1:]):
        assert getattr(mirror, f).offset == off, f


def _set(struct, base, over):
    for k, v in {**base, **over}.items():
        if k == "reserved":
            struct.reserved[0] = v
        else:
            setattr(struct, k, v)
    return struct


# ---- the C entry points ----------------------------------------------------------


def _verify(lib, ptr=A, dtype=0, dims={}, draft=A, tokens=A, u=A, target=None):
    d = _set(ops.gdn_verify_dims(), dict(batch=2, num_tokens=6, vocab=100, max_T=3), dims)
    return lib.gdn_verify_drafts(ptr if target is None else target, draft, tokens, u, ptr, ptr, None, ptr, ptr,
                                 ctypes.byref(d), dtype, None, None)


@pytest.mark.parametrize("over", [dict(batch=-1), dict(num_tokens=-1), dict(vocab=0), dict(max_T=0), dict(max_T=33),
                                  dict(target_stride=-1), dict(draft_stride=-1), dict(draft_seq=-1), dict(token_stride=-1),
                                  dict(vocab=2 ** 31 - 1), dict(batch=2 ** 30)])
def test_verify_bad_sizes(lib, over):
    assert _verify(lib, dims=over) == BAD_SHAPE


def test_verify_bad_pointers(lib):
    assert _verify(lib, ptr=None) == NULL
    assert _verify(lib, tokens=None) == NULL
    assert _verify(lib, u=None) == NULL
    assert _verify(lib, dtype=3) == UNSUPPORTED
    assert _verify(lib, target=A + 2) == MISALIGNED                     # fp32 rows
    assert _verify(lib, target=A + 1, dtype=1) == MISALIGNED            # bf16 rows need 2 bytes
    assert _verify(lib, tokens=A + 2) == MISALIGNED
    assert _verify(lib, ptr=None, dims=dict(batch=0)) == 0              # nothing to do
    assert lib.gdn_verify_drafts(*([None] * 9), None, 0, None, None) == NULL


def _tables(lib, dims={}, **ptrs):
    d = _set(ops.gdn_tables_dims(), dict(batch=4, num_tokens=9, spec_stride=3, num_requests=8), dims)
    names = ["q", "spec", "request", "slots", "accepted", "pair", "turn", "cu", "starts", "indx", "idx", "acc", "cin", "cout"]
    p = {**{n: A for n in names}, **ptrs}
    return lib.gdn_step_tables(*[p[n] for n in names], ctypes.byref(d), None, None)


@pytest.mark.parametrize("over", [dict(batch=-1), dict(num_tokens=-1), dict(spec_stride=0), dict(num_requests=-1),
                                  dict(spec_stride=2 ** 31 - 1)])
def test_tables_bad_sizes(lib, over):
    assert _tables(lib, over) == BAD_SHAPE


def test_tables_bad_pointers(lib):
    for n in ("q", "slots", "accepted", "cu", "indx", "idx", "acc", "pair", "turn", "cin", "cout"):
        assert _tables(lib, **{n: None}) == NULL, n
    for n in ("q", "spec", "request", "starts", "cout"):
        assert _tables(lib, **{n: A + 2}) == MISALIGNED, n
    assert _tables(lib, dict(batch=9), request=None) == BAD_SHAPE       # more requests than rows of the tables


def _conv(lib, cd={}, x=A, w=A, bias=A, pool=A, y=A, tab=A, batch=2, n=8, dim=64, y_stride=0):
    c = _set(binding.gdn_conv_dims(), dict(width=4, state_len=4, num_conv_slots=3), cd)
    return lib.gdn_conv_prefill(x, w, bias, pool, tab, tab, tab, y, batch, n, dim, y_stride, ctypes.byref(c), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(cd=dict(width=0)), BAD_SHAPE), (dict(cd=dict(width=5)), BAD_SHAPE), (dict(cd=dict(state_len=3)), BAD_SHAPE),
    (dict(cd=dict(num_conv_slots=0)), BAD_SHAPE), (dict(cd=dict(x_stride=-4)), BAD_SHAPE), (dict(cd=dict(reserved=1)), BAD_SHAPE),
    (dict(dim=66), BAD_SHAPE), (dict(dim=0), BAD_SHAPE), (dict(batch=-1), BAD_SHAPE), (dict(n=-1), BAD_SHAPE),
    (dict(y_stride=-4), BAD_SHAPE), (dict(cd=dict(x_stride=66)), MISALIGNED), (dict(y_stride=70), MISALIGNED),
    (dict(x=A + 4), MISALIGNED), (dict(bias=A + 2), MISALIGNED), (dict(tab=A + 1), MISALIGNED), (dict(x=None), NULL),
    (dict(pool=None), NULL), (dict(y=None), NULL), (dict(tab=None), NULL), (dict(w=None), NULL),
    (dict(batch=0, x=None), 0), (dict(n=0, x=None), 0)])
def test_conv_refusals(lib, kw, code):
    assert _conv(lib, **kw) == code


SSM = dict(batch=2, num_tokens=8, H=4, G=2, P=64, N=64, spec_stride=2, max_T=2, num_slots=6)
BAD_SSM = [(dict(batch=-1), BAD_SHAPE), (dict(num_tokens=-1), BAD_SHAPE), (dict(H=0), BAD_SHAPE), (dict(G=3), BAD_SHAPE),
           (dict(G=0), BAD_SHAPE), (dict(num_slots=0), BAD_SHAPE), (dict(dt_stride=-1), BAD_SHAPE), (dict(reserved=1), BAD_SHAPE),
           (dict(N=32), UNSUPPORTED), (dict(N=256), UNSUPPORTED), (dict(P=96), UNSUPPORTED), (dict(P=320), UNSUPPORTED),
           (dict(batch=2 ** 30), BAD_SHAPE)]


def _prefill(lib, dims={}, ptr=A, x=A, z=A, D=A, tab=A, dtype=0, ws=A, ws_bytes=1 << 40):
    d = _set(ops.gdn_ssm_dims(), SSM, dims)
    return lib.gdn_ssm_prefill(x, ptr, ptr, ptr, z, ptr, ptr, D, ptr, tab, tab, ptr, ptr, ws, ws_bytes, ctypes.byref(d), dtype,
                               None, None)


@pytest.mark.parametrize("over,code", BAD_SSM)
def test_ssm_bad_sizes(lib, over, code):
    assert _prefill(lib, over) == code
    assert _decode(lib, over) == code
    d = _set(ops.gdn_ssm_dims(), SSM, over)
    assert lib.gdn_ssm_prefill_workspace(ctypes.byref(d)) == -1


def test_ssm_prefill_refusals(lib):
    assert _prefill(lib, ptr=None) == NULL
    assert _prefill(lib, x=None) == NULL
    assert _prefill(lib, tab=None) == NULL
    assert _prefill(lib, dtype=5) == UNSUPPORTED
    assert _prefill(lib, x=A + 8) == MISALIGNED
    assert _prefill(lib, z=A + 8) == MISALIGNED
    assert _prefill(lib, D=A + 2) == MISALIGNED
    assert _prefill(lib, tab=A + 2) == MISALIGNED
    assert _prefill(lib, dict(x_stride=260)) == MISALIGNED
    assert _prefill(lib, dict(out_stride=260)) == MISALIGNED
    assert _prefill(lib, dict(batch=0), ptr=None) == 0
    assert _prefill(lib, dict(num_tokens=0), ptr=None) == 0


def _decode(lib, dims={}, cd={}, ptr=A, x=A, w=A, bias=A, tab=A, dtype=0):
    d = _set(ops.gdn_ssm_dims(), SSM, dims)
    c = _set(binding.gdn_conv_dims(), dict(width=4, state_len=5, num_conv_slots=3), cd)
    return lib.gdn_ssm_decode(x, w, bias, ptr, tab, tab, ctypes.byref(c), ptr, ptr, ptr, ptr, ptr, ptr, tab, tab, ptr, None, ptr,
                              ctypes.byref(d), dtype, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dims=dict(max_T=0)), BAD_SHAPE), (dict(dims=dict(max_T=9)), BAD_SHAPE), (dict(dims=dict(spec_stride=0)), BAD_SHAPE),
    (dict(cd=dict(width=5)), BAD_SHAPE), (dict(cd=dict(state_len=4)), BAD_SHAPE), (dict(cd=dict(num_conv_slots=0)), BAD_SHAPE),
    (dict(cd=dict(reserved=1)), BAD_SHAPE), (dict(ptr=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL),
    (dict(tab=None), NULL), (dict(dtype=-1), UNSUPPORTED), (dict(x=A + 4), MISALIGNED), (dict(bias=A + 4), MISALIGNED),
    (dict(ptr=A + 8), MISALIGNED), (dict(cd=dict(x_stride=515)), MISALIGNED), (dict(dims=dict(z_stride=258)), MISALIGNED),
    (dict(dims=dict(batch=0), ptr=None), 0)])
def test_ssm_decode_refusals(lib, kw, code):
    assert _decode(lib, **kw) == code


def test_more_rows_than_a_call_takes(lib):
    n = 2 ** 30 + 1
    assert _verify(lib, dims=dict(num_tokens=n)) == BAD_SHAPE
    assert _tables(lib, dict(num_tokens=n)) == BAD_SHAPE
    assert _tables(lib, dict(batch=n, num_requests=n)) == BAD_SHAPE
    assert _conv(lib, n=n) == BAD_SHAPE and _conv(lib, batch=n) == BAD_SHAPE
    assert _prefill(lib, dict(num_tokens=n)) == BAD_SHAPE and _decode(lib, dict(num_tokens=n)) == BAD_SHAPE


# ---- the binding -----------------------------------------------------------------


@pytest.fixture
def no_library(monkeypatch):
    def reached():
        raise AssertionError("the library was reached")
    monkeypatch.setattr(binding, "load_library", reached)


def _i(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _b(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _verify_args(**over):
    d = dict(target_probs=torch.zeros(6, 50), draft_tokens=_i(2, 2), accept_u=torch.zeros(2, 2), sample_u=torch.zeros(2),
             cu_seqlens=_i(3), out_tokens=_i(2, 3), num_accepted=_i(2), draft_probs=torch.zeros(2, 2, 50))
    return {**d, **over}


@pytest.mark.parametrize("over", [dict(target_probs=torch.zeros(50)), dict(draft_tokens=_i(2, 1)), dict(accept_u=torch.zeros(1, 2)),
                                  dict(sample_u=torch.zeros(3)), dict(cu_seqlens=_i(2)), dict(num_accepted=_i(1)),
                                  dict(draft_probs=torch.zeros(2, 2, 49)), dict(draft_probs=torch.zeros(2, 1, 50)),
                                  dict(out_tokens=_i(2))])
def test_verify_sizes_are_refused_before_the_library(no_library, over):
    with pytest.raises(ValueError, match="expected"):
        gdn.gdn_verify_drafts(**_verify_args(**over))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_verify_drafts(**_verify_args())


def test_tables_sizes_are_refused_before_the_library(no_library):
    d = dict(q_lens=_i(3), slot_table=_i(5, 2), cu_seqlens=_i(4), token_indx=_i(6), state_indices=_i(3, 2), num_accepted=_i(3),
             accepted=_i(5), conv_table=_i(5, 2), conv_turn=_i(5), conv_in=_i(3), conv_out=_i(3), spec=_i(3), request=_i(3),
             row_starts=_i(4))
    for k, bad in dict(q_lens=_i(3, 1), slot_table=_i(5), cu_seqlens=_i(3), state_indices=_i(3, 3), num_accepted=_i(2),
                       accepted=_i(4), conv_table=_i(5, 3), conv_turn=_i(3), conv_in=_i(2), conv_out=_i(5), spec=_i(2),
                       request=_i(4), row_starts=_i(3)).items():
        with pytest.raises(ValueError, match="expected"):
            gdn.gdn_step_tables(**{**d, k: bad})
    with pytest.raises(ValueError, match="all be given"):
        gdn.gdn_step_tables(**{**d, "conv_in": None})
    with pytest.raises(ValueError, match="expected slot_table"):
        gdn.gdn_step_tables(**{**d, "request": None, "slot_table": _i(2, 2), "accepted": _i(2), "conv_table": _i(2, 2),
                               "conv_turn": _i(2)})
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_step_tables(**d)


def test_conv_sizes_are_refused_before_the_library(no_library):
    d = dict(x=_b(9, 64), conv_weight=_b(64, 4), conv_bias=_b(64), conv_pool=_b(5, 4, 64), conv_in=_i(2), conv_out=_i(2),
             cu_seqlens=_i(3), y=_b(9, 64))
    for k, bad in dict(x=_b(9, 2, 32), conv_weight=_b(60, 4), conv_bias=_b(32), conv_pool=_b(5, 4, 60), conv_in=_i(3),
                       conv_out=_i(1), cu_seqlens=_i(4), y=_b(8, 64)).items():
        with pytest.raises(ValueError, match="expected"):
            gdn.gdn_conv_prefill(**{**d, k: bad})
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_conv_prefill(**d)


def _layer(N=9, H=4, P=64):
    return dict(dt=_b(N, H), z=_b(N, H, P), A_log=torch.zeros(H), dt_bias=_b(H), D=torch.zeros(H), out=_b(N, H, P),
                state_pool=torch.zeros(3, H, 64, P))


LAYER_BAD = dict(dt=_b(9, 3), z=_b(9, 4, 32), A_log=torch.zeros(3), dt_bias=_b(5), D=torch.zeros(1), out=_b(8, 4, 64))


def test_ssm_prefill_sizes_are_refused_before_the_library(no_library):
    d = dict(x=_b(9, 4, 64), B=_b(9, 2, 64), C=_b(9, 2, 64), read_slots=_i(2), write_slots=_i(2), cu_seqlens=_i(3), **_layer())
    for k, bad in dict(x=_b(9, 256), B=_b(8, 2, 64), C=_b(9, 1, 64), read_slots=_i(2, 1), write_slots=_i(3), cu_seqlens=_i(2),
                       state_pool=torch.zeros(3, 4, 128, 64), **LAYER_BAD).items():
        with pytest.raises(ValueError, match="expected"):
            gdn.gdn_ssm_prefill(**{**d, k: bad})
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_ssm_prefill(**d)


def test_ssm_decode_sizes_are_refused_before_the_library(no_library):
    CD = 4 * 64 + 2 * 2 * 64
    d = dict(xbc=_b(9, CD), conv_weight=_b(CD, 4), conv_bias=_b(CD), conv_pool=_b(5, 5, CD), conv_in=_i(2), conv_out=_i(2),
             state_indices=_i(2, 2), num_accepted=_i(2), cu_seqlens=_i(3), G=2, **_layer())
    for k, bad in dict(xbc=_b(9, CD - 4), conv_weight=_b(CD, 4, 1), conv_bias=_b(4), conv_pool=_b(5, CD), conv_in=_i(1),
                       conv_out=_i(3), state_indices=_i(2), num_accepted=_i(3), cu_seqlens=_i(2), G=3,
                       state_pool=torch.zeros(3, 4, 64), **LAYER_BAD).items():
        with pytest.raises(ValueError, match="expected"):
            gdn.gdn_ssm_decode(**{**d, k: bad})
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_ssm_decode(**d)


def test_row_strides():
    assert ops._rows(_b(5, 4, 8), "t") == 32
    assert ops._rows(_b(5, 40)[:, :32], "t") == 40
    assert ops._rows(_b(5, 6, 8)[:, 2:4], "t") == 48
    assert ops._rows(_b(1, 40)[:, :32], "t") == 32                      # one row: the dense stride
    assert ops._rows(_b(0, 7), "t") == 7
    with pytest.raises(ValueError, match="contiguous"):
        ops._rows(_b(5, 8, 4).transpose(1, 2), "t")
    with pytest.raises(ValueError, match="overlap"):
        ops._rows(_b(1, 8).expand(5, 8), "t")


# ---- the references ----------------------------------------------------------------


def test_reference_sampling_is_the_inverse_distribution():
    """Over a grid of sampling numbers every token appears in proportion, in order."""
    p = np.array([[0.25, 0.0, 0.5, 0.125, 0.125]])
    u = (np.arange(1000) + 0.5) / 1000
    got = [ops_ref.verify(p, None, np.zeros((1, 0), int), None, [x], [[0]], 1)[0][0, 0] for x in u]
    assert np.bincount(got, minlength=5).tolist() == [250, 0, 500, 125, 125] and got == sorted(got)


def test_reference_first_token_has_the_targets_distribution():
    """min(p, q) kept plus the rest resampled is p: summed exactly over drafts, with the acceptance and the
    sampling numbers on grids."""
    p, q = np.array([0.5, 0.25, 0.25, 0.0]), np.array([0.125, 0.25, 0.125, 0.5])
    n = 64
    grid = (np.arange(n) + 0.5) / n
    mass = np.zeros(4)
    for d in range(4):
        for ua in grid:
            for us in grid:
                out, acc, _ = ops_ref.verify(np.stack([p, p]), q[None, None], np.array([[d]]), np.array([[ua]]), [us], [[0, 1]], 2)
                mass[out[0, 0]] += q[d] / n / n
    assert np.allclose(mass, p, atol=1e-12)


def test_reference_layer_step_is_linear_attention_without_decay():
    rng = np.random.default_rng(0)
    H, N, P, T = 2, 5, 3, 6
    B, C, x = rng.normal(size=(T, H, N)), rng.normal(size=(T, H, N)), rng.normal(size=(T, H, P))
    S = M = np.zeros((H, N, P))
    for t in range(T):
        S, M, y, _ = ops_ref.layer_step(S, M, np.ones(H), np.ones(H), B[t], C[t], x[t], np.zeros(H), np.ones((H, P)))
        want = np.einsum("hn,shn,shp->hp", C[t], B[:t + 1], x[:t + 1])
        assert np.allclose(y, want)
    assert (M >= np.abs(S) - 1e-12).all()


def test_reference_tables_of_the_mixed_batch():
    """Speculative and other requests interleaved: the gather of the speculative rows, and the rest behind."""
    slots = np.arange(12).reshape(4, 3)
    t, flags = ops_ref.tables([2, 1, 3, 1], slots, [1, 2, 3, 0], 9, spec=[1, 0, 1, 0])
    assert flags == 0 and t["cu_seqlens"] == [0, 2, 2, 5, 5] and t["row_starts"] == [0, 2, 3, 6, 7]
    assert t["token_indx"] == [0, 1, 3, 4, 5, 2, 6]
    assert t["state_indices"] == [[0, 1, 2], [-1] * 3, [6, 7, 8], [-1] * 3] and t["num_accepted"] == [1, 0, 3, 0]
