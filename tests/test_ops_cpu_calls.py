"""Further refusals of the calls around the step, without a GPU: the C entry
points before anything is launched, the binding before the library is reached."""
from __future__ import annotations

import ctypes

import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from gated_deltanet_linear_sm_gb300 import ops
from tests.test_ops_cpu import (A, BAD_SHAPE, MISALIGNED, NULL, UNSUPPORTED, _conv, _i, _set, _tables,  # noqa: F401
                                _verify_args, lib, no_library)


def _by_request(lib, dims={}, request=A, counts=A, num_requests=4, dtype=0):
    d = _set(ops.gdn_verify_dims(), dict(batch=2, num_tokens=6, vocab=100, max_T=3), dims)
    return lib.gdn_verify_drafts_by_request(A, A, A, A, A, A, None, request, A, counts, ctypes.byref(d), num_requests, dtype, None,
                                            None)


def test_verify_by_request_refusals(lib):  # noqa: F811
    assert _by_request(lib, request=None) == NULL
    assert _by_request(lib, counts=None) == NULL
    assert _by_request(lib, request=A + 2) == MISALIGNED
    assert _by_request(lib, num_requests=-1) == BAD_SHAPE
    assert _by_request(lib, dict(max_T=33)) == BAD_SHAPE
    assert _by_request(lib, dtype=3) == UNSUPPORTED
    assert _by_request(lib, dict(batch=0), request=None) == 0           # nothing to do
    assert lib.gdn_verify_drafts_by_request(*([None] * 10), None, 0, 0, None, None) == NULL


def test_verify_by_request_sizes_are_refused_before_the_library(no_library):  # noqa: F811
    args = _verify_args(request=_i(2), num_accepted=_i(9))
    for bad in (dict(request=_i(3)), dict(request=_i(2, 1)), dict(num_accepted=_i(9, 1))):
        with pytest.raises(ValueError, match="expected"):
            gdn.gdn_verify_drafts(**{**args, **bad})
    with pytest.raises(ValueError, match="CUDA"):                       # as many counts as there are requests
        gdn.gdn_verify_drafts(**args)


@pytest.mark.parametrize("name", ["draft_tokens", "accept_u"])
def test_verify_without_its_drafts_is_refused(no_library, name):  # noqa: F811
    with pytest.raises(ValueError, match=f"expected {name}"):
        gdn.gdn_verify_drafts(**_verify_args(**{name: None}))


@pytest.mark.parametrize("dim", [2 ** 30 + 4, 2 ** 31 - 1020, 2 ** 31 - 4])
def test_conv_of_more_channels_than_it_counts(lib, dim):  # noqa: F811
    """The last CTA's channel numbers would pass 31 bits."""
    assert _conv(lib, dim=dim) == BAD_SHAPE


def test_more_sequences_than_each_cta_can_look_at(lib):  # noqa: F811
    n = 2 ** 20 + 1
    assert _tables(lib, dict(batch=n, num_requests=n)) == BAD_SHAPE
    assert _conv(lib, batch=n) == BAD_SHAPE


# ---- sizes that do not fit the 32 bits of the C structs (tensors without memory) ----

BIG = 2 ** 32 + 5


def _m(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def _mi(*shape):
    return _m(*shape, dtype=torch.int32)


def _too_large(call, **args):
    with pytest.raises(ValueError, match="at most 2\\^31 - 1"):
        call(**args)


@pytest.mark.parametrize("B,N,V,T,R", [(BIG, 6, 50, 3, 4), (2, BIG, 50, 3, 4), (2, 6, BIG, 3, 4), (2, 6, 50, BIG, 4), (2, 6, 50, 3, BIG)])
def test_verify_sizes_beyond_32_bits(no_library, B, N, V, T, R):  # noqa: F811
    _too_large(gdn.gdn_verify_drafts, target_probs=_m(N, V), draft_tokens=_mi(B, T - 1), accept_u=_m(B, T - 1, dtype=torch.float32),
               sample_u=_m(B, dtype=torch.float32), cu_seqlens=_mi(B + 1), out_tokens=_mi(B, T), num_accepted=_mi(R),
               request=_mi(B))


@pytest.mark.parametrize("B,N,S,R", [(BIG, 6, 2, 3), (3, BIG, 2, 3), (3, 6, BIG, 3), (3, 6, 2, BIG)])
def test_tables_sizes_beyond_32_bits(no_library, B, N, S, R):  # noqa: F811
    _too_large(gdn.gdn_step_tables, q_lens=_mi(B), slot_table=_mi(R, S), cu_seqlens=_mi(B + 1), token_indx=_mi(N),
               state_indices=_mi(B, S), num_accepted=_mi(B), accepted=_mi(R), request=_mi(B))


@pytest.mark.parametrize("B,N,D,L", [(BIG, 9, 64, 4), (2, BIG, 64, 4), (2, 9, BIG, 4), (2, 9, 64, BIG)])
def test_conv_sizes_beyond_32_bits(no_library, B, N, D, L):  # noqa: F811
    _too_large(gdn.gdn_conv_prefill, x=_m(N, D), conv_weight=_m(D, 4), conv_bias=None, conv_pool=_m(3, L, D), conv_in=_mi(B),
               conv_out=_mi(B), cu_seqlens=_mi(B + 1), y=_m(N, D))


@pytest.mark.parametrize("n,N,H,G,P,S", [(BIG, 9, 4, 2, 64, 64), (2, BIG, 4, 2, 64, 64), (2, 9, BIG, 1, 64, 64),
                                         (2, 9, 4, BIG, 64, 64), (2, 9, 4, 2, BIG, 64), (2, 9, 4, 2, 64, BIG)])
def test_ssm_sizes_beyond_32_bits(no_library, n, N, H, G, P, S):  # noqa: F811
    f = torch.float32
    layer = dict(dt=_m(N, H), z=None, A_log=_m(H, dtype=f), dt_bias=_m(H), D=None, state_pool=_m(3, H, S, P, dtype=f),
                 out=_m(N, H, P), cu_seqlens=_mi(n + 1))
    _too_large(gdn.gdn_ssm_prefill, x=_m(N, H, P), B=_m(N, G, S), C=_m(N, G, S), read_slots=_mi(n), write_slots=_mi(n), **layer)
    if H % G == 0:
        CD = H * P + 2 * G * S
        _too_large(gdn.gdn_ssm_decode, xbc=_m(N, CD), conv_weight=_m(CD, 4), conv_bias=None, conv_pool=_m(5, 5, CD),
                   conv_in=_mi(n), conv_out=_mi(n), state_indices=_mi(n, 2), num_accepted=_mi(n), G=G, **layer)


def test_ssm_decode_max_T_beyond_32_bits(no_library):  # noqa: F811
    CD, f = 4 * 64 + 2 * 2 * 64, torch.float32
    _too_large(gdn.gdn_ssm_decode, xbc=_m(9, CD), conv_weight=_m(CD, 4), conv_bias=None, conv_pool=_m(5, 5, CD), conv_in=_mi(2),
               conv_out=_mi(2), state_indices=_mi(2, 2), num_accepted=_mi(2), G=2, dt=_m(9, 4), z=None, A_log=_m(4, dtype=f),
               dt_bias=_m(4), D=None, state_pool=_m(3, 4, 64, 64, dtype=f), out=_m(9, 4, 64), cu_seqlens=_mi(3), max_T=2 ** 32 + 1)
