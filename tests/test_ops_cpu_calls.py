"""Further refusals of the calls around the step, without a GPU: the C entry
points before anything is launched, the binding before the library is reached."""
from __future__ import annotations

import ctypes

import pytest
import torch

import gated_deltanet_linear_sm_gb300 as gdn
from gated_deltanet_linear_sm_gb300 import ops
from tests.test_ops_cpu import (A, BAD_SHAPE, MISALIGNED, NULL, UNSUPPORTED, _i, _set, _verify_args, lib,  # noqa: F401
                                no_library)


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
