"""Python binding of the calls around the step (include/gdnspec.h): draft
verification, the step's tables, the convolution over prompts, and the
state-space layer.  Argument marshalling only, as in binding.py.

Every call has a prepared form (``prepare_...``) that checks and marshals its
arguments once and returns an object to invoke per step, on a given stream or
the current one, directly or while a CUDA graph is captured.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import _STATE_DTYPES, GdnError, gdn_conv_dims

_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32


class gdn_verify_dims(ctypes.Structure):
    """Mirror of gdn_verify_dims in include/gdnspec.h."""

    _fields_ = [
        ("batch", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
        ("vocab", ctypes.c_int32), ("max_T", ctypes.c_int32),
        ("target_stride", ctypes.c_int64), ("draft_stride", ctypes.c_int64),
        ("draft_seq", ctypes.c_int64), ("token_stride", ctypes.c_int64),
    ]


class gdn_tables_dims(ctypes.Structure):
    """Mirror of gdn_tables_dims in include/gdnspec.h."""

    _fields_ = [("batch", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
                ("spec_stride", ctypes.c_int32), ("num_requests", ctypes.c_int32)]


class gdn_ssm_dims(ctypes.Structure):
    """Mirror of gdn_ssm_dims in include/gdnspec.h."""

    _fields_ = [
        ("batch", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
        ("H", ctypes.c_int32), ("G", ctypes.c_int32), ("P", ctypes.c_int32), ("N", ctypes.c_int32),
        ("spec_stride", ctypes.c_int32), ("max_T", ctypes.c_int32), ("num_slots", ctypes.c_int64),
        ("x_stride", ctypes.c_int64), ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64),
        ("dt_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
        ("reserved", ctypes.c_int32 * 2),
    ]


_VP = ctypes.c_void_p
binding.EXPORTS.update({
    "gdn_verify_drafts": (ctypes.c_int, [_VP] * 9 + [ctypes.POINTER(gdn_verify_dims), ctypes.c_int, _VP, _VP]),
    "gdn_verify_drafts_by_request": (ctypes.c_int, [_VP] * 10 + [ctypes.POINTER(gdn_verify_dims), ctypes.c_int32, ctypes.c_int,
                                                                 _VP, _VP]),
    "gdn_step_tables": (ctypes.c_int, [_VP] * 14 + [ctypes.POINTER(gdn_tables_dims), _VP, _VP]),
    "gdn_conv_prefill": (ctypes.c_int, [_VP] * 8 + [ctypes.c_int32] * 3 +
                         [ctypes.c_int64, ctypes.POINTER(gdn_conv_dims), _VP, _VP]),
    "gdn_ssm_prefill": (ctypes.c_int, [_VP] * 14 + [ctypes.c_int64, ctypes.POINTER(gdn_ssm_dims), ctypes.c_int, _VP, _VP]),
    "gdn_ssm_prefill_workspace": (ctypes.c_int64, [ctypes.POINTER(gdn_ssm_dims)]),
    "gdn_ssm_decode": (ctypes.c_int, [_VP] * 6 + [ctypes.POINTER(gdn_conv_dims)] + [_VP] * 11 +
                       [ctypes.POINTER(gdn_ssm_dims), ctypes.c_int, _VP, _VP]),
})


class PreparedOp:
    """A marshalled call; invoking it launches on the given stream (default:
    the current stream of its device).  It keeps its tensors alive; keep it
    while a graph that captured it may be replayed."""

    __slots__ = ("_fn", "_args", "_device", "_index", "_keep")

    def __init__(self, entry, args, device, keep):
        self._fn = getattr(binding.load_library(), entry)
        # converted once: a call only adds the stream handle
        self._args = tuple(t(a) if not isinstance(a, (ctypes._SimpleCData, ctypes.Structure)) else
                           (ctypes.byref(a) if isinstance(a, ctypes.Structure) else a)
                           for a, t in zip(args, self._fn.argtypes))
        self._device = device
        self._index = device.index if device.index is not None else torch.cuda.current_device()
        self._keep = (args, keep)

    def __call__(self, stream=None):
        """Launch on `stream`: a torch.cuda.Stream, a raw cudaStream_t handle
        (int), or None for the current stream."""
        # (the handle and the device without the objects around them: the host's time bounds the
        # smallest calls, 5.2 us each with torch.cuda.current_stream, 3.8 like this)
        if stream is None:
            handle = torch._C._cuda_getCurrentRawStream(self._index)
        else:
            handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
        self._launch(self._args, handle)

    def _launch(self, args, handle):
        if torch._C._cuda_getDevice() == self._index:
            rc = self._fn(*args, handle)
        else:
            with torch.cuda.device(self._index):
                rc = self._fn(*args, handle)
        if rc != 0:
            raise GdnError(rc, binding.status_str(rc))


class PreparedScan(PreparedOp):
    """A prepared gdn_ssm_prefill or gdn_attn_decode whose caller gave no
    workspace: each launch takes one from the memory of the stream that it runs on, where nothing else
    can be given it before the launch has run.  So one such call may run on
    several streams at once and be dropped while it runs, and a graph that
    captures it (through torch.cuda.graph, whose memory that is; a capture
    begun by other means needs a given workspace) holds one of its own."""

    __slots__ = ("_at", "_bytes")

    def __init__(self, entry, args, device, keep, at, nbytes):
        super().__init__(entry, args, device, keep)
        self._at, self._bytes = at, nbytes

    def _launch(self, args, handle):
        workspace = torch.cuda.caching_allocator_alloc(self._bytes, self._index, handle)
        try:
            super()._launch(args[:self._at] + (workspace,) + args[self._at + 1:], handle)
        finally:
            torch.cuda.caching_allocator_delete(workspace)


# ---- checks ------------------------------------------------------------------
# (sizes first, so that no call with a short buffer gets any further; then
# devices, dtypes and layouts)


def _shape(t, name, want):
    """`want`: sizes, with None where any size will do."""
    if t.dim() != len(want) or any(w is not None and w != s for s, w in zip(t.shape, want)):
        sizes = ", ".join("*" if w is None else str(w) for w in want)
        raise ValueError(f"expected {name} [{sizes}]; got {tuple(t.shape)}")


def _int32(**sizes):
    """Sizes that a call takes as 32-bit numbers (ctypes would cut larger ones off)."""
    for name, v in sizes.items():
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"{name} = {v}: a call takes at most 2^31 - 1")


def _dense(dev, **tensors):
    """Contiguous int32 tensors (or None) on the device."""
    for name, t in tensors.items():
        if t is not None:
            binding._check(t, name, _I32, dev)
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")


def _typed(dev, dtype, contiguous=False, **tensors):
    for name, t in tensors.items():
        if t is not None:
            binding._check(t, name, dtype, dev)
            if contiguous and not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")


def _rows(t, name):
    """Elements between rows (dim 0); what is in a row must be dense and rows
    must not overlap."""
    inner = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size > 1 and stride != inner:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        inner *= size
    if t.shape[0] <= 1:
        return inner
    if t.stride(0) < inner:
        raise ValueError(f"{name}: rows overlap")
    return t.stride(0)


def _cuda(dev, entry):
    if dev.type != "cuda":
        raise ValueError(f"{entry} runs on CUDA tensors only")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _pool(pool, dev):
    if pool.dtype not in _STATE_DTYPES:
        raise TypeError(f"state_pool: dtype {pool.dtype} not in fp32 / bf16 / fp16")
    if pool.device != dev or not pool.is_contiguous():
        raise ValueError("state_pool must be a contiguous tensor on the same device")


# ---- gdn_verify_drafts ---------------------------------------------------------


def prepare_verify_drafts(target_probs, draft_tokens, accept_u, sample_u, cu_seqlens, out_tokens, num_accepted, *,
                          draft_probs=None, spec_token_indx=None, request=None, status=None) -> PreparedOp:
    """A prepared gdn_verify_drafts call (see there)."""
    if target_probs.dim() != 2 or out_tokens.dim() != 2 or target_probs.shape[1] < 1 or out_tokens.shape[1] < 1:
        raise ValueError(f"expected target_probs [N, V] and out_tokens [B, T]; got {tuple(target_probs.shape)}, "
                         f"{tuple(out_tokens.shape)}")
    N, V = target_probs.shape
    B, T = out_tokens.shape
    if T > 1:
        for t, n in ((draft_tokens, "draft_tokens"), (accept_u, "accept_u")):
            if t is None or t.dim() != 2 or t.shape[0] != B or t.shape[1] < T - 1:
                raise ValueError(f"expected {n} [B={B}, at least T-1={T - 1}]; got {None if t is None else tuple(t.shape)}")
        if draft_probs is not None and (draft_probs.dim() != 3 or draft_probs.shape[0] != B or
                                        draft_probs.shape[1] < T - 1 or draft_probs.shape[2] != V):
            raise ValueError(f"expected draft_probs [B={B}, at least T-1={T - 1}, V={V}]; got {tuple(draft_probs.shape)}")
    else:
        draft_tokens = accept_u = draft_probs = None
    _shape(sample_u, "sample_u", (B,))
    if request is not None:
        _shape(request, "request", (B,))
    _shape(num_accepted, "num_accepted", (B if request is None else None,))
    _shape(cu_seqlens, "cu_seqlens", (B + 1,))
    _int32(sequences=B, rows=N, vocab=V, T=T, requests=num_accepted.shape[0])
    dev = target_probs.device
    _cuda(dev, "gdn_verify_drafts")
    if target_probs.dtype not in _STATE_DTYPES:
        raise TypeError(f"target_probs: dtype {target_probs.dtype} not in fp32 / bf16 / fp16")
    _typed(dev, target_probs.dtype, draft_probs=draft_probs)
    _typed(dev, _F32, accept_u=accept_u)
    _typed(dev, _F32, contiguous=True, sample_u=sample_u)
    _typed(dev, _I32, draft_tokens=draft_tokens)
    _dense(dev, cu_seqlens=cu_seqlens, spec_token_indx=spec_token_indx, request=request,
           out_tokens=out_tokens, num_accepted=num_accepted, status=status)
    d = gdn_verify_dims()
    d.batch, d.num_tokens, d.vocab, d.max_T = B, N, V, T
    d.target_stride = _rows(target_probs, "target_probs")
    if T > 1:
        d.token_stride = _rows(draft_tokens, "draft_tokens")
        if _rows(accept_u, "accept_u") != d.token_stride and B > 1:    # (one sequence: no stride is used)
            raise ValueError("draft_tokens and accept_u must have the same row stride")
        if draft_probs is not None:
            if V > 1 and draft_probs.stride(2) != 1:
                raise ValueError("draft_probs: the elements of a row must be contiguous")
            # a drafter that runs step by step may stack its rows [T-1, B, V] and pass the transposed view
            d.draft_seq = draft_probs.stride(0) if B > 1 else 0
            d.draft_stride = draft_probs.stride(1) if draft_probs.shape[1] > 1 else 0
            if (B > 1 and d.draft_seq < V) or (draft_probs.shape[1] > 1 and d.draft_stride < V):
                raise ValueError("draft_probs: rows overlap")
    ins = [_ptr(target_probs), _ptr(draft_probs), _ptr(draft_tokens), _ptr(accept_u), _ptr(sample_u), _ptr(cu_seqlens),
           _ptr(spec_token_indx)]
    outs, dtype = [_ptr(out_tokens), _ptr(num_accepted), d], _STATE_DTYPES[target_probs.dtype]
    keep = (target_probs, draft_probs, draft_tokens, accept_u, sample_u, cu_seqlens, spec_token_indx, request, out_tokens,
            num_accepted, status)
    if request is None:
        return PreparedOp("gdn_verify_drafts", ins + outs + [dtype, _ptr(status)], dev, keep)
    return PreparedOp("gdn_verify_drafts_by_request",
                      ins + [_ptr(request)] + outs + [num_accepted.shape[0], dtype, _ptr(status)], dev, keep)


def gdn_verify_drafts(target_probs, draft_tokens, accept_u, sample_u, cu_seqlens, out_tokens, num_accepted, *,
                      draft_probs=None, spec_token_indx=None, request=None, status=None, stream=None):
    """Which drafted tokens the target keeps, and the next token (see
    include/gdnspec.h): target_probs [N, V] fp32 / bf16 / fp16; draft_tokens
    int32 and accept_u fp32 [B, T-1]; sample_u [B] fp32; cu_seqlens [B+1];
    draft_probs [B, T-1, V] of target_probs' dtype, or None for drafts without
    distributions.  Writes out_tokens [B, T] and num_accepted [B] (int32);
    returns both.  With ``request`` [B] (as given to gdn_step_tables)
    num_accepted is that call's ``accepted`` [R] and sequence i's count goes to
    its entry request[i].  With T = 1 the draft arguments are not used."""
    prepare_verify_drafts(target_probs, draft_tokens, accept_u, sample_u, cu_seqlens, out_tokens, num_accepted,
                          draft_probs=draft_probs, spec_token_indx=spec_token_indx, request=request,
                          status=status)(stream)
    return out_tokens, num_accepted


# ---- gdn_step_tables -----------------------------------------------------------


def prepare_step_tables(q_lens, slot_table, cu_seqlens, token_indx, state_indices, num_accepted, *, accepted, spec=None,
                        request=None, row_starts=None, conv_table=None, conv_turn=None, conv_in=None, conv_out=None,
                        status=None) -> PreparedOp:
    """A prepared gdn_step_tables call (see there)."""
    if q_lens.dim() != 1 or slot_table.dim() != 2 or slot_table.shape[1] < 1 or token_indx.dim() != 1:
        raise ValueError(f"expected q_lens [B], slot_table [R, S] and token_indx [N]; got {tuple(q_lens.shape)}, "
                         f"{tuple(slot_table.shape)}, {tuple(token_indx.shape)}")
    B, (R, S) = q_lens.shape[0], slot_table.shape
    conv = (conv_table, conv_turn, conv_in, conv_out)
    if any(t is None for t in conv) and any(t is not None for t in conv):
        raise ValueError("conv_table, conv_turn, conv_in and conv_out must all be given or none")
    if request is None and B > R:
        raise ValueError(f"expected slot_table [R >= B={B}, S] without request; got {tuple(slot_table.shape)}")
    for t, n, want in ((cu_seqlens, "cu_seqlens", (B + 1,)), (state_indices, "state_indices", (B, S)),
                       (num_accepted, "num_accepted", (B,)), (accepted, "accepted", (R,)), (spec, "spec", (B,)),
                       (request, "request", (B,)), (row_starts, "row_starts", (B + 1,)),
                       (conv_table, "conv_table", (R, 2)), (conv_turn, "conv_turn", (R,)), (conv_in, "conv_in", (B,)),
                       (conv_out, "conv_out", (B,))):
        if t is not None:
            _shape(t, n, want)
    _int32(requests=B, rows=token_indx.shape[0], slots_of_a_request=S, request_rows=R)
    dev = q_lens.device
    _cuda(dev, "gdn_step_tables")
    _dense(dev, q_lens=q_lens, slot_table=slot_table, cu_seqlens=cu_seqlens, token_indx=token_indx,
           state_indices=state_indices, num_accepted=num_accepted, accepted=accepted, spec=spec, request=request,
           row_starts=row_starts, conv_table=conv_table, conv_turn=conv_turn, conv_in=conv_in, conv_out=conv_out,
           status=status)
    d = gdn_tables_dims()
    d.batch, d.num_tokens, d.spec_stride, d.num_requests = B, token_indx.shape[0], S, R
    return PreparedOp("gdn_step_tables",
                      [_ptr(q_lens), _ptr(spec), _ptr(request), _ptr(slot_table), _ptr(accepted), _ptr(conv_table),
                       _ptr(conv_turn), _ptr(cu_seqlens), _ptr(row_starts), _ptr(token_indx), _ptr(state_indices),
                       _ptr(num_accepted), _ptr(conv_in), _ptr(conv_out), d, _ptr(status)], dev,
                      (q_lens, spec, request, slot_table, accepted, conv, cu_seqlens, row_starts, token_indx,
                       state_indices, num_accepted, status))


def gdn_step_tables(q_lens, slot_table, cu_seqlens, token_indx, state_indices, num_accepted, *, accepted, spec=None,
                    request=None, row_starts=None, conv_table=None, conv_turn=None, conv_in=None, conv_out=None,
                    status=None, stream=None):
    """The tables of one step from its requests' lengths (see
    include/gdnspec.h); every tensor int32: q_lens [B], slot_table [R, S],
    accepted [R] (by request: see gdn_verify_drafts), optional spec [B], request [B], conv_table [R, 2] and
    conv_turn [R] (updated).  Writes cu_seqlens [B+1], token_indx [N],
    state_indices [B, S], num_accepted [B], and where given row_starts [B+1],
    conv_in and conv_out [B]."""
    prepare_step_tables(q_lens, slot_table, cu_seqlens, token_indx, state_indices, num_accepted, accepted=accepted,
                        spec=spec, request=request, row_starts=row_starts, conv_table=conv_table, conv_turn=conv_turn,
                        conv_in=conv_in, conv_out=conv_out, status=status)(stream)


# ---- gdn_conv_prefill ----------------------------------------------------------


def _conv_dims(conv_weight, conv_bias, conv_pool, conv_in, conv_out, B, D) -> gdn_conv_dims:
    _shape(conv_weight, "conv_weight", (D, None))
    _shape(conv_pool, "conv_pool", (None, None, D))
    if conv_bias is not None:
        _shape(conv_bias, "conv_bias", (D,))
    _shape(conv_in, "conv_in", (B,))
    _shape(conv_out, "conv_out", (B,))
    _int32(width=conv_weight.shape[1], state_len=conv_pool.shape[1])
    cd = gdn_conv_dims()
    cd.width = conv_weight.shape[1]
    cd.num_conv_slots, cd.state_len = conv_pool.shape[0], conv_pool.shape[1]
    return cd


def prepare_conv_prefill(x, conv_weight, conv_bias, conv_pool, conv_in, conv_out, cu_seqlens, y, *,
                         status=None) -> PreparedOp:
    """A prepared gdn_conv_prefill call (see there)."""
    _shape(x, "x", (None, None))
    N, D = x.shape
    _shape(y, "y", (N, D))
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError(f"expected cu_seqlens [B+1]; got {tuple(cu_seqlens.shape)}")
    B = cu_seqlens.shape[0] - 1
    _int32(sequences=B, rows=N, channels=D)
    cd = _conv_dims(conv_weight, conv_bias, conv_pool, conv_in, conv_out, B, D)
    dev = x.device
    _cuda(dev, "gdn_conv_prefill")
    _typed(dev, _BF16, x=x, y=y)
    _typed(dev, _BF16, contiguous=True, conv_weight=conv_weight, conv_bias=conv_bias, conv_pool=conv_pool)
    _dense(dev, conv_in=conv_in, conv_out=conv_out, cu_seqlens=cu_seqlens, status=status)
    cd.x_stride = _rows(x, "x")
    return PreparedOp("gdn_conv_prefill",
                      [_ptr(x), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_pool), _ptr(conv_in), _ptr(conv_out),
                       _ptr(cu_seqlens), _ptr(y), B, N, D, _rows(y, "y"), cd, _ptr(status)], dev,
                      (x, conv_weight, conv_bias, conv_pool, conv_in, conv_out, cu_seqlens, y, status))


def gdn_conv_prefill(x, conv_weight, conv_bias, conv_pool, conv_in, conv_out, cu_seqlens, y, *, status=None,
                     stream=None):
    """The short causal convolution over prompts (see include/gdnspec.h): x, y
    [N, conv_dim] bf16 (rows may be strided), conv_weight [conv_dim, W] bf16,
    conv_bias [conv_dim] bf16 or None, conv_pool [slots, state_len, conv_dim]
    bf16 (slots conv_out written), conv_in, conv_out [B] and cu_seqlens [B+1]
    int32.  Returns ``y``."""
    prepare_conv_prefill(x, conv_weight, conv_bias, conv_pool, conv_in, conv_out, cu_seqlens, y, status=status)(stream)
    return y


# ---- the state-space layer -----------------------------------------------------


def _layer_shapes(N, H, P, dt, z, A_log, dt_bias, D, out):
    for t, n, want in ((dt, "dt", (N, H)), (z, "z", (N, H, P)), (A_log, "A_log", (H,)), (dt_bias, "dt_bias", (H,)),
                       (D, "D", (H,)), (out, "out", (N, H, P))):
        if t is not None:
            _shape(t, n, want)


def _layer_types(dev, dt, z, A_log, dt_bias, D, out, state_pool):
    _typed(dev, _BF16, dt=dt, z=z, out=out)
    _typed(dev, _BF16, contiguous=True, dt_bias=dt_bias)
    _typed(dev, _F32, contiguous=True, A_log=A_log, D=D)
    _pool(state_pool, dev)


def _ssm_dims(B, N, H, G, P, S, state_pool, dt, z, out) -> gdn_ssm_dims:
    d = gdn_ssm_dims()
    d.batch, d.num_tokens, d.H, d.G, d.P, d.N = B, N, H, G, P, S
    d.spec_stride = d.max_T = 1
    d.num_slots = state_pool.shape[0]
    d.dt_stride = _rows(dt, "dt")
    d.z_stride = _rows(z, "z") if z is not None else 0
    d.out_stride = _rows(out, "out")
    return d


def prepare_ssm_prefill(x, B, C, dt, z, A_log, dt_bias, D, state_pool, read_slots, write_slots, cu_seqlens, out, *,
                        workspace=None, status=None) -> PreparedOp:
    """A prepared gdn_ssm_prefill call (see there).  Without ``workspace`` each
    of its launches takes one (PreparedScan); with it, calls on two streams or
    from two graphs must not run at the same time."""
    _shape(x, "x", (None, None, None))
    N, H, P = x.shape
    _shape(B, "B", (N, None, None))
    _shape(C, "C", tuple(B.shape))
    G, S = B.shape[1:]
    _layer_shapes(N, H, P, dt, z, A_log, dt_bias, D, out)
    _shape(state_pool, "state_pool", (None, H, S, P))
    _shape(read_slots, "read_slots", (None,))
    n = read_slots.shape[0]
    _shape(write_slots, "write_slots", (n,))
    _shape(cu_seqlens, "cu_seqlens", (n + 1,))
    _int32(sequences=n, rows=N, H=H, G=G, P=P, S=S)
    dev = x.device
    _cuda(dev, "gdn_ssm_prefill")
    _typed(dev, _BF16, x=x, B=B, C=C)
    _layer_types(dev, dt, z, A_log, dt_bias, D, out, state_pool)
    _dense(dev, read_slots=read_slots, write_slots=write_slots, cu_seqlens=cu_seqlens, status=status)
    d = _ssm_dims(n, N, H, G, P, S, state_pool, dt, z, out)
    d.x_stride, d.b_stride, d.c_stride = _rows(x, "x"), _rows(B, "B"), _rows(C, "C")
    need = ssm_prefill_workspace(d, dev)
    if workspace is not None:
        _typed(dev, torch.uint8, contiguous=True, workspace=workspace)
        if workspace.numel() < need:
            raise ValueError(f"expected workspace of at least {need} bytes; got {workspace.numel()}")
    args = [_ptr(x), _ptr(B), _ptr(C), _ptr(dt), _ptr(z), _ptr(A_log), _ptr(dt_bias), _ptr(D), _ptr(state_pool),
            _ptr(read_slots), _ptr(write_slots), _ptr(cu_seqlens), _ptr(out), _ptr(workspace), need, d,
            _STATE_DTYPES[state_pool.dtype], _ptr(status)]
    keep = (x, B, C, dt, z, A_log, dt_bias, D, state_pool, read_slots, write_slots, cu_seqlens, out, workspace, status)
    if need == 0 or workspace is not None:
        return PreparedOp("gdn_ssm_prefill", args, dev, keep)
    return PreparedScan("gdn_ssm_prefill", args, dev, keep, at=13, nbytes=need)


def ssm_prefill_workspace(dims, device=None) -> int:
    """Bytes of workspace that gdn_ssm_prefill needs for these gdn_ssm_dims on
    the device (default: the current one).  Raises GdnError for invalid sizes."""
    with torch.cuda.device(device):
        need = int(binding.load_library().gdn_ssm_prefill_workspace(ctypes.byref(dims)))
    if need < 0:
        raise GdnError(3, "unsupported sizes of the state-space layer")
    return need


def gdn_ssm_prefill(x, B, C, dt, z, A_log, dt_bias, D, state_pool, read_slots, write_slots, cu_seqlens, out, *,
                    workspace=None, status=None, stream=None):
    """The state-space layer over prompts (see include/gdnspec.h): x, z, out
    [N, H, P] and B, C [N, G, S] bf16 (rows may be strided), dt [N, H] and
    dt_bias [H] bf16, A_log and D [H] fp32 (z and D may be None), state_pool
    [slots, H, S, P] fp32 / bf16 / fp16 (slots write_slots written), read_slots,
    write_slots [B] and cu_seqlens [B+1] int32.  ``workspace``: uint8, at least
    what gdn_ssm_prefill_workspace asks for, used by this call alone until it
    has run (default: each launch takes one on its stream).  Returns ``out``."""
    prepare_ssm_prefill(x, B, C, dt, z, A_log, dt_bias, D, state_pool, read_slots, write_slots, cu_seqlens, out,
                        workspace=workspace, status=status)(stream)
    return out


def prepare_ssm_decode(xbc, conv_weight, conv_bias, conv_pool, conv_in, conv_out, dt, z, A_log, dt_bias, D, state_pool,
                       state_indices, num_accepted, cu_seqlens, out, *, G, spec_token_indx=None, max_T=None,
                       status=None) -> PreparedOp:
    """A prepared gdn_ssm_decode call (see there)."""
    _shape(xbc, "xbc", (None, None))
    _shape(state_pool, "state_pool", (None, None, None, None))
    N, CD = xbc.shape
    H, S, P = state_pool.shape[1:]
    if G < 1 or H % G != 0 or CD != H * P + 2 * G * S:
        raise ValueError(f"expected xbc [N, H P + 2 G N = {H * P + 2 * G * S}] with H a multiple of G; got "
                         f"{tuple(xbc.shape)}, H={H}, G={G}")
    _layer_shapes(N, H, P, dt, z, A_log, dt_bias, D, out)
    _shape(state_indices, "state_indices", (None, None))
    n, stride = state_indices.shape
    _shape(num_accepted, "num_accepted", (n,))
    _shape(cu_seqlens, "cu_seqlens", (n + 1,))
    if max_T is None:
        max_T = min(stride, 8)
    _int32(sequences=n, rows=N, channels=CD, H=H, G=G, P=P, S=S, slots_of_a_sequence=stride, max_T=max_T)
    cd = _conv_dims(conv_weight, conv_bias, conv_pool, conv_in, conv_out, n, CD)
    dev = xbc.device
    _cuda(dev, "gdn_ssm_decode")
    _typed(dev, _BF16, xbc=xbc)
    _typed(dev, _BF16, contiguous=True, conv_weight=conv_weight, conv_bias=conv_bias, conv_pool=conv_pool)
    _layer_types(dev, dt, z, A_log, dt_bias, D, out, state_pool)
    _dense(dev, conv_in=conv_in, conv_out=conv_out, state_indices=state_indices, num_accepted=num_accepted,
           cu_seqlens=cu_seqlens, spec_token_indx=spec_token_indx, status=status)
    d = _ssm_dims(n, N, H, G, P, S, state_pool, dt, z, out)
    d.spec_stride = stride
    d.max_T = max_T
    cd.x_stride = _rows(xbc, "xbc")
    return PreparedOp("gdn_ssm_decode",
                      [_ptr(xbc), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_pool), _ptr(conv_in), _ptr(conv_out), cd,
                       _ptr(dt), _ptr(z), _ptr(A_log), _ptr(dt_bias), _ptr(D), _ptr(state_pool), _ptr(state_indices),
                       _ptr(num_accepted), _ptr(cu_seqlens), _ptr(spec_token_indx), _ptr(out), d,
                       _STATE_DTYPES[state_pool.dtype], _ptr(status)], dev,
                      (xbc, conv_weight, conv_bias, conv_pool, conv_in, conv_out, dt, z, A_log, dt_bias, D, state_pool,
                       state_indices, num_accepted, cu_seqlens, spec_token_indx, out, status))


def gdn_ssm_decode(xbc, conv_weight, conv_bias, conv_pool, conv_in, conv_out, dt, z, A_log, dt_bias, D, state_pool,
                   state_indices, num_accepted, cu_seqlens, out, *, G, spec_token_indx=None, max_T=None, status=None,
                   stream=None):
    """The state-space layer over one to eight tokens of each sequence, with
    the convolution and the rewind in front (see include/gdnspec.h): xbc
    [N, H P + 2 G S] bf16 projection rows (channels x | B | C), the conv
    tensors as for gdn_spec_decode_conv, the layer's as for gdn_ssm_prefill,
    state_indices [B, spec_stride], num_accepted [B] and cu_seqlens [B+1]
    int32.  Returns ``out``."""
    prepare_ssm_decode(xbc, conv_weight, conv_bias, conv_pool, conv_in, conv_out, dt, z, A_log, dt_bias, D, state_pool,
                       state_indices, num_accepted, cu_seqlens, out, G=G, spec_token_indx=spec_token_indx, max_T=max_T,
                       status=status)(stream)
    return out
