/*
 * libgdnspec -- the speculative / MTP decode step of a Gated DeltaNet (GDN)
 * linear-attention layer, as hand-written CUDA for sm_103a (GB300), behind a
 * plain C ABI.
 *
 * The operation follows these vLLM pull-request report pages:
 *   "PR #51674 report -- [Kernel][Perf] Add fused CUDA post-conv MTP decode
 *    kernel for Qwen3.5 GDN", implementation steps 1-3 and the
 *    _custom_ops.py listing (one fused step per (request, v-head): rewind to
 *    the last accepted state slot, up to 8 draft tokens through the gated
 *    delta rule in order, gated RMSNorm epilogue; scale = 128^-0.5,
 *    norm_eps = 1e-5; K = V = 128; the state is updated in place);
 *   "PR #46090 report -- [CPU][Spec Decode] Support DFlash speculative
 *    decoding for GDN models on CPU", implementation step 3 and the fla.cpp
 *    listing (initial slot spec_indices[i, max(num_accepted-1, 0)], the
 *    state after every token written to its own slot, q_len <= 0 skipped,
 *    v-head h uses key head h / (H_v / H_k));
 *   "PR #52191 report -- [CPU] Support FP16/BF16 persisted GDN state on
 *    AMX", implementation steps 3-4 (arithmetic in FP32, the state stored as
 *    FP32 / BF16 / FP16 with one rounding per slot write);
 *   "PR #51812 report -- [Bugfix] Align Qwen GDN gates with speculative
 *    tokens", implementation steps 1-3 (q/k/v and the a/b gates gathered with
 *    one shared spec_token_indx in a mixed batch).
 *
 * Per (sequence i, v-head h), with S the K x V state (V contiguous) and
 * r(t) the token row of draft token t:
 *     S <- state_pool[state_indices[i, max(num_accepted[i]-1, 0)], h]
 *     for t in 0 .. q_len-1:
 *         g = -exp(A_log[h]) * softplus(a[r,h] + dt_bias[h]);  beta = sigmoid(b[r,h])
 *         k^ = k[r,kh] / |k[r,kh]|;  q^ = q[r,kh] / |q[r,kh]| * scale
 *         S <- S e^g;  v' = beta (v[r,h] - S^T k^);  S <- S + k^ v'^T;  o = S^T q^
 *         if state_indices[i, t] >= 0: state_pool[state_indices[i, t], h] <- round(S)
 *         out[r,h] = round_bf16( o * rsqrt(mean(o^2) + eps) * norm_w * silu(z[r,h]) )
 * (softplus(x) = x above 20; |x| = sqrt(sum x^2 + 1e-6).)
 *
 * Everything here is asynchronous on the caller's stream: the library never
 * synchronises, never reads device data on the host and allocates nothing, so
 * a call can be captured in a CUDA graph.  All tensor pointers are
 * caller-owned DEVICE memory (for example PyTorch tensors); the library keeps
 * no pointer after the call returns.
 */
#ifndef GDNSPEC_H
#define GDNSPEC_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* 2: gdn_spec_decode_split takes the state dtype; dims->split accepts GDN_SPLIT_NARROW
   3: dims->flags (formerly reserved): GDN_PRE_INDEX, GDN_PRE_TOKENS, GDN_PRE_STATE
   4: dims->split accepts GDN_SPLIT_HALFK | 1 and | 2, the automatic choice for small
      FP32 batches
   5: gdn_verify_drafts, gdn_step_tables, gdn_conv_prefill, gdn_ssm_prefill, gdn_ssm_decode
      and GDN_FLAG_NO_TOKEN
   6: gdn_verify_drafts_by_request
   7: gdn_kv_write, gdn_kv_read, gdn_attn_decode, GDN_E4M3 and GDN_I8 (their caches' types; no
      other call takes these two) */
#define GDNSPEC_VERSION 7

#if defined(__GNUC__)
#define GDNSPEC_API __attribute__((visibility("default")))
#else
#define GDNSPEC_API
#endif

/* Host-side result of a call.  Nothing is launched unless GDN_OK. */
typedef enum {
    GDN_OK = 0,
    GDN_ERR_NULL_ARG = 1,    /* a required pointer is NULL, or z / norm_w not both set */
    GDN_ERR_BAD_SHAPE = 2,   /* negative sizes, H_v % H_k != 0, spec_stride < 1, max_T outside 1..8, ... */
    GDN_ERR_UNSUPPORTED = 3, /* K != 128, V != 128, unknown state dtype, bad split */
    GDN_ERR_MISALIGNED = 4,  /* a pointer or row stride breaks the alignment rules below */
    GDN_ERR_CUDA = 5         /* the launch failed (the CUDA error is left for the caller to query) */
} gdn_status;

/* Element type of the recurrent-state pool (the first three), or of a key-value cache (the
 * last four; with GDN_E4M3 and GDN_I8 every head's row has a scale). */
typedef enum { GDN_F32 = 0, GDN_BF16 = 1, GDN_F16 = 2, GDN_E4M3 = 3, GDN_I8 = 4 } gdn_dtype;

/*
 * Bits the kernel ORs into *status_word (when given) for bad DEVICE data.
 * The offending sequence (or, for a bad write slot, just that slot write) is
 * skipped; nothing traps and nothing waits.
 */
#define GDN_FLAG_SLOT_RANGE 1  /* a read or write slot >= num_slots (read: sequence skipped; write: that write skipped) */
#define GDN_FLAG_ACCEPTED   2  /* num_accepted[i] > spec_stride: sequence skipped */
#define GDN_FLAG_QLEN       4  /* q_len > max_T or q_len > spec_stride: sequence skipped */
#define GDN_FLAG_TOKEN_ROW  8  /* a token row outside [0, num_tokens), or cu_seqlens[i] < 0 or
                                  cu_seqlens[i+1] > cu_seqlens[batch]: sequence skipped */
#define GDN_FLAG_TIMEOUT    16 /* gdn_prefill_chunked, gdn_ssm_prefill and gdn_attn_decode only: a wait on
                                  the tensor cores ran past its bound (gdn_set_wait_limit); that sequence's
                                  outputs and final state are incomplete (gdn_attn_decode: the call's) */
#define GDN_FLAG_DRAIN      32 /* the same three only: after such a timeout, the wait (with the
                                  default bound) for the products still in flight ran out too; the
                                  CTA released its tensor memory regardless, since holding it would
                                  block every later kernel on that SM */
#define GDN_FLAG_NO_TOKEN   64 /* gdn_verify_drafts only: what is left to sample from (r there) counts
                                  as 0 throughout, or sums to 16 or more: no token was emitted */

/*
 * dims->split flag: each warp of the decode step owns 8 of a unit's 128 V
 * columns instead of 16, so a unit runs on 16 warps with half the state per
 * lane and half the work per token.  Meant for small batches, where most SMs
 * would otherwise idle: the unit's warps spread over a 2- or 4-CTA cluster.
 * Same results up to FP32 rounding order.
 */
#define GDN_SPLIT_NARROW 0x100

/*
 * dims->split flag (GDN_SPLIT_HALFK | 1 or | 2): each warp keeps 16 V columns
 * but only half of their 128 K rows, the two warps of a column block adding
 * their partial products through shared memory once per token, so its
 * tensor stores keep the 16-column rows.  A unit's 16 warps run in one CTA
 * (| 1) or over a 2-CTA cluster (| 2, half of a unit's work per SM).  Meant
 * for small batches.  Same results up to FP32 rounding order.
 */
#define GDN_SPLIT_HALFK 0x200

/*
 * dims->flags: what the caller promises about the kernel launched on the
 * stream immediately before this call.  Each decode launch lets the next
 * launch on the stream start its CTAs while it finishes (programmatic
 * dependent launch); a CTA then waits for its predecessor to complete before
 * it touches memory that the predecessor may have written.  With these flags
 * it reads some inputs before that wait, which hides their latency behind the
 * predecessor's tail:
 *   GDN_PRE_INDEX   state_indices, num_accepted, cu_seqlens and
 *                   spec_token_indx were not written by the preceding kernel
 *                   (for example: they were filled at the start of the step);
 *   GDN_PRE_TOKENS  with GDN_PRE_INDEX: neither were q, k, v, a, b, z, A_log,
 *                   dt_bias and norm_w (for example: the batch's inputs are
 *                   resident and the preceding kernel is another decode step);
 *   GDN_PRE_STATE   with GDN_PRE_INDEX: nor were the state slots this call
 *                   reads (the rewound slots).  True in a model's forward
 *                   pass, where the kernel before a layer's step is never that
 *                   layer's own step; false for two steps of one layer in a
 *                   row where the second rewinds into the first's slots.
 * out, status_word and every slot write are accessed after the wait; without
 * GDN_PRE_STATE so is the state read, so back-to-back steps that rewind into
 * each other's slots stay ordered.  A
 * decode launch signals its successor only after its own wait, so when the
 * preceding kernel is one of this library's decode launches, or a kernel that
 * does not use programmatic dependent launch, every kernel before it has
 * completed when the early reads happen.
 * For gdn_spec_decode_conv, GDN_PRE_STATE also covers the conv slots the call
 * reads (its conv history), and the token prologue, which convolves that
 * history, runs early only with both GDN_PRE_TOKENS and GDN_PRE_STATE set.
 * The prefill entry points take no flags.
 */
#define GDN_PRE_INDEX  0x1
#define GDN_PRE_TOKENS 0x2
#define GDN_PRE_STATE  0x4

/* Opaque CUDA stream handle; the same type as cudaStream_t (NULL = legacy default stream). */
typedef struct CUstream_st* gdn_stream_t;

/* Sizes.  All host-side integers: the launch shape never depends on device data. */
typedef struct {
    int32_t batch;        /* number of speculative sequences (rows of state_indices) */
    int32_t num_tokens;   /* rows of q, k, v, a, b, z and out */
    int32_t H_k, H_v;     /* key heads and value heads; H_v % H_k == 0 (the tuned case is H_v = 8 H_k) */
    int32_t K, V;         /* head dims; both must be 128 */
    int32_t spec_stride;  /* columns of state_indices (>= every q_len) */
    int32_t max_T;        /* host-known bound on every q_len, 1..8 */
    int64_t num_slots;    /* slots in state_pool */
    /* Row strides between consecutive tokens, in ELEMENTS; 0 selects the dense
       default (q, k: H_k*K; v, z, out: H_v*V; a, b: H_v).  Within a row the
       heads are contiguous.  A packed mixed_qkv tensor [N, 2*H_k*K + H_v*V]
       is passed as three pointers into it with q_stride = k_stride =
       v_stride = 2*H_k*K + H_v*V. */
    int64_t q_stride, k_stride, v_stride, a_stride, b_stride, z_stride, out_stride;
    int32_t split;        /* CTAs per (sequence, v-head), one thread-block cluster:
                             0 = chosen from the batch size; else 1, 2, 4 or 8
                             (each warp owns 16 V columns), GDN_SPLIT_NARROW
                             | 2 or | 4 (each warp owns 8 V columns: 16 warps
                             per unit over 2 or 4 CTAs), or GDN_SPLIT_HALFK | 1
                             or | 2 (16 columns and half the K rows per warp:
                             16 warps per unit in 1 or 2 CTAs) */
    int32_t flags;        /* 0, or GDN_PRE_INDEX [| GDN_PRE_TOKENS] [| GDN_PRE_STATE] (above); 0 for prefill */
} gdn_dims;

/*
 * gdn_spec_decode -- one speculative decode step over a batch.
 *
 * Arguments (device pointers unless stated; element types fixed):
 *   q, k            bf16 [num_tokens, H_k, K]  (row stride q_stride / k_stride)
 *   v               bf16 [num_tokens, H_v, V]  (row stride v_stride)
 *   a, b            bf16 [num_tokens, H_v]     (row strides a_stride, b_stride)
 *   z               bf16 [num_tokens, H_v, V] output gate, or NULL
 *   A_log           fp32 [H_v]
 *   dt_bias         bf16 [H_v]
 *   norm_w          bf16 [V] gated-RMSNorm weight, or NULL.  z and norm_w are
 *                   both NULL or both set; with both NULL no epilogue runs
 *                   and out holds the raw readout o.
 *   state_pool      state_dtype [num_slots, H_v, K, V], V contiguous; read
 *                   and written in place
 *   state_indices   int32 [batch, spec_stride]; -1 marks a padded slot
 *   num_accepted    int32 [batch]; values < 1 read position 0
 *   cu_seqlens      int32 [batch + 1]; q_len_i = cu_seqlens[i+1] - cu_seqlens[i]
 *   spec_token_indx int32 [cu_seqlens[batch]] token row of every spec token,
 *                   or NULL when the spec tokens are rows cu_seqlens[i] + t
 *   out             bf16 [num_tokens, H_v, V] (row stride out_stride);
 *                   written only at the rows of active spec tokens, other
 *                   rows keep the caller's contents (zero-fill them first if
 *                   padded rows flow onward, as under CUDA graphs)
 *   dims            HOST pointer, read during the call only
 *   scale           query scale (128^-0.5 in the pages' default)
 *   eps             RMSNorm epsilon (1e-5 in the pages' default)
 *   state_dtype     GDN_F32, GDN_BF16 or GDN_F16
 *   status_word     device int32 that receives GDN_FLAG_* bits, or NULL
 *   stream          CUDA stream to launch on
 *
 * Skips: q_len <= 0, or a read slot < 0 (a padded sequence), write nothing
 * for that sequence.  A write slot < 0 skips only that write.
 *
 * Caller contract (not checked on the device): non-negative write slots are
 * distinct across the batch; no sequence reads a slot that another sequence
 * writes; token rows are used by at most one spec token.
 *
 * Alignment: state_pool 16 bytes; q, k, v, z, out, norm_w 8 bytes with
 * q/k/v/z/out row strides multiples of 4 elements; int32 tables 4 bytes.
 * Size limit: num_slots * H_v * K < 2^31 (the slot writes address the pool
 * as one 2-D tensor with 32-bit row coordinates); beyond it the call returns
 * GDN_ERR_UNSUPPORTED.  The call encodes that tensor's description on the
 * host the first time it sees a pool (cached per host thread for the last 4
 * pools); no device memory is allocated.
 */
GDNSPEC_API gdn_status gdn_spec_decode(
    const void* q, const void* k, const void* v,
    const void* a, const void* b, const void* z,
    const float* A_log, const void* dt_bias, const void* norm_w,
    void* state_pool,
    const int32_t* state_indices, const int32_t* num_accepted,
    const int32_t* cu_seqlens, const int32_t* spec_token_indx,
    void* out,
    const gdn_dims* dims, float scale, float eps, gdn_dtype state_dtype,
    int32_t* status_word, gdn_stream_t stream);

/*
 * gdn_prefill -- the same gated delta rule over whole prompts: the prefill
 * path whose state is carried across the prompt and written back to its slot
 * ("PR #52191 report -- [CPU] Support FP16/BF16 persisted GDN state on AMX",
 * implementation steps 3-4: arithmetic in FP32, the slot written in the pool
 * dtype, rounded once).
 *
 * Sequence i is token rows cu_seqlens[i] .. cu_seqlens[i+1]-1, in order (no
 * gather).  It starts from slot read_slots[i], or from the zero state when
 * read_slots[i] < 0; every token writes its output row (with the gated RMSNorm
 * epilogue when z / norm_w are given); the state after its last token goes to
 * slot write_slots[i] (no write when negative).  read_slots[i] ==
 * write_slots[i] updates a slot in place.
 *
 *   read_slots, write_slots   int32 [batch] (device)
 *   every other argument       as for gdn_spec_decode; dims->spec_stride,
 *                              max_T and split are not used
 *
 * Caller contract: non-negative write slots are distinct; no sequence reads a
 * slot that another sequence writes.  Bad device data skips the sequence:
 * a slot >= num_slots sets GDN_FLAG_SLOT_RANGE, rows outside [0, num_tokens)
 * set GDN_FLAG_TOKEN_ROW.  Asynchronous on `stream`, allocates nothing.
 */
GDNSPEC_API gdn_status gdn_prefill(
    const void* q, const void* k, const void* v,
    const void* a, const void* b, const void* z,
    const float* A_log, const void* dt_bias, const void* norm_w,
    void* state_pool,
    const int32_t* read_slots, const int32_t* write_slots,
    const int32_t* cu_seqlens,
    void* out,
    const gdn_dims* dims, float scale, float eps, gdn_dtype state_dtype,
    int32_t* status_word, gdn_stream_t stream);

/*
 * gdn_prefill_chunked -- what gdn_prefill computes, in the chunked form that
 * runs on the tensor cores: the prompt is cut into chunks of 64 tokens and the
 * per-token recurrence inside a chunk is unrolled into dense products
 * ("PR #52191 report", implementation steps 3-4: the inter-chunk recurrence
 * kernel with all products and the exp(g_last) rescale in FP32 buffers).
 * With G_t the running sum of the log-decays g inside the chunk, S the state
 * at its start and k^, q^ the normalised rows:
 *     (I + A) V' = B,  A_ts = beta_t e^(G_t - G_s) k^_t.k^_s (s < t),
 *                      B_t  = beta_t (v_t - e^(G_t) S^T k^_t)
 *     o_t = e^(G_t) S^T q^_t + sum_{s <= t} e^(G_t - G_s) (q^_t.k^_s) v'_s
 *     S  <- e^(G_last) S + sum_s e^(G_last - G_s) k^_s v'_s^T
 * which is the same quantity as the token recurrence, in exact arithmetic.
 * The products run on the tensor cores at FP32 accuracy: each operand is
 * carried as a bf16 hi part and a bf16 lo part (hi + lo within 2^-18 of the
 * FP32 value) and the hi.hi, lo.hi and hi.lo products accumulate in FP32; the
 * carried state, the triangular solve and the epilogue are FP32.  The state
 * is rounded to the pool dtype once, when it is stored at the end of the
 * prompt.
 *
 * Arguments, layouts, the caller contract and the status bits are those of
 * gdn_prefill; in addition GDN_FLAG_TIMEOUT reports a tensor-core wait that
 * ran past its bound.  One CTA per (sequence, v-head) unit, holding the
 * whole 512-column tensor memory of its SM (~218 KiB of shared memory); with
 * fewer units than half the device's SMs, two CTAs per unit as a cluster,
 * each with 64 of the value columns (~210 KiB of shared memory each).  The
 * results do not depend on which form runs beyond FP32 rounding order.
 * Asynchronous on `stream`, allocates nothing.
 */
GDNSPEC_API gdn_status gdn_prefill_chunked(
    const void* q, const void* k, const void* v,
    const void* a, const void* b, const void* z,
    const float* A_log, const void* dt_bias, const void* norm_w,
    void* state_pool,
    const int32_t* read_slots, const int32_t* write_slots,
    const int32_t* cu_seqlens,
    void* out,
    const gdn_dims* dims, float scale, float eps, gdn_dtype state_dtype,
    int32_t* status_word, gdn_stream_t stream);

/* Sizes of the short causal convolution in front of the step (gdn_spec_decode_conv). */
typedef struct {
    int32_t width;          /* taps W, 1..4 */
    int32_t state_len;      /* rows per conv slot; >= W - 1 + spec_stride */
    int64_t num_conv_slots; /* slots in conv_pool */
    int64_t x_stride;       /* elements between rows of x; 0 = conv_dim (dense); multiple of 4 */
    int32_t reserved[2];    /* must be 0 */
} gdn_conv_dims;

/*
 * gdn_spec_decode_conv -- gdn_spec_decode with the depthwise causal
 * convolution that produces q, k and v fused in front of it ("PR #46090
 * report", implementation step 2: the speculative conv state is a wide
 * rolling buffer sliced per token, convolved and written back; "PR #51674
 * report", implementation step 3: the speculative path runs
 * causal_conv1d_update with rewind before the post-conv decode kernel).
 *
 * Instead of q, k, v the call takes the projection rows x
 * [num_tokens, conv_dim] (bf16, conv_dim = 2 H_k K + H_v V, channels in the
 * order q | k | v; row r of token t is gathered like every other input).  For
 * a processed sequence i (one that gdn_spec_decode would not skip), with
 * a = max(num_accepted[i], 1):
 *   history   the W-1 rows a .. a+W-2 of conv slot conv_in[i] (zeros when
 *             conv_in[i] < 0): the inputs up to the previous step's last
 *             accepted token;
 *   conv      y_t[c] = silu(bias[c] + sum_{w<W} weight[c][w] x_{t-W+1+w}[c])
 *             over (history, this step's rows) in time order, in FP32; y
 *             feeds the step as q | k | v (never rounded to bf16);
 *   new slot  conv slot conv_out[i] (skipped when < 0): rows 0 .. W-2 = the
 *             history, rows W-1 .. W-2+q_len = this step's rows, bit for bit;
 *             later rows are left as they were.
 * After a prefill the caller seeds a slot with the prompt's last W inputs in
 * rows 0 .. W-1 and passes num_accepted = 1.
 *
 *   x             bf16 [num_tokens, conv_dim], row stride cdims->x_stride
 *   conv_weight   bf16 [conv_dim, W]
 *   conv_bias     bf16 [conv_dim], or NULL (no bias)
 *   conv_pool     bf16 [num_conv_slots, state_len, conv_dim], caller-owned
 *   conv_in, conv_out  int32 [batch] (device)
 *   every other argument as for gdn_spec_decode; dims->q_stride, k_stride and
 *   v_stride are not used, dims->split must be 0 or 1.
 *
 * Caller contract (in addition to gdn_spec_decode's): no conv_out[j] >= 0
 * equals any conv_in[i] of the call (a slot is never read and written by one
 * step: the CTAs of a sequence share its q / k channels), and the
 * non-negative conv_out are distinct.  A conv slot >= num_conv_slots sets
 * GDN_FLAG_SLOT_RANGE and skips the sequence.  Host errors: width outside
 * 1..4, state_len too small or non-zero reserved -> GDN_ERR_BAD_SHAPE; x /
 * conv_pool / conv_bias not 8-byte aligned, conv_weight not 16-byte aligned
 * when W = 4, or x_stride not a multiple of 4 -> GDN_ERR_MISALIGNED.  Asynchronous on `stream`, allocates nothing.
 */
GDNSPEC_API gdn_status gdn_spec_decode_conv(
    const void* x, const void* conv_weight, const void* conv_bias, void* conv_pool,
    const int32_t* conv_in, const int32_t* conv_out, const gdn_conv_dims* cdims,
    const void* a, const void* b, const void* z,
    const float* A_log, const void* dt_bias, const void* norm_w,
    void* state_pool,
    const int32_t* state_indices, const int32_t* num_accepted,
    const int32_t* cu_seqlens, const int32_t* spec_token_indx,
    void* out,
    const gdn_dims* dims, float scale, float eps, gdn_dtype state_dtype,
    int32_t* status_word, gdn_stream_t stream);

/* ---- around the step: verification, tables, the convolution over prompts, and
 *      the state-space layer ------------------------------------------------------
 *
 * These serve the same loop as the entry points above and share their slots,
 * tables, status bits and conventions: asynchronous on `stream`, no allocation,
 * no host read of device data, capturable.  The device data of a call (tables,
 * lengths, slots) is checked on the device and reported through `status_word`;
 * outputs must not overlap inputs unless a call says so.  A call takes at most
 * 2^30 rows, and gdn_step_tables and gdn_conv_prefill at most 2^20 sequences
 * (GDN_ERR_BAD_SHAPE beyond).
 * Like the steps they start early behind a predecessor that lets them, and touch
 * memory only when it has completed.  gdn_ssm_prefill and gdn_ssm_decode let
 * their successor start early too, once their own predecessors have completed;
 * the others, which write tables and conv slots, do not, so that a step right
 * behind them reads what they wrote (without the GDN_PRE flag that covers it).
 */

/* Sizes of gdn_verify_drafts. */
typedef struct {
    int32_t batch;          /* sequences */
    int32_t num_tokens;     /* rows of target_probs */
    int32_t vocab;          /* entries of a row, >= 1 */
    int32_t max_T;          /* columns of out_tokens: host-known bound on every q_len, 1..32 */
    /* strides in ELEMENTS; 0 selects the dense default */
    int64_t target_stride;  /* between rows of target_probs (vocab) */
    int64_t draft_stride;   /* between drafts of a sequence in draft_probs (vocab) */
    int64_t draft_seq;      /* between sequences in draft_probs ((max_T - 1) * draft_stride) */
    int64_t token_stride;   /* between sequences in draft_tokens and accept_u (max_T - 1) */
} gdn_verify_dims;

/*
 * gdn_verify_drafts -- which drafted tokens the target model keeps, and the
 * token that follows them: what sets the num_accepted of the next step.
 *
 * Sequence i made q_len_i = cu_seqlens[i+1] - cu_seqlens[i] rows of
 * target_probs (the target's distribution after each of the step's tokens, the
 * last sampled token and n = q_len_i - 1 drafts).  With p_t its row t, d_t its
 * draft t, q_t the drafter's distribution for that draft and u_t = accept_u:
 *     draft t is kept iff every earlier one was and u_t q_t(d_t) < p_t(d_t);
 *     a = the number kept;  r = max(p_a - q_a, 0) if a < n, else p_n
 *         (p_a itself where that leaves nothing);
 *     the next token is the lowest v with sum_{w <= v} r_w > sample_u_i sum_w r_w.
 * Without draft_probs q_t is 1 at d_t and 0 elsewhere.  A draft token outside
 * [0, vocab) is never kept, and its place is sampled from p alone.
 *
 *   out_tokens[i]    d_0 .. d_{a-1}, the next token, then -1 up to max_T
 *   num_accepted[i]  a + 1: the step's tokens that stay, as gdn_spec_decode
 *                    and gdn_ssm_decode count them (the state after the last
 *                    kept token is in slot state_indices[i, a]); in batch order:
 *                    with request tables, see gdn_verify_drafts_by_request
 *
 * Arithmetic: a probability counts as a whole multiple of 2^-52 (rounded to
 * nearest; below 0 and NaN count as 0, above 1 as 1), so that the sums are
 * exact and the token does not depend on how a row is split.  The product
 * u q is formed in 64 bits; sample_u is taken into [0, 1).
 *
 *   target_probs   prob_dtype [num_tokens, vocab]
 *   draft_probs    prob_dtype [batch, max_T - 1, vocab], or NULL
 *   draft_tokens   int32 [batch, max_T - 1]   (NULL with max_T = 1)
 *   accept_u       fp32  [batch, max_T - 1], uniform in [0, 1)   (NULL with max_T = 1)
 *   sample_u       fp32  [batch], uniform in [0, 1)
 *   cu_seqlens     int32 [batch + 1]
 *   spec_token_indx int32 [cu_seqlens[batch]] row of every position, or NULL
 *                  when sequence i's rows are cu_seqlens[i] + t
 *   out_tokens     int32 [batch, max_T];  num_accepted int32 [batch]
 *
 * A sequence with q_len <= 0 gets no tokens (-1 throughout) and keeps its
 * num_accepted, as its states keep theirs; so does one with bad data, which the
 * step skips too (q_len > max_T: GDN_FLAG_QLEN; a row outside [0, num_tokens),
 * or cu_seqlens out of order with cu_seqlens[batch]: GDN_FLAG_TOKEN_ROW).  A
 * sequence whose r counts as 0 throughout, or sums to 16 or more (scores instead of
 * probabilities), emits -1 in the next token's place and sets GDN_FLAG_NO_TOKEN; a
 * row of p or q that sums to more is fine where r does not.
 * Every pointer needs only its element's alignment.
 */
GDNSPEC_API gdn_status gdn_verify_drafts(
    const void* target_probs, const void* draft_probs, const int32_t* draft_tokens,
    const float* accept_u, const float* sample_u,
    const int32_t* cu_seqlens, const int32_t* spec_token_indx,
    int32_t* out_tokens, int32_t* num_accepted,
    const gdn_verify_dims* dims, gdn_dtype prob_dtype,
    int32_t* status_word, gdn_stream_t stream);

/*
 * gdn_verify_drafts_by_request -- the same where the sequences of the batch are
 * requests in some other order: sequence i's count goes to
 * num_accepted[request[i]], the table by request that gdn_step_tables reads as
 * `accepted` (the entries of requests that are not in the batch stay).  out_tokens
 * and everything else stay in batch order.
 *
 *   request        int32 [batch], as given to gdn_step_tables; negative: no request,
 *                  its count is not kept; those that have rows are distinct
 *   num_accepted   int32 [num_requests]
 *
 * The request of a sequence that is skipped is not looked at.  A request >=
 * num_requests sets GDN_FLAG_SLOT_RANGE; its tokens are written, its count is not.
 */
GDNSPEC_API gdn_status gdn_verify_drafts_by_request(
    const void* target_probs, const void* draft_probs, const int32_t* draft_tokens,
    const float* accept_u, const float* sample_u,
    const int32_t* cu_seqlens, const int32_t* spec_token_indx, const int32_t* request,
    int32_t* out_tokens, int32_t* num_accepted,
    const gdn_verify_dims* dims, int32_t num_requests, gdn_dtype prob_dtype,
    int32_t* status_word, gdn_stream_t stream);

/* Sizes of gdn_step_tables. */
typedef struct {
    int32_t batch;          /* requests of this step */
    int32_t num_tokens;     /* entries of token_indx: host-known bound on the step's rows */
    int32_t spec_stride;    /* columns of slot_table and state_indices */
    int32_t num_requests;   /* rows of slot_table, accepted, conv_table and conv_turn */
} gdn_tables_dims;

/*
 * gdn_step_tables -- the tables of one step, from the lengths of its requests:
 * the offsets, the row gather, the slots and the conv slots that
 * gdn_spec_decode, gdn_spec_decode_conv, gdn_ssm_decode and gdn_verify_drafts
 * read.  The requests' rows follow one another in the token batch.  With q_i =
 * max(q_lens[i], 0), r = request[i] and m_i = "request i is speculative"
 * (spec[i] != 0, 0 <= r < num_requests, q_i <= spec_stride):
 *     row_starts[i]  = sum_{j < i} q_j                   (batch + 1 entries)
 *     cu_seqlens[i]  = sum_{j < i} q_j m_j               (batch + 1 entries)
 *     token_indx     = the rows of the speculative requests in order, then all
 *                      other rows in order: its first cu_seqlens[batch] entries
 *                      are the spec_token_indx of the other calls; entries from
 *                      row_starts[batch] on are left as they were
 *     state_indices[i] = m_i ? slot_table[r] : -1 ...
 *     num_accepted[i]  = m_i ? accepted[r] : 0
 *     conv_in[i], conv_out[i] = m_i ? conv_table[r, c], conv_table[r, 1 - c] : -1, -1
 *                      with c = conv_turn[r] & 1; where m_i and q_i > 0,
 *                      conv_turn[r] <- 1 - c, so that the next step reads the
 *                      slot that this one writes
 *
 *   q_lens       int32 [batch]
 *   spec         int32 [batch], or NULL (every request is speculative)
 *   request      int32 [batch] row of the request in the tables below, or NULL
 *                (row i); negative: none (a padded entry); distinct
 *   slot_table   int32 [num_requests, spec_stride] the state slots of a request
 *   accepted     int32 [num_requests], by request: gdn_verify_drafts' num_accepted
 *                where sequence i is request i, else gdn_verify_drafts_by_request's
 *   conv_table   int32 [num_requests, 2], conv_turn int32 [num_requests]
 *                (updated), conv_in, conv_out int32 [batch]: all four or none
 *   row_starts   may be NULL
 *
 * A request row >= num_requests sets GDN_FLAG_SLOT_RANGE and a speculative
 * request with q_i > spec_stride sets GDN_FLAG_QLEN; either counts as not
 * speculative.  More than num_tokens rows in all set GDN_FLAG_TOKEN_ROW and
 * give an empty step: every q_i counts as 0 and no request as speculative.
 */
GDNSPEC_API gdn_status gdn_step_tables(
    const int32_t* q_lens, const int32_t* spec, const int32_t* request,
    const int32_t* slot_table, const int32_t* accepted,
    const int32_t* conv_table, int32_t* conv_turn,
    int32_t* cu_seqlens, int32_t* row_starts, int32_t* token_indx,
    int32_t* state_indices, int32_t* num_accepted, int32_t* conv_in, int32_t* conv_out,
    const gdn_tables_dims* dims, int32_t* status_word, gdn_stream_t stream);

/*
 * gdn_conv_prefill -- the depthwise causal convolution of gdn_spec_decode_conv
 * over whole prompts, or over the next chunk of prompts: it makes the rows
 * that gdn_prefill, gdn_prefill_chunked and gdn_ssm_prefill read, and seeds the
 * conv slots of the steps that follow.
 *
 * Sequence i is rows cu_seqlens[i] .. cu_seqlens[i+1]-1 of x.  With x_t for
 * t < 0 the history: rows 1 .. W-1 of conv slot conv_in[i] in time order
 * (zeros when conv_in[i] < 0):
 *     y_t[c] = round_bf16( silu( bias[c] + sum_{w<W} weight[c][w] x_{t-W+1+w}[c] ) )
 * in FP32, and conv slot conv_out[i] (skipped when < 0) gets the last W inputs
 * (history included) in rows 0 .. W-1, bit for bit; its other rows are left as
 * they were.  A step after it passes num_accepted = 1; a further chunk of the
 * prompt passes conv_in[i] = that slot.  conv_in[i] == conv_out[i] updates a
 * slot in place.  A sequence without rows (cu_seqlens[i+1] <= cu_seqlens[i]) is
 * skipped: slot conv_out[i] keeps what it holds, also where conv_in[i] is another
 * slot, so its history stays in slot conv_in[i].
 *
 *   x            bf16 [num_tokens, conv_dim], row stride cdims->x_stride
 *   conv_weight  bf16 [conv_dim, W];  conv_bias bf16 [conv_dim], or NULL
 *   conv_pool    bf16 [num_conv_slots, state_len, conv_dim], state_len >= W
 *   conv_in, conv_out int32 [batch];  cu_seqlens int32 [batch + 1]
 *   y            bf16 [num_tokens, conv_dim], row stride y_stride (0: conv_dim);
 *                rows of no sequence are left as they were
 *
 * cdims->width 1..4.  conv_dim a multiple of 4, at most 2^30; x, y, conv_weight, conv_bias
 * and conv_pool 8-byte aligned; x_stride and y_stride multiples of 4 (16-byte
 * aligned pointers and multiples of 8 run faster over many rows).  Sequences follow one
 * another: cu_seqlens does not decrease.  No conv_out[j] >= 0 equals another
 * sequence's conv_in or conv_out.  Bad device data skips the sequence: a conv
 * slot >= num_conv_slots sets GDN_FLAG_SLOT_RANGE, rows outside
 * [0, num_tokens) set GDN_FLAG_TOKEN_ROW.
 */
GDNSPEC_API gdn_status gdn_conv_prefill(
    const void* x, const void* conv_weight, const void* conv_bias, void* conv_pool,
    const int32_t* conv_in, const int32_t* conv_out, const int32_t* cu_seqlens,
    void* y, int32_t batch, int32_t num_tokens, int32_t conv_dim, int64_t y_stride,
    const gdn_conv_dims* cdims, int32_t* status_word, gdn_stream_t stream);

/* Sizes of the state-space layer. */
typedef struct {
    int32_t batch;        /* sequences */
    int32_t num_tokens;   /* rows of the token tensors */
    int32_t H, G;         /* heads, and groups of heads that share B and C; H % G == 0 */
    int32_t P, N;         /* head dim (a multiple of 64, at most 256) and state dim (64 or 128) */
    int32_t spec_stride;  /* gdn_ssm_decode: columns of state_indices */
    int32_t max_T;        /* gdn_ssm_decode: host-known bound on every q_len, 1..8 */
    int64_t num_slots;    /* slots in state_pool */
    /* row strides in ELEMENTS, 0 = dense (x, z, out: H*P; B, C: G*N; dt: H) */
    int64_t x_stride, b_stride, c_stride, dt_stride, z_stride, out_stride;
    int32_t reserved[2];  /* must be 0 */
} gdn_ssm_dims;

/*
 * gdn_ssm_prefill -- a selective state-space layer over whole prompts: the
 * gated linear recurrence of this library without the delta term, with one
 * decay per head and token.  Head h uses group g = h / (H / G).  With S the
 * N x P state of (sequence i, head h), P contiguous:
 *     d = softplus(dt[r,h] + dt_bias[h])                (as in gdn_spec_decode)
 *     S <- e^(-exp(A_log[h]) d) S + B[r,g] (d x[r,h])^T
 *     out[r,h] = round_bf16( (S^T C[r,g] + D[h] x[r,h]) silu(z[r,h]) )
 * Sequence i is rows cu_seqlens[i] .. cu_seqlens[i+1]-1; it starts from slot
 * read_slots[i] (the zero state when < 0) and its last state goes to slot
 * write_slots[i] (no write when < 0; in place when equal), rounded once.
 *
 *   x            bf16 [num_tokens, H, P];  B, C bf16 [num_tokens, G, N]
 *   dt           bf16 [num_tokens, H];  dt_bias bf16 [H];  A_log fp32 [H]
 *   z            bf16 [num_tokens, H, P], or NULL (no gate);  D fp32 [H], or NULL (0)
 *   state_pool   state_dtype [num_slots, H, N, P]
 *   out          bf16 [num_tokens, H, P]; rows of no sequence are left as they were
 *   workspace    gdn_ssm_prefill_workspace(dims) bytes of device memory, 16-byte
 *                aligned, used by this call alone until it has run (NULL when that
 *                is 0); what it holds before and after does not matter
 *
 * Within a row the heads (groups) are contiguous; x, B and C may be views into
 * one packed row.  x, B, C, z, out and state_pool are 16-byte aligned and
 * x/B/C/z/out strides multiples of 8.  A head dim P > 64 runs as P / 64 column
 * blocks.  Caller contract and skips as for gdn_prefill (a sequence without rows
 * writes no slot: its state stays in slot read_slots[i]); sequences do not
 * overlap (cu_seqlens does not decrease).  An infinite or NaN
 * input spoils rows and the last state of its own sequence (rows shortly before
 * it among them: the products run over tiles of tokens), and no other's.
 */
GDNSPEC_API gdn_status gdn_ssm_prefill(
    const void* x, const void* B, const void* C, const void* dt, const void* z,
    const float* A_log, const void* dt_bias, const float* D,
    void* state_pool, const int32_t* read_slots, const int32_t* write_slots,
    const int32_t* cu_seqlens, void* out, void* workspace, int64_t workspace_bytes,
    const gdn_ssm_dims* dims, gdn_dtype state_dtype,
    int32_t* status_word, gdn_stream_t stream);

/* Workspace that gdn_ssm_prefill needs for these sizes, in bytes (-1: invalid dims).
 * Host only; depends on the current device's number of SMs. */
GDNSPEC_API int64_t gdn_ssm_prefill_workspace(const gdn_ssm_dims* dims);

/*
 * gdn_ssm_decode -- the state-space layer over one to eight tokens of each
 * sequence, with the short causal convolution fused in front and the rewind of
 * gdn_spec_decode_conv: projection rows xbc [num_tokens, conv_dim] (conv_dim =
 * H P + 2 G N, channels x | B | C) are convolved (silu, never rounded to bf16),
 * the state starts from slot state_indices[i, max(num_accepted[i]-1, 0)], and
 * the state after token t goes to slot state_indices[i, t] (skipped when < 0),
 * rounded once.  A single-token step is spec_stride = max_T = 1.
 *
 * The conv slots (history rows, new rows, seeding), the gather, the skips, the
 * caller contract and the status bits are those of gdn_spec_decode_conv; the
 * recurrence, dt, z, D and the pool are those of gdn_ssm_prefill.
 * cdims->x_stride is the row stride of xbc; dims->x_stride, b_stride and
 * c_stride are not used.  state_pool 16-byte aligned; xbc, conv_weight (W = 4),
 * conv_bias, conv_pool, z and out 8-byte aligned with xbc/z/out strides
 * multiples of 4.
 */
GDNSPEC_API gdn_status gdn_ssm_decode(
    const void* xbc, const void* conv_weight, const void* conv_bias, void* conv_pool,
    const int32_t* conv_in, const int32_t* conv_out, const gdn_conv_dims* cdims,
    const void* dt, const void* z, const float* A_log, const void* dt_bias, const float* D,
    void* state_pool, const int32_t* state_indices, const int32_t* num_accepted,
    const int32_t* cu_seqlens, const int32_t* spec_token_indx, void* out,
    const gdn_ssm_dims* dims, gdn_dtype state_dtype,
    int32_t* status_word, gdn_stream_t stream);

/* ---- the attention layers beside the recurrent ones: a paged key-value cache, and the
 *      attention of a step's tokens over it ------------------------------------------------
 *
 * A hybrid model's full attention layers run in the same loop, on the same batches and
 * tables (cu_seqlens and spec_token_indx from gdn_step_tables): gdn_kv_write puts the
 * step's keys and values behind the sequence's cached ones, gdn_attn_decode attends to
 * all of them, and what gdn_verify_drafts keeps moves the length on (kv_lens[i] +=
 * num_accepted[i]; rows behind it are written again by the next step).  The conventions
 * of the calls around the step hold; all three calls let their successor start early
 * once their own predecessors have completed.
 *
 * The cache.  k_cache and v_cache hold num_pages pages of page_size positions of H_kv rows
 * of D elements; position x of sequence i is row x % page_size of page
 * page_table[i, x / page_size].  page_table is int32 [batch, table_cols], rows
 * table_stride apart.  A negative page is none: its positions are not written, not read
 * and not attended to.  A page >= num_pages counts as none and sets GDN_FLAG_SLOT_RANGE.
 * Both caches have the same strides (in elements, any order of pages, positions and
 * heads; a row's D elements are contiguous), so they may be views of one tensor.
 *
 * 8-bit caches (GDN_E4M3, GDN_I8) hold codes; k_scale and v_scale, fp32 [num_pages,
 * page_size, H_kv] with strides of their own, a scale for each row: the row's elements
 * stand for code * scale.  gdn_kv_write makes them from the row's largest absolute value a:
 *     GDN_E4M3  scale = 2^e, the least e >= -100 with a <= 448 * 2^e; codes are rounded to
 *               the nearest e4m3 value (a power of two: x / scale is exact, and so is what
 *               a bf16 row reads back)
 *     GDN_I8    scale = a / 127 rounded up to 8 significant bits, at least 2^-100; codes
 *               are x / scale rounded to the nearest whole number
 * (ties to even).  A row that holds an infinity or NaN gets the scale NaN and codes 0: it
 * reads back as NaN and spoils the attention of those that see it.
 */

/* Sizes of the key-value cache and of the calls on it. */
typedef struct {
    int32_t batch;          /* sequences */
    int32_t num_tokens;     /* rows of the token tensors */
    int32_t H_q, H_kv;      /* heads of q (gdn_attn_decode alone), and of the cache; H_q % H_kv == 0 */
    int32_t D;              /* head dim: 64, 128, 192 or 256 */
    int32_t page_size;      /* positions of a page, >= 1 */
    int32_t table_cols;     /* columns of page_table */
    int32_t max_T;          /* gdn_attn_decode: host-known bound on every q_len, 1..8 */
    int32_t window;         /* gdn_attn_decode: a token sees this many positions, itself included; 0: all */
    int32_t reserved;       /* must be 0 */
    int64_t num_pages;      /* pages of the caches */
    /* strides in ELEMENTS, 0 = dense ([pages, positions, heads, D]; rows H*D apart; table_cols) */
    int64_t page_stride, token_stride, head_stride;
    int64_t scale_page_stride, scale_token_stride, scale_head_stride;
    int64_t table_stride;
    int64_t q_stride, k_stride, v_stride, z_stride, out_stride;   /* k, v: rows of gdn_kv_write and gdn_kv_read */
} gdn_kv_dims;

/*
 * gdn_kv_write -- rows of keys and values into the cache, quantised where it has 8 bits.
 * Sequence i's rows are cu_seqlens[i] .. cu_seqlens[i+1]-1 (of the token batch, or of
 * spec_token_indx); row t of it goes to position kv_lens[i] + t.  One step's drafted
 * tokens or whole prompts alike.
 *
 *   k, v         bf16 [num_tokens, H_kv, D], rows k_stride, v_stride apart
 *   k_cache, v_cache  cache_type; k_scale, v_scale fp32 (8-bit types; else not used)
 *   page_table   int32;  kv_lens int32 [batch];  cu_seqlens int32 [batch + 1]
 *   spec_token_indx  int32 [cu_seqlens[batch]], or NULL
 *
 * A 16-bit cache gets each element rounded to its type.  cu_seqlens does not decrease; no
 * two rows of a call go to the same place.  Bad device data skips the sequence: kv_lens[i]
 * < 0 or kv_lens[i] + q_len > table_cols * page_size sets GDN_FLAG_SLOT_RANGE, rows outside
 * [0, num_tokens) set GDN_FLAG_TOKEN_ROW (an entry of spec_token_indx outside skips its row
 * alone).  k, v and the caches 16-byte aligned, k_stride and v_stride multiples of 8, the
 * caches' strides multiples of 16 bytes; scales 4-byte aligned.
 */
GDNSPEC_API gdn_status gdn_kv_write(
    const void* k, const void* v, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
    const int32_t* page_table, const int32_t* kv_lens, const int32_t* cu_seqlens,
    const int32_t* spec_token_indx, const gdn_kv_dims* dims, gdn_dtype cache_type,
    int32_t* status_word, gdn_stream_t stream);

/*
 * gdn_kv_read -- cached rows back as dense ones: positions kv_begin[i] + t (t alone where
 * kv_begin is NULL) of sequence i to rows cu_seqlens[i] + t of k and v.  For a prompt's
 * attention over a cached prefix, or to move a sequence.
 *
 *   k, v         row_type (GDN_F32, GDN_BF16 or GDN_F16) [num_tokens, H_kv, D], rows k_stride,
 *                v_stride apart; each element code * scale in FP32, rounded to the type
 *   kv_begin     int32 [batch], or NULL;  everything else as for gdn_kv_write
 *
 * Rows of no sequence, of a skipped sequence and of positions without a page are left as
 * they were.  k and v do not overlap the cache.  Strides of k and v: multiples of 8.
 */
GDNSPEC_API gdn_status gdn_kv_read(
    const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
    const int32_t* page_table, const int32_t* kv_begin, const int32_t* cu_seqlens,
    void* k, void* v, const gdn_kv_dims* dims, gdn_dtype cache_type, gdn_dtype row_type,
    int32_t* status_word, gdn_stream_t stream);

/*
 * gdn_attn_decode -- the attention of one to eight tokens of each sequence over its cached
 * keys and values, those of the step itself (written before, by gdn_kv_write) among them.
 * With x = kv_lens[i] + t the position of token t, row r = its row, head h using head
 * h / (H_q / H_kv) of the cache:
 *     s_j  = scale * q[r,h] . k_j    for max(0, x - window + 1) <= j <= x (window 0: from 0)
 *     o    = sum_j e^(s_j) v_j / sum_j e^(s_j)          (0 where no position is left)
 *     out[r,h] = round_bf16( o * sigmoid(z[r,h]) )       (o itself without z)
 *
 *   q, z, out    bf16 [num_tokens, H_q, D]; z may be NULL; rows of no sequence and of skipped
 *                ones are left as they were
 *   spec_token_indx  int32 [cu_seqlens[batch]], or NULL
 *   workspace    gdn_attn_decode_workspace(dims, cache_type) bytes of device memory, 16-byte
 *                aligned, used by this call alone until it has run; what it holds before and
 *                after does not matter
 *
 * Scores, the softmax's maximum and sum, and the output are held in FP32; the weights are
 * rounded to 16 significant bits for a bf16 cache (two bf16 parts) and to 11 for the others
 * (fp16), or to half of 2^-30 of the row's largest where that is more.  In an 8-bit cache that
 * is weight times scale of the value (all bits where a row's largest product is 2^-74 or more,
 * its largest weight being 1).  Values may be as large as FP32 and bf16 are (those of a bf16 cache
 * below 2^-90 lose bits).  q is exact, its elements below 2^-24 of a head's largest to 2^-31 of
 * that.  The positions of a batch are cut evenly among the CTAs and the parts joined in order, so
 * equal calls give equal results; how a sequence is cut depends on the others' lengths, by rounding
 * in FP32.  Bad device data: q_len > max_T sets GDN_FLAG_QLEN, the rest as for gdn_kv_write, except
 * that any row of a sequence outside [0, num_tokens) skips the
 * sequence.  An infinity or NaN in k or v spoils the tokens that see it, in q its own row.  (In an
 * 8-bit cache that is a scale; a GDN_E4M3 code that is NaN, which gdn_kv_write never makes, may spoil
 * other tokens of its sequence too.)
 * q, z, out 16-byte aligned with strides that are multiples of 8; the caches as above.
 * batch at most 2^20 sequences.
 */
GDNSPEC_API gdn_status gdn_attn_decode(
    const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
    const int32_t* page_table, const int32_t* kv_lens, const int32_t* cu_seqlens,
    const int32_t* spec_token_indx, const void* z, void* out, void* workspace, int64_t workspace_bytes,
    const gdn_kv_dims* dims, float scale, gdn_dtype cache_type,
    int32_t* status_word, gdn_stream_t stream);

/* Workspace that gdn_attn_decode needs for these sizes, in bytes (-1: invalid dims or type).
 * Host only; depends on the current device's number of SMs. */
GDNSPEC_API int64_t gdn_attn_decode_workspace(const gdn_kv_dims* dims, gdn_dtype cache_type);

/*
 * The split code that gdn_spec_decode would use for these sizes and state
 * dtype (dims->split itself when it is not 0; else, for an FP32 state,
 * GDN_SPLIT_HALFK | 2 with batch * H_v <= 64 and GDN_SPLIT_HALFK | 1 with
 * batch * H_v <= 128; else 1), or 0 for invalid dims or dtype.
 * Host only; reads no device state.
 */
GDNSPEC_API int32_t gdn_spec_decode_split(const gdn_dims* dims, gdn_dtype state_dtype);

/*
 * Bound on each wait of gdn_prefill_chunked for its tensor-core products, and
 * of gdn_ssm_prefill and gdn_attn_decode (many query rows) for those, their copies and their own
 * warps: 0 (the default)
 * waits with blocking polls of the barrier, 2^24 of them (2^17 of up to 20 us;
 * well over a second either way); a non-zero bound counts non-blocking polls
 * instead, so that a small one runs out for certain.  A wait that runs out
 * sets GDN_FLAG_TIMEOUT; the unit writes no final state and its CTAs end
 * after waiting, with the default bound, for the products still in flight
 * (a 2-CTA unit first runs its remaining chunks, whose outputs are invalid).  Process-wide, read at every
 * launch; meant for exercising that path in tests.  No counterpart on the
 * report pages.
 */
GDNSPEC_API void gdn_set_wait_limit(uint32_t polls);

/* Static English text for a status code (never NULL). */
GDNSPEC_API const char* gdn_status_str(gdn_status status);

/* GDNSPEC_VERSION of the loaded library. */
GDNSPEC_API int32_t gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDNSPEC_H */
