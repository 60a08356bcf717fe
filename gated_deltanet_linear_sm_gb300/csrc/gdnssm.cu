// libgdnspec: the short causal convolution over prompts (gdn_conv_prefill) and
// the state-space layer's step over one to eight tokens (gdn_ssm_decode), with
// the C entry points of the layer.  Declared in include/gdnspec.h.
#include <type_traits>

#include "gdnssm.h"
#include "gdnssm_recur.cuh"

using namespace gdn_common;
using namespace gdn_ssm;

namespace {

// ---- gdn_conv_prefill --------------------------------------------------------------
//
// A thread owns 8 (or 4) neighbouring channels of a run of rows and slides a
// window of the last W - 1 inputs, in FP32 registers, along them: x is read
// once (W - 1 rows a run twice) and y written once, in 16-byte accesses.  Up to 8
// rows a thread are on their way through asynchronous copies into places of its
// own in shared memory; the arithmetic runs on pairs of channels.  Rows are cut into runs of the whole token batch,
// not of a sequence, so ragged prompts fill the GPU evenly; a run that crosses
// the start of a sequence takes its window from the conv slot instead.  The
// first W - 1 rows of a sequence always belong to the run that holds its first
// row: that run alone reads the sequence's slot, and writes the new one after
// it, so a slot may be updated in place.  HBM bandwidth bounds it: 16211 rows of
// 4352 channels take 52.5 us, 5.4 TB/s of 6.8 measured (with the copies in registers 65, and
// with one channel an instruction 81); half of the issue slots are in use, so the
// rest is the start and the end of the runs.  (The window behind the sequence's last rows
// is picked by a number known at run time: 48 bytes of local memory a thread with W = 4
// and 8 channels, used once a sequence.)
// (No early start of the next kernel: the step reads conv slots through __ldg,
// which may run before its wait.)

constexpr int kCThreads = 128;                      // at most

struct ConvParams {
    const __nv_bfloat16* x;
    const __nv_bfloat16* w;
    const __nv_bfloat16* bias;
    __nv_bfloat16* pool;
    const int32_t* in;
    const int32_t* out;
    const int32_t* cu;
    __nv_bfloat16* y;
    int32_t* status;
    int64_t x_stride, y_stride, num_slots, slot;    // slot: elements of a conv slot
    int32_t batch, num_tokens, dim, run, col_blocks;
};

// CV channels of one row, raw bf16
template <int CV>
using Raw = std::conditional_t<CV == 8, uint4, uint2>;

template <int CV>
__device__ __forceinline__ void widen_all(const Raw<CV>& raw, u64 (&x)[CV / 2]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
    for (int e = 0; e < CV / 2; ++e) x[e] = widen(w[e]);
}

// one row's channels into shared memory, asynchronously
template <int CV>
__device__ __forceinline__ void copy_async(Raw<CV>* dst, const __nv_bfloat16* src) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (CV == 8)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(src) : "memory");
}

// whether sequence j may run: its rows and conv slots are in range
__device__ __forceinline__ int conv_flag(const ConvParams& p, int s, int e, int j) {
    if (s < 0 || e > p.num_tokens) return GDN_FLAG_TOKEN_ROW;
    if (ld(p.in + j) >= p.num_slots || ld(p.out + j) >= p.num_slots) return GDN_FLAG_SLOT_RANGE;
    return 0;
}

template <int CV, int W>
__global__ void __launch_bounds__(kCThreads, 4) gdn_conv_prefill_kernel(const ConvParams p) {
    constexpr int HN = W > 1 ? W - 1 : 1;
    constexpr int U = 4, kAhead = 2, kRing = U * (kAhead + 1);
    __shared__ Raw<CV> ring[kRing][kCThreads];
    dep_wait();
    const int cb = blockIdx.x % p.col_blocks;
    const int r0 = static_cast<int>(blockIdx.x / p.col_blocks) * p.run;
    const int r1 = min(p.num_tokens, r0 + p.run);
    if (blockIdx.x == 0) {                          // bad data, reported once
        for (int j = threadIdx.x; j < p.batch; j += blockDim.x) {
            const int s = ld(p.cu + j), e = ld(p.cu + j + 1);
            const int flag = e > s ? conv_flag(p, s, e, j) : 0;
            if (flag) raise(p.status, flag);
        }
    }
    // the first sequence that ends behind r0
    int j = 0;
    for (int base = 0; base < p.batch; base += blockDim.x) {
        const int k = base + threadIdx.x;
        const int done = __syncthreads_count(k < p.batch && ld(p.cu + k + 1) <= r0);
        j += done;
        if (done < static_cast<int>(blockDim.x)) break;
    }
    const int c = (cb * static_cast<int>(blockDim.x) + threadIdx.x) * CV;
    if (c >= p.dim) return;

    u64 wt2[CV / 2][W], bias2[CV / 2];              // pairs of channels
    {
        float wt[CV][W], bias[CV];
#pragma unroll
        for (int e = 0; e < CV; ++e) bias[e] = 0.f;
        if constexpr (W == 4) {                     // CV channels' taps: CV 8-byte words
#pragma unroll
            for (int e = 0; e < CV; ++e)
                unpack4(ld(reinterpret_cast<const uint2*>(p.w + static_cast<int64_t>(c + e) * 4)), wt[e]);
        } else {
#pragma unroll
            for (int e = 0; e < CV; ++e)
#pragma unroll
                for (int k = 0; k < W; ++k) wt[e][k] = __bfloat162float(p.w[static_cast<int64_t>(c + e) * W + k]);
        }
        if (p.bias) {
#pragma unroll
            for (int e = 0; e < CV; ++e) bias[e] = __bfloat162float(p.bias[c + e]);
        }
#pragma unroll
        for (int e = 0; e < CV / 2; ++e) {
            bias2[e] = pk2(bias[2 * e], bias[2 * e + 1]);
#pragma unroll
            for (int k = 0; k < W; ++k) wt2[e][k] = pk2(wt[2 * e][k], wt[2 * e + 1][k]);
        }
    }

    auto row_of_x = [&](int64_t r) { return ld(reinterpret_cast<const Raw<CV>*>(p.x + r * p.x_stride + c)); };
    for (; j < p.batch; ++j) {
        const int s = ld(p.cu + j), e = ld(p.cu + j + 1);
        if (s >= r1) break;
        if (e <= s || conv_flag(p, s, e, j)) continue;
        const bool first = s >= r0;
        int a = max(s, r0), b = min(e, r1);
        if (first) b = max(b, min(e, s + W - 1));   // its first W - 1 rows, whole
        else a = max(a, min(e, s + W - 1));
        if (a >= b) continue;
        // U rows a batch; kAhead batches on their way into this thread's own places of the ring
        auto fetch = [&](int r) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u < b)
                    copy_async<CV>(&ring[(r - a + u) % kRing][threadIdx.x], p.x + (r + u) * p.x_stride + c);
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k) fetch(a + k * U);
        Raw<CV> win[HN] = {};
        if (W > 1 && first) {
            const int in = ld(p.in + j);
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                if (in >= 0) win[k] = *reinterpret_cast<const Raw<CV>*>(p.pool + in * p.slot + (k + 1) * static_cast<int64_t>(p.dim) + c);
        } else if (W > 1) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) win[k] = row_of_x(a - (W - 1) + k);
        }
        if (first) {
            const int out = ld(p.out + j);
            if (out >= 0) {
                __nv_bfloat16* dst = p.pool + out * p.slot + c;
#pragma unroll
                for (int k = 0; k < W; ++k) {       // input e - W + k, or the history in front of the sequence
                    const int t = e - s - W + k;
                    Raw<CV> v = {};
                    if (t >= 0) {
                        v = row_of_x(s + t);
                    } else {
#pragma unroll
                        for (int h = 0; h < W - 1; ++h)
                            if (t + W - 1 == h) v = win[h];
                    }
                    *reinterpret_cast<Raw<CV>*>(dst + k * static_cast<int64_t>(p.dim)) = v;
                }
            }
        }
        // pairs of channels: each tap is one instruction a pair
        u64 f[HN][CV / 2];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) widen_all<CV>(win[k], f[k]);
        for (int r = a; r < b; r += U) {
            fetch(r + kAhead * U);
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
            Raw<CV> raw[U];                         // (rows behind b are worked on too, for the sake of one block of code)
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = ring[(r - a + u) % kRing][threadIdx.x];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                u64 v[CV / 2];
                widen_all<CV>(raw[u], v);
                Raw<CV> o;
                uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
                for (int e2 = 0; e2 < CV / 2; ++e2) {
                    u64 acc = bias2[e2];
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) acc = ffma2(wt2[e2][k], f[k][e2], acc);
                    acc = silu2(ffma2(wt2[e2][W - 1], v[e2], acc));
                    ow[e2] = pack2(lo2(acc), hi2(acc));
                }
#pragma unroll
                for (int k = 0; k + 1 < W - 1; ++k)
#pragma unroll
                    for (int e2 = 0; e2 < CV / 2; ++e2) f[k][e2] = f[k + 1][e2];
                if constexpr (W > 1) {
#pragma unroll
                    for (int e2 = 0; e2 < CV / 2; ++e2) f[W - 2][e2] = v[e2];
                }
                if (r + u < b) *reinterpret_cast<Raw<CV>*>(p.y + (r + u) * p.y_stride + c) = o;
            }
        }
    }
}

template <int CV>
cudaError_t launch_conv(ConvParams p, int width, cudaStream_t stream) {
    // CTAs of 64, 96 or 128 threads, whichever leaves the fewest idle behind the last channel
    const int64_t threads = (p.dim + CV - 1) / CV;
    int width_of = kCThreads;
    for (int t : {96, 64})
        if ((threads + t - 1) / t * t < (threads + width_of - 1) / width_of * width_of) width_of = t;
    p.col_blocks = static_cast<int>((threads + width_of - 1) / width_of);
    // Rows of a run: few enough that every SM has its 512 threads, and so that the last round of
    // CTAs is no small one.  A run costs kStart rows' time beside its own (its taps, its window).
    constexpr int kStart = 8;
    const int64_t resident = static_cast<int64_t>(sm_count() ? sm_count() : 148) * (512 / width_of);
    double best = 1e300;
    for (int run = 4; run <= 64; ++run) {
        const int64_t n = (static_cast<int64_t>(p.num_tokens) + run - 1) / run * p.col_blocks;
        const double cost = static_cast<double>((n + resident - 1) / resident) * (run + kStart);
        if (cost <= best) {
            best = cost;
            p.run = run;
        }
    }
    const int64_t ctas = (static_cast<int64_t>(p.num_tokens) + p.run - 1) / p.run * p.col_blocks;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(width_of), 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (width) {
    case 1: return cudaLaunchKernelEx(&cfg, gdn_conv_prefill_kernel<CV, 1>, p);
    case 2: return cudaLaunchKernelEx(&cfg, gdn_conv_prefill_kernel<CV, 2>, p);
    case 3: return cudaLaunchKernelEx(&cfg, gdn_conv_prefill_kernel<CV, 3>, p);
    default: return cudaLaunchKernelEx(&cfg, gdn_conv_prefill_kernel<CV, 4>, p);
    }
}

// ---- gdn_ssm_decode ----------------------------------------------------------------
//
// One CTA of 128 threads per (sequence, head, 64 columns of the head dim).
// The state block is read once into FP32 registers (issued first, so that it
// arrives while the convolution runs), goes through the tokens in order and is
// written after each, straight from registers in whole 128-byte lines.  The
// convolution of the block's 64 + 2 N channels is one thread a channel quad:
// the heads of a group repeat that of B and C (a few KB from L2 against 16 or
// 32 KB of state a token), and the group's first CTA alone writes those
// channels' conv slot.  HBM bandwidth on the state bounds large batches, the
// chain of dependent reads small ones: 64 sequences of up to 4 tokens and 64 heads with
// N = 128 and FP32 states take 76.5 us, 6.0 TB/s of 6.8 measured (with the projection's rows
// behind the state's 99); 2 of one token and 32 heads 5.2.  States of 16 bits or of N = 64 put
// half the bytes or fewer behind the same chain: 3.8 TB/s at 256 x 4 tokens, N = 64, bf16.

template <typename StateT, int N>
__global__ void __launch_bounds__(kRThreads, 4) gdn_ssm_decode_kernel(const Params p) {
    constexpr int R = N / 16;
    constexpr int kQuads = 16 + N / 2;              // channel quads of x, B and C
    static_assert(kQuads + kMaxT <= kRThreads, "one thread a quad, and one a token");
    __shared__ Round<N> s;
    const int tid = threadIdx.x, cg = tid & 7, rg = tid >> 3;
    const int pb = static_cast<int>(blockIdx.x % p.blocks);
    const int unit = static_cast<int>(blockIdx.x / p.blocks);
    const int i = unit / p.H, h = unit - i * p.H;
    const int g = h / p.group;
    dep_wait();
    dep_launch();

    // ---- the work item (every thread finds the same) ----
    const int32_t* slot_row = p.idx + static_cast<int64_t>(i) * p.stride;
    const int bos = ld(p.cu + i);
    const int eos = ld(p.cu + i + 1);
    const int acc = ld(p.num_acc + i);
    const int total = ld(p.cu + p.batch);
    const long long cin = ld(p.conv_in + i), cout = ld(p.conv_out + i);
    if (eos <= bos) return;
    const int n = bos < 0 ? 0 : eos - bos;
    int flag = 0;
    if (bos < 0 || eos > total) flag = GDN_FLAG_TOKEN_ROW;
    else if (acc > p.stride) flag = GDN_FLAG_ACCEPTED;
    else if (n > p.max_T || n > p.stride) flag = GDN_FLAG_QLEN;
    if (flag) {
        if (tid == 0) raise(p.status, flag);
        return;
    }
    const long long rs = ld(slot_row + max(acc - 1, 0));
    if (rs < 0) return;                             // a padded sequence
    if (rs >= p.num_slots || cin >= p.num_conv_slots || cout >= p.num_conv_slots) {
        if (tid == 0) raise(p.status, GDN_FLAG_SLOT_RANGE);
        return;
    }
    u64 S[R][4];
    const int64_t tile = static_cast<int64_t>(N) * p.P;
    const int64_t at = h * tile + static_cast<int64_t>(rg * R) * p.P + pb * kPB;
    {
        const StateT* src = static_cast<const StateT*>(p.pool) + rs * p.H * tile + at;
#pragma unroll
        for (int j = 0; j < R; ++j) Row8<StateT>::load(src + static_cast<int64_t>(j) * p.P, cg, S[j]);
    }
    // ---- rows, decays, the gate's quads: every thread finds the rows it needs, so that the
    //      projection's rows are on their way together with the state ----
    int bad = 0;
    auto row_at = [&](int t) {
        const int r = p.sti ? ld(p.sti + bos + t) : bos + t;
        if (r >= 0 && r < p.num_tokens) return r;
        bad = 1;
        return 0;                                   // (no row exists only where bad data is reported anyway)
    };
    const int to = tid >> 4, qo = tid & 15;         // the token and column quad this thread writes out
    const int col = h * p.P + pb * kPB;
    uint2 zraw = make_uint2(0, 0);
    if (p.z && to < n) zraw = ld(reinterpret_cast<const uint2*>(p.z + row_at(to) * p.z_stride + col + 4 * qo));
    // quad q of x | B | C, all tokens
    const int W = p.conv_width;
    const int HP = p.H * p.P;
    const int ch = tid < 16           ? col + 4 * tid
                   : tid < 16 + N / 4 ? HP + g * N + 4 * (tid - 16)
                                      : HP + p.G * N + g * N + 4 * (tid - 16 - N / 4);
    uint2 raw[kMaxT + 3];                           // history (the last 3 before the step), then the step's rows
    if (tid < kQuads) {
        const __nv_bfloat16* hist =
            cin < 0 ? nullptr : p.conv_pool + (cin * p.conv_state_len + max(acc, 1)) * static_cast<int64_t>(p.conv_dim) + ch;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int m = k - (4 - W);              // history row m of W - 1
            raw[k] = make_uint2(0, 0);
            if (m >= 0 && hist) raw[k] = ld(reinterpret_cast<const uint2*>(hist + static_cast<int64_t>(m) * p.conv_dim));
        }
#pragma unroll
        for (int t = 0; t < kMaxT; ++t)
            if (t < n) raw[3 + t] = ld(reinterpret_cast<const uint2*>(p.x + row_at(t) * p.x_stride + ch));
    } else if (tid - kQuads < n) {                  // (the threads behind the quads: at least 48)
        const int t = tid - kQuads, r = row_at(t);
        s.row[t] = r;
        s.slot[t] = ld(slot_row + t);
        const float d = softplus(__bfloat162float(p.dt[r * p.dt_stride + h]) + __bfloat162float(p.dt_bias[h]));
        s.step[t] = d;
        s.decay[t] = expf(-expf(ld(p.A_log + h)) * d);
    }
    // ---- the convolution ----
    if (tid < kQuads) {
        u64 wt2[2][4], bias2[2] = {0, 0};           // taps right-aligned: tap 3 is the token itself
        {
            float wt[4][4], b4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    wt[e][k] = k >= 4 - W ? __bfloat162float(p.conv_w[static_cast<int64_t>(ch + e) * W + k - (4 - W)]) : 0.f;
            if (p.conv_b) unpack4(ld(reinterpret_cast<const uint2*>(p.conv_b + ch)), b4);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                bias2[e] = pk2(b4[2 * e], b4[2 * e + 1]);
#pragma unroll
                for (int k = 0; k < 4; ++k) wt2[e][k] = pk2(wt[2 * e][k], wt[2 * e + 1][k]);
            }
        }
        float* dst = tid < 16 ? &s.x[0][4 * tid] : tid < 16 + N / 4 ? &s.B[0][4 * (tid - 16)] : &s.C[0][4 * (tid - 16 - N / 4)];
        const int pitch = tid < 16 ? 64 : N;
#pragma unroll
        for (int t = 0; t < kMaxT; ++t) {
            if (t >= n) break;
            u64 y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                y[e] = bias2[e];
#pragma unroll
                for (int k = 0; k < 4; ++k)         // a tap that the width lacks reads no row, so adds nothing
                    if (k >= 4 - W) y[e] = ffma2(wt2[e][k], widen(e ? raw[t + k].y : raw[t + k].x), y[e]);
                y[e] = silu2(y[e]);
            }
            *reinterpret_cast<float4*>(dst + t * pitch) = make_float4(lo2(y[0]), hi2(y[0]), lo2(y[1]), hi2(y[1]));
        }
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) raise(p.status, GDN_FLAG_TOKEN_ROW);
        return;
    }
    // the new conv slot: the history, then this step's rows; a group's B and C once
    if (cout >= 0 && tid < kQuads && (tid < 16 || (h % p.group == 0 && pb == 0))) {
        __nv_bfloat16* o = p.conv_pool + cout * p.conv_state_len * static_cast<int64_t>(p.conv_dim) + ch;
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k >= 4 - W) *reinterpret_cast<uint2*>(o + static_cast<int64_t>(k - (4 - W)) * p.conv_dim) = raw[k];
#pragma unroll
        for (int t = 0; t < kMaxT; ++t)
            if (t < n) *reinterpret_cast<uint2*>(o + static_cast<int64_t>(W - 1 + t) * p.conv_dim) = raw[3 + t];
    }
    // ---- the tokens ----
    for (int t = 0; t < n; ++t) {
        token<StateT, N>(S, s, t);
        const long long ws = s.slot[t];
        if (ws >= 0 && ws < p.num_slots) {
            StateT* dst = static_cast<StateT*>(p.pool) + ws * p.H * tile + at;
#pragma unroll
            for (int j = 0; j < R; ++j) Row8<StateT>::store(dst + static_cast<int64_t>(j) * p.P, cg, S[j]);
        } else if (ws >= 0 && tid == 0) {
            raise(p.status, GDN_FLAG_SLOT_RANGE);
        }
    }
    __syncthreads();
    if (to < n)
        write_out(s, to, qo, p.D ? ld(p.D + h) : 0.f, p.z != nullptr, zraw,
                  p.out + s.row[to] * p.out_stride + col + 4 * qo);
}

template <typename StateT>
cudaError_t launch_decode(const Params& p, int N, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(p.batch) * p.H * p.blocks), 1, 1);
    cfg.blockDim = dim3(kRThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return N == 64 ? cudaLaunchKernelEx(&cfg, gdn_ssm_decode_kernel<StateT, 64>, p)
                   : cudaLaunchKernelEx(&cfg, gdn_ssm_decode_kernel<StateT, 128>, p);
}

// sizes that both entry points of the layer share
gdn_status check_dims(const gdn_ssm_dims* d) {
    if (d == nullptr) return GDN_ERR_NULL_ARG;
    if (d->batch < 0 || d->num_tokens < 0 || d->num_tokens > kMaxRows || d->H < 1 || d->G < 1 || d->H % d->G != 0 || d->P < 1 || d->N < 1 ||
        d->num_slots < 1 || d->x_stride < 0 || d->b_stride < 0 || d->c_stride < 0 || d->dt_stride < 0 ||
        d->z_stride < 0 || d->out_stride < 0 || d->reserved[0] != 0 || d->reserved[1] != 0)
        return GDN_ERR_BAD_SHAPE;
    if ((d->N != 64 && d->N != 128) || d->P % kPB != 0 || d->P > 256) return GDN_ERR_UNSUPPORTED;
    if (d->H > (1 << 20) || static_cast<int64_t>(d->batch) * d->H * (d->P / kPB) > 0x7fffffffLL) return GDN_ERR_BAD_SHAPE;
    return GDN_OK;
}

// what both fill in and check the same way; strides come in resolved
gdn_status make_params(Params& p, const void* dt, const void* z, const float* A_log, const void* dt_bias, const float* D,
                       void* pool, const int32_t* cu, void* out, const gdn_ssm_dims* d, int32_t* status) {
    if (!dt || !A_log || !dt_bias || !pool || !cu || !out) return GDN_ERR_NULL_ARG;
    const int64_t HP = static_cast<int64_t>(d->H) * d->P;
    p = Params{};
    p.dt = static_cast<const __nv_bfloat16*>(dt);
    p.z = static_cast<const __nv_bfloat16*>(z);
    p.A_log = A_log;
    p.dt_bias = static_cast<const __nv_bfloat16*>(dt_bias);
    p.D = D;
    p.pool = pool;
    p.cu = cu;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.status = status;
    p.dt_stride = d->dt_stride ? d->dt_stride : d->H;
    p.z_stride = d->z_stride ? d->z_stride : HP;
    p.out_stride = d->out_stride ? d->out_stride : HP;
    p.num_slots = d->num_slots;
    p.batch = d->batch;
    p.num_tokens = d->num_tokens;
    p.H = d->H;
    p.G = d->G;
    p.P = d->P;
    p.group = d->H / d->G;
    p.blocks = d->P / kPB;
    if (!aligned(pool, 16) || !aligned(dt, 2) || !aligned(dt_bias, 2) || !aligned(A_log, 4) || !aligned(D, 4) ||
        !aligned(cu, 4) || !aligned(status, 4))
        return GDN_ERR_MISALIGNED;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_conv_prefill(const void* x, const void* conv_weight, const void* conv_bias, void* conv_pool,
                            const int32_t* conv_in, const int32_t* conv_out, const int32_t* cu_seqlens, void* y,
                            int32_t batch, int32_t num_tokens, int32_t conv_dim, int64_t y_stride,
                            const gdn_conv_dims* cdims, int32_t* status_word, gdn_stream_t stream) {
    if (cdims == nullptr) return GDN_ERR_NULL_ARG;
    // (channels: those that a CTA's threads would have behind the last one stay in 32 bits)
    if (batch < 0 || num_tokens < 0 || batch > kMaxScanned || num_tokens > kMaxRows || conv_dim < 1 || conv_dim > kMaxRows ||
        conv_dim % 4 != 0 || y_stride < 0 || cdims->x_stride < 0 || cdims->width < 1 || cdims->width > 4 ||
        cdims->state_len < cdims->width || cdims->num_conv_slots < 1 || cdims->reserved[0] != 0 || cdims->reserved[1] != 0)
        return GDN_ERR_BAD_SHAPE;
    if (batch == 0 || num_tokens == 0) return GDN_OK;
    if (!x || !conv_weight || !conv_pool || !conv_in || !conv_out || !cu_seqlens || !y) return GDN_ERR_NULL_ARG;
    if (!aligned(x, 8) || !aligned(y, 8) || !aligned(conv_pool, 8) || !aligned(conv_weight, 8) || !aligned(conv_bias, 8) ||
        !aligned(conv_in, 4) || !aligned(conv_out, 4) || !aligned(cu_seqlens, 4) || !aligned(status_word, 4) ||
        cdims->x_stride % 4 != 0 || y_stride % 4 != 0)
        return GDN_ERR_MISALIGNED;
    ConvParams p;
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.w = static_cast<const __nv_bfloat16*>(conv_weight);
    p.bias = static_cast<const __nv_bfloat16*>(conv_bias);
    p.pool = static_cast<__nv_bfloat16*>(conv_pool);
    p.in = conv_in;
    p.out = conv_out;
    p.cu = cu_seqlens;
    p.y = static_cast<__nv_bfloat16*>(y);
    p.status = status_word;
    p.x_stride = cdims->x_stride ? cdims->x_stride : conv_dim;
    p.y_stride = y_stride ? y_stride : conv_dim;
    p.num_slots = cdims->num_conv_slots;
    p.slot = static_cast<int64_t>(cdims->state_len) * conv_dim;
    p.batch = batch;
    p.num_tokens = num_tokens;
    p.dim = conv_dim;
    // 8 channels a thread need twice the registers of 4, so half as many warps are resident: with few rows
    // for each that shows (4096 rows of 2560 channels, 17 a thread: 13.4 us with 8, 12.5 with 4; 1000 of
    // 2560, 4: 6.1 and 5.3; 2048 of 4352, 14: 11.9 and 11.0), with many the wider accesses do (16211 of 4352,
    // 113: 52.1 and 56.6; 2048 of 8448, 28: 16.9 and 19.1; 8000 of 2560, 33: 20.1 and 21.8)
    constexpr int kWideRows = 20;
    const int64_t resident = static_cast<int64_t>(sm_count() ? sm_count() : 148) * 512;
    const bool wide = static_cast<int64_t>(num_tokens) * (conv_dim / 8) >= kWideRows * resident && conv_dim % 8 == 0 && p.x_stride % 8 == 0 && p.y_stride % 8 == 0 && aligned(x, 16) && aligned(y, 16) &&
                      aligned(conv_pool, 16) && aligned(conv_bias, 16);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = wide ? launch_conv<8>(p, cdims->width, st) : launch_conv<4>(p, cdims->width, st);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_ssm_decode(const void* xbc, const void* conv_weight, const void* conv_bias, void* conv_pool,
                          const int32_t* conv_in, const int32_t* conv_out, const gdn_conv_dims* cdims, const void* dt,
                          const void* z, const float* A_log, const void* dt_bias, const float* D, void* state_pool,
                          const int32_t* state_indices, const int32_t* num_accepted, const int32_t* cu_seqlens,
                          const int32_t* spec_token_indx, void* out, const gdn_ssm_dims* dims, gdn_dtype state_dtype,
                          int32_t* status_word, gdn_stream_t stream) {
    const gdn_status ds = check_dims(dims);
    if (ds != GDN_OK) return ds;
    if (cdims == nullptr) return GDN_ERR_NULL_ARG;
    const int64_t conv_dim = static_cast<int64_t>(dims->H) * dims->P + 2 * static_cast<int64_t>(dims->G) * dims->N;
    if (dims->spec_stride < 1 || dims->max_T < 1 || dims->max_T > kMaxT || cdims->width < 1 || cdims->width > 4 ||
        cdims->num_conv_slots < 1 || cdims->x_stride < 0 || cdims->reserved[0] != 0 || cdims->reserved[1] != 0 ||
        static_cast<int64_t>(cdims->state_len) < cdims->width - 1 + static_cast<int64_t>(dims->spec_stride) ||
        conv_dim > 0x7fffffffLL)
        return GDN_ERR_BAD_SHAPE;
    if (!is_dtype(state_dtype)) return GDN_ERR_UNSUPPORTED;
    if (dims->batch == 0 || dims->num_tokens == 0) return GDN_OK;
    if (!xbc || !conv_weight || !conv_pool || !conv_in || !conv_out || !state_indices || !num_accepted)
        return GDN_ERR_NULL_ARG;
    Params p;
    const gdn_status ps = make_params(p, dt, z, A_log, dt_bias, D, state_pool, cu_seqlens, out, dims, status_word);
    if (ps != GDN_OK) return ps;
    if (!aligned(xbc, 8) || !aligned(conv_weight, 2) || !aligned(conv_bias, 8) || !aligned(conv_pool, 8) || !aligned(z, 8) ||
        !aligned(out, 8) || !aligned(conv_in, 4) || !aligned(conv_out, 4) || !aligned(state_indices, 4) ||
        !aligned(num_accepted, 4) || !aligned(spec_token_indx, 4) || cdims->x_stride % 4 != 0 || p.z_stride % 4 != 0 ||
        p.out_stride % 4 != 0)
        return GDN_ERR_MISALIGNED;
    p.x = static_cast<const __nv_bfloat16*>(xbc);
    p.x_stride = cdims->x_stride ? cdims->x_stride : conv_dim;
    p.conv_w = static_cast<const __nv_bfloat16*>(conv_weight);
    p.conv_b = static_cast<const __nv_bfloat16*>(conv_bias);
    p.conv_pool = static_cast<__nv_bfloat16*>(conv_pool);
    p.conv_in = conv_in;
    p.conv_out = conv_out;
    p.num_conv_slots = cdims->num_conv_slots;
    p.conv_dim = static_cast<int32_t>(conv_dim);
    p.conv_width = cdims->width;
    p.conv_state_len = cdims->state_len;
    p.idx = state_indices;
    p.num_acc = num_accepted;
    p.sti = spec_token_indx;
    p.stride = dims->spec_stride;
    p.max_T = dims->max_T;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = state_dtype == GDN_F32    ? launch_decode<float>(p, dims->N, st)
                            : state_dtype == GDN_BF16 ? launch_decode<__nv_bfloat16>(p, dims->N, st)
                                                      : launch_decode<__half>(p, dims->N, st);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int64_t gdn_ssm_prefill_workspace(const gdn_ssm_dims* dims) {
    if (check_dims(dims) != GDN_OK) return -1;
    return prefill_workspace(dims->batch, dims->num_tokens, dims->H * (dims->P / kPB), dims->N);
}

gdn_status gdn_ssm_prefill(const void* x, const void* B, const void* C, const void* dt, const void* z, const float* A_log,
                           const void* dt_bias, const float* D, void* state_pool, const int32_t* read_slots,
                           const int32_t* write_slots, const int32_t* cu_seqlens, void* out, void* workspace,
                           int64_t workspace_bytes, const gdn_ssm_dims* dims, gdn_dtype state_dtype, int32_t* status_word,
                           gdn_stream_t stream) {
    const gdn_status ds = check_dims(dims);
    if (ds != GDN_OK) return ds;
    if (!is_dtype(state_dtype)) return GDN_ERR_UNSUPPORTED;
    if (dims->batch == 0 || dims->num_tokens == 0) return GDN_OK;
    if (!x || !B || !C || !read_slots || !write_slots) return GDN_ERR_NULL_ARG;
    Params p;
    const gdn_status ps = make_params(p, dt, z, A_log, dt_bias, D, state_pool, cu_seqlens, out, dims, status_word);
    if (ps != GDN_OK) return ps;
    const int64_t need = gdn_ssm_prefill_workspace(dims);
    if (need > 0 && !workspace) return GDN_ERR_NULL_ARG;
    if (workspace_bytes < need) return GDN_ERR_BAD_SHAPE;
    const int64_t GN = static_cast<int64_t>(dims->G) * dims->N;
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.B = static_cast<const __nv_bfloat16*>(B);
    p.C = static_cast<const __nv_bfloat16*>(C);
    p.x_stride = dims->x_stride ? dims->x_stride : static_cast<int64_t>(dims->H) * dims->P;
    p.b_stride = dims->b_stride ? dims->b_stride : GN;
    p.c_stride = dims->c_stride ? dims->c_stride : GN;
    p.read_slots = read_slots;
    p.write_slots = write_slots;
    if (!aligned(x, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(z, 16) || !aligned(out, 16) ||
        !aligned(workspace, 16) || !aligned(read_slots, 4) || !aligned(write_slots, 4) || p.x_stride % 8 != 0 ||
        p.b_stride % 8 != 0 || p.c_stride % 8 != 0 || p.z_stride % 8 != 0 || p.out_stride % 8 != 0)
        return GDN_ERR_MISALIGNED;
    const cudaError_t err = launch_prefill(p, dims->N, state_dtype, workspace, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
