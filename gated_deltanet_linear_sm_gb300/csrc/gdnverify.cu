// libgdnspec: what runs between two steps of speculative decoding -- the
// verification of the drafted tokens (gdn_verify_drafts, and with its counts by
// request gdn_verify_drafts_by_request) and the tables of the next step
// (gdn_step_tables).  Declared in include/gdnspec.h.
#include <cooperative_groups.h>

#include "gdn_common.h"
#include "gdn_pairs.h"

namespace cg = cooperative_groups;
using namespace gdn_common;

namespace {

// ---- gdn_verify_drafts ------------------------------------------------------------
//
// One cluster of 1 to 8 CTAs per sequence.  Every CTA decides for itself which
// drafts are kept (warp 0, one lane per draft: a few dependent loads), then the
// cluster reads the one row that the next token is sampled from, once: each
// warp adds up its contiguous piece, the CTAs exchange their sums through
// distributed shared memory, and the CTA whose piece holds the crossing reads
// that one warp's piece again (it is in L2) to find the entry.
//
// A probability is held as a whole multiple of 2^-52 in 64 bits, so the sums
// are exact: the token depends neither on the order of the additions nor on
// the number of CTAs, and no floating-point prefix sum has to be reproduced.
// The integers are not made entry by entry (the conversion of a float to 64 bits
// runs on a slow pipe: it held this kernel to a tenth of the memory's rate) but
// as three sums of 22, 22 and 8 bits that floating-point additions of a constant
// leave in the low bits of a float (Sums below).  The chain of dependent loads
// bounds small batches (1 sequence of 5 rows of 32000: 5.2 us; 32 of up to 8 rows of 151936
// FP32 entries, a row of each and the drafter's where a draft was refused, 1.4 on average:
// 11.0, 2.4 TB/s), the issue slots of the sums large
// ones (256 sequences of 128256 bf16 entries: 24.7 us, 2.7 TB/s; 92 with an integer an entry).

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxDraftT = 32;                  // rows of a sequence: one lane each

struct VerifyParams {
    const void* target;
    const void* draft;
    const int32_t* tokens;
    const float* accept_u;
    const float* sample_u;
    const int32_t* cu;
    const int32_t* sti;
    const int32_t* request;                     // null: counts in batch order
    int32_t* out;
    int32_t* accepted;
    int32_t* status;
    int64_t target_stride, draft_stride, draft_seq, token_stride;
    int32_t batch, num_tokens, vocab, max_T, num_requests;
};

__device__ __forceinline__ float clamp01(float p) { return fminf(fmaxf(p, 0.0f), 1.0f); }   // NaN -> 0
// a probability in units of 2^-52 (the scaling is exact, the conversion rounds to nearest)
__device__ __forceinline__ u64 fixed(float p) {
    return static_cast<u64>(__float2ll_rn(clamp01(p) * 4503599627370496.0f));
}

// What an entry of the row counts as: p, or what the drafter's distribution
// leaves of it.  take: 0 = p (nothing to subtract), 1 = p without entry d,
// 2 = max(p - q, 0).
__device__ __forceinline__ u64 rest(int take, u64 P, u64 Q, bool at_d) {
    if (take == 2) return P > Q ? P - Q : 0;
    return (take == 1 && at_d) ? 0 : P;
}

// the E = 16 / sizeof(T) entries of one 16-byte vector, clamped to [0, 1], as pairs
// (clamped as packed words where they come packed)
template <typename T>
struct Vec;

template <>
struct Vec<float> {
    static constexpr int E = 4;
    __device__ static void pairs(uint4 v, u64 (&x)[2]) {
        x[0] = pk2(clamp01(__uint_as_float(v.x)), clamp01(__uint_as_float(v.y)));
        x[1] = pk2(clamp01(__uint_as_float(v.z)), clamp01(__uint_as_float(v.w)));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int E = 8;
    __device__ static void pairs(uint4 v, u64 (&x)[4]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 c = __hmin2(__hmax2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]), __floats2bfloat162_rn(0.f, 0.f)),
                                             __floats2bfloat162_rn(1.f, 1.f));
            x[k] = widen(*reinterpret_cast<const uint32_t*>(&c));
        }
    }
};
template <>
struct Vec<__half> {
    static constexpr int E = 8;
    __device__ static void pairs(uint4 v, u64 (&x)[4]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(__hmin2(__hmax2(*reinterpret_cast<const __half2*>(&w[k]), __floats2half2_rn(0.f, 0.f)),
                                                    __floats2half2_rn(1.f, 1.f)));
            x[k] = pk2(f.x, f.y);
        }
    }
};

__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(kFull, x, m);
    return x;
}

// The sum of fixed(p) over up to 256 entries.  Adding 2 to p in [0, 1] rounds it
// to a multiple h of 2^-22, whose integer the float's low bits hold; p - h is
// exact and at most 2^-23, so adding 1.5 * 2^-21 gives its multiple m of 2^-44 in
// the same way, and 1.5 * 2^-29 the rest's nearest multiple l of 2^-52 (to even).
// p = h + m + l then rounds as fixed(p) does.
struct Sums {
    uint32_t h = 0, m = 0, l = 0;
    static constexpr float kH = 2.0f, kM = 1.5f / (1 << 21), kL = 1.5f / (1 << 29);
    __device__ __forceinline__ void add(u64 p) {                // two entries
        const u64 t = add2(p, dup2(kH));
        const u64 r = sub2(p, add2(t, dup2(-kH)));
        const u64 u = add2(r, dup2(kM));
        const u64 q = add2(sub2(r, add2(u, dup2(-kM))), dup2(kL));
        h += static_cast<uint32_t>(t) + static_cast<uint32_t>(t >> 32);
        m += static_cast<uint32_t>(u) + static_cast<uint32_t>(u >> 32);
        l += static_cast<uint32_t>(q) + static_cast<uint32_t>(q >> 32);
    }
    // what `count` added entries sum to (32-bit sums of the parts fit: 256 * 2^22)
    __device__ __forceinline__ long long value(uint32_t count) const {
        const uint32_t hh = h - count * __float_as_uint(kH);
        const int32_t mm = static_cast<int32_t>(m - count * __float_as_uint(kM));
        const int32_t ll = static_cast<int32_t>(l - count * __float_as_uint(kL));
        return (static_cast<long long>(hh) << 30) + static_cast<long long>(mm) * 256 + ll;
    }
};

// Sums of up to 32 of these stay in 64 bits whatever a row holds, and only where what is
// left to sample from sums to 16 or more (of a distribution it does not) one of them is met.
constexpr long long kTooMuch = 1LL << 57;
constexpr u64 kRowLimit = 1ULL << 56;

struct VerifySmem {
    u64 warp_sum[kVWarps];                         // of each warp's piece
    u64 cta_sum[2][kMaxCluster];                   // and of each CTA's, written by its owner (two attempts)
    u64 scan[kVWarps], level;
    int kept, take, d, valid;                      // the decision on the drafts
    int64_t row;                                   // row to sample from
};

template <typename T>
__global__ void __launch_bounds__(kVThreads, 2) gdn_verify_kernel(const VerifyParams p) {
    constexpr int E = Vec<T>::E;
    __shared__ VerifySmem s;
    cg::cluster_group cl = cg::this_cluster();
    const int CL = static_cast<int>(cl.num_blocks());
    const int rank = static_cast<int>(cl.block_rank());
    const int i = blockIdx.x / CL;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T* target = static_cast<const T*>(p.target);
    const T* draft = static_cast<const T*>(p.draft);
    // every CTA of the cluster runs before one writes into another's memory (waited for below)
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    dep_wait();

    const float sample_u = ld(p.sample_u + i);
    // ---- which drafts stay ----
    if (warp == 0) {
        const int bos = ld(p.cu + i);
        const int eos = ld(p.cu + i + 1), last = ld(p.cu + p.batch);
        // (loaded whatever the length is, beside the offsets)
        int d = -1;
        float u = 0.f;
        if (lane < p.max_T - 1) {
            d = ld(p.tokens + i * p.token_stride + lane);
            u = ld(p.accept_u + i * p.token_stride + lane);
        }
        const int n = (eos > bos && bos >= 0) ? eos - bos : 0;
        int flag = 0;
        int64_t row = 0;
        if (eos > bos && bos < 0) {
            flag = GDN_FLAG_TOKEN_ROW;
        } else if (n > p.max_T) {
            flag = GDN_FLAG_QLEN;
        } else if (n > 0) {
            bool bad = eos > last;
            if (!bad && lane < n) {
                row = p.sti ? ld(p.sti + bos + lane) : bos + lane;
                bad = row < 0 || row >= p.num_tokens;
            }
            if (__any_sync(kFull, bad)) flag = GDN_FLAG_TOKEN_ROW;
        }
        const bool valid = n > 0 && flag == 0;
        bool keep = false, in_range = false;
        if (valid && lane < n - 1) {
            in_range = d >= 0 && d < p.vocab;
            if (in_range) {
                const float pd = clamp01(to_f(target[row * p.target_stride + d]));
                const float qd =
                    draft ? clamp01(to_f(draft[i * p.draft_seq + lane * p.draft_stride + d])) : 1.0f;
                keep = static_cast<double>(u) * static_cast<double>(qd) < static_cast<double>(pd);   // the product of two floats is exact
            }
        }
        const unsigned stays = __ballot_sync(kFull, keep);
        const int kept = valid ? min(n - 1, __ffs(~stays) - 1) : 0;   // lane n - 1 and beyond keep nothing
        const int da = __shfl_sync(kFull, d, kept);
        const bool ra = __shfl_sync(kFull, in_range ? 1 : 0, kept) != 0;
        const int64_t rowa = __shfl_sync(kFull, row, kept);
        if (lane == 0) {
            s.kept = kept;
            s.take = (valid && kept < n - 1 && ra) ? (draft ? 2 : 1) : 0;
            s.d = da;
            s.row = rowa;
            s.valid = valid;
        }
        if (rank == 0) {
            if (lane < p.max_T && !(valid && lane == kept))
                p.out[static_cast<int64_t>(i) * p.max_T + lane] = valid && lane < kept ? d : -1;
            if (lane == 0) {
                if (valid) {                       // (read only here: beside the offsets it costs 256 x 128256 2.8 us, by the
                                                   //  order that the compiler then gives the sums)
                    const int at = p.request ? ld(p.request + i) : i;
                    if (p.request && at >= p.num_requests) flag = GDN_FLAG_SLOT_RANGE;
                    else if (at >= 0) p.accepted[at] = kept + 1;
                }
                if (flag) raise(p.status, flag);
            }
        }
    }
    __syncthreads();
    if (!s.valid) {                                // the same for every CTA of the cluster
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        return;
    }

    // ---- the sums of the row's pieces ----
    int take = s.take;
    const int d = s.d, V = p.vocab;
    const T* prow = target + s.row * p.target_stride;
    const T* qrow = take == 2 ? draft + i * p.draft_seq + s.kept * p.draft_stride : prow;
    // vector v covers entries v E - mis .. v E - mis + E - 1; only those inside the row are read
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(prow) / sizeof(T)) % E);
    const bool qvec = static_cast<int>((reinterpret_cast<uintptr_t>(qrow) / sizeof(T)) % E) == mis;
    const int NV = static_cast<int>((static_cast<int64_t>(mis) + V + E - 1) / E);
    const int per = (NV + CL * kVWarps - 1) / (CL * kVWarps);
    const int v0 = min(NV, (rank * kVWarps + warp) * per), v1 = min(NV, v0 + per);
    // the warp's vectors that lie inside the row whole; the row's two ends come one by one
    const int in0 = max(v0, mis > 0 ? 1 : 0), in1 = min(v1, static_cast<int>((static_cast<int64_t>(mis) + V) / E));

    // entries count as p (take 0), as p but for entry d (1), or as max(p - q, 0) (2):
    // fixed does not decrease, so the last is fixed(max(p, q)) - fixed(q), a difference of two sums
    auto left_pair = [](u64 p, u64 q, Sums& P, Sums& Q) {
        P.add(pk2(fmaxf(lo2(p), lo2(q)), fmaxf(hi2(p), hi2(q))));
        Q.add(q);
    };
    auto piece = [&](int how) {
        // up to 256 entries a lane between two foldings into 64 bits; the loads of U vectors (UQ of each of two
        // rows) go out together (1, 2, 3 of each: 12.9, 11.2, 13.2 us for 32 sequences of 151936 FP32 entries)
        constexpr int kFold = 256 / E, U = 4, UQ = 2;
        const uint4 none = make_uint4(0, 0, 0, 0);
        long long sum = 0;
        for (int base = in0 + lane; base < in1; base += 32 * kFold) {
            Sums P, Q;
            uint32_t n = 0;
            const int stop = min(in1, base + 32 * kFold);
            if (how == 2 && qvec) {
                for (int v = base; v < stop; v += 32 * UQ) {
                    uint4 pr[UQ], qr[UQ];
#pragma unroll
                    for (int u = 0; u < UQ; ++u) {
                        const int e = (v + 32 * u) * E - mis;
                        const bool in = v + 32 * u < stop;
                        pr[u] = in ? ld(reinterpret_cast<const uint4*>(prow + e)) : none;
                        qr[u] = in ? ld(reinterpret_cast<const uint4*>(qrow + e)) : none;
                    }
#pragma unroll
                    for (int u = 0; u < UQ; ++u) {
                        u64 pe[E / 2], qe[E / 2];
                        Vec<T>::pairs(pr[u], pe);
                        Vec<T>::pairs(qr[u], qe);
#pragma unroll
                        for (int k = 0; k < E / 2; ++k) left_pair(pe[k], qe[k], P, Q);
                    }
                    n += UQ * E;
                }
            } else if (how == 2) {
                for (int v = base; v < stop; v += 32) {          // the rows lie differently: q entry by entry
                    const int e = v * E - mis;
                    u64 pe[E / 2];
                    Vec<T>::pairs(ld(reinterpret_cast<const uint4*>(prow + e)), pe);
#pragma unroll
                    for (int k = 0; k < E / 2; ++k)
                        left_pair(pe[k], pk2(clamp01(to_f(qrow[e + 2 * k])), clamp01(to_f(qrow[e + 2 * k + 1]))), P, Q);
                    n += E;
                }
            } else {
                for (int v = base; v < stop; v += 32 * U) {
                    uint4 pr[U];
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        pr[u] = v + 32 * u < stop ? ld(reinterpret_cast<const uint4*>(prow + (v + 32 * u) * E - mis)) : none;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        u64 pe[E / 2];
                        Vec<T>::pairs(pr[u], pe);
#pragma unroll
                        for (int k = 0; k < E / 2; ++k) P.add(pe[k]);
                    }
                    n += U * E;
                }
            }
            sum = min(sum + P.value(n) - (how == 2 ? Q.value(n) : 0), kTooMuch);
        }
        // the ends of the row, if they are this warp's: lane k the entry k of a cut vector
        auto cut = [&](int v) {
            const int e = v * E - mis + lane;
            if (lane < E && e >= 0 && e < V)
                sum += static_cast<long long>(rest(how == 2 ? 2 : 0, fixed(to_f(prow[e])), how == 2 ? fixed(to_f(qrow[e])) : 0, false));
        };
        if (v0 < v1 && v0 < in0) cut(v0);
        if (in1 < v1 && in1 >= in0) cut(v1 - 1);
        u64 total = warp_sum(static_cast<u64>(sum));
        if (how == 1 && d >= v0 * E - mis && d < v1 * E - mis) total -= fixed(to_f(prow[d]));
        return min(total, static_cast<u64>(kTooMuch));
    };
    u64 total = 0;
    int attempt = 0;
    for (;; ++attempt) {
        const u64 mine = piece(take);
        if (lane == 0) s.warp_sum[warp] = mine;
        __syncthreads();
        if (attempt == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (tid < CL) {
            u64 a = 0;
            for (int w = 0; w < kVWarps; ++w) a += s.warp_sum[w];
            cl.map_shared_rank(&s, tid)->cta_sum[attempt][rank] = min(a, static_cast<u64>(kTooMuch));
        }
        cl.sync();                                 // this attempt's sums are read from this CTA's own memory
        total = 0;
        for (int c = 0; c < CL; ++c) total += s.cta_sum[attempt][c];
        if (total != 0 || take == 0) break;
        take = 0;                                  // nothing left of p: sample from p itself
    }

    // ---- where the cumulative sum passes sample_u of the total ----
    const int64_t slot = static_cast<int64_t>(i) * p.max_T + s.kept;
    if (total == 0 || total >= kRowLimit) {
        if (rank == 0 && tid == 0) {
            p.out[slot] = -1;
            raise(p.status, GDN_FLAG_NO_TOKEN);
        }
        return;
    }
    if (tid == 0) {                                // (64-bit arithmetic: one thread of a CTA)
        const double x = fmax(static_cast<double>(sample_u) * static_cast<double>(total), 0.0);   // NaN -> 0
        const u64 at = x < static_cast<double>(total) ? static_cast<u64>(x) : total - 1;
        s.level = at < total ? at : total - 1;
    }
    __syncthreads();
    u64 level = s.level;
    int owner = 0;
    while (owner < CL - 1 && level >= s.cta_sum[attempt][owner]) level -= s.cta_sum[attempt][owner++];
    if (owner != rank) return;
    int w = 0;
    while (w < kVWarps - 1 && level >= s.warp_sum[w]) level -= s.warp_sum[w++];

    // the entries of that warp's piece, spread over the CTA in order
    const int w0 = min(NV, (rank * kVWarps + w) * per), w1 = min(NV, w0 + per);
    const int e_lo = max(0, w0 * E - mis), e_hi = min(V, w1 * E - mis);
    const int each = (e_hi - e_lo + kVThreads - 1) / kVThreads;
    const int m0 = min(e_hi, e_lo + tid * each), m1 = min(e_hi, m0 + each);
    auto entry = [&](int e) {
        const u64 P = fixed(to_f(prow[e]));
        return rest(take, P, take == 2 ? fixed(to_f(qrow[e])) : 0, e == d);
    };
    u64 mine = 0;
    for (int f0 = m0; f0 < m1; f0 += 128) {
        Sums P, Q;
        const int f1 = min(m1, f0 + 128);
        for (int e = f0; e < f1; ++e) {
            const float a = clamp01(to_f(prow[e])), b = take == 2 ? clamp01(to_f(qrow[e])) : 0.f;
            const bool in = take == 2 ? a > b : take == 0 || e != d;
            P.add(pk2(in ? a : 0.f, 0.f));
            Q.add(pk2(in ? b : 0.f, 0.f));
        }
        mine += P.value(2 * (f1 - f0)) - Q.value(2 * (f1 - f0));
    }
    u64 upto = mine;                               // inclusive scan over the CTA
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31) s.scan[warp] = upto;
    __syncthreads();
    for (int k = 0; k < warp; ++k) upto += s.scan[k];
    u64 before = upto - mine;
    if (before <= level && level < upto) {
        int e = m0;
        for (; e < m1 - 1; ++e) {
            before += entry(e);
            if (level < before) break;
        }
        p.out[slot] = e;
    }
}

// CTAs per sequence: as many as are resident at once (two an SM: a second round
// pays the chain of dependent loads again; 256 sequences of 128256 bf16 entries
// take 24.7 us with one CTA each; when that was 26, two each took 30) and leave each
// at least 1024 entries.
int verify_cluster(int batch, int vocab) {
    const int64_t room = 2 * static_cast<int64_t>(sm_count() ? sm_count() : 148);
    int cl = 1;
    while (cl < kMaxCluster && static_cast<int64_t>(batch) * cl * 2 <= room && vocab / (cl * 2) >= 1024) cl *= 2;
    return cl;
}

template <typename T>
cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
    const int cl = verify_cluster(p.batch, p.vocab);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * cl, 1, 1);
    cfg.blockDim = dim3(kVThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cl;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, gdn_verify_kernel<T>, p);
}

// ---- gdn_step_tables ---------------------------------------------------------------
//
// One launch.  A CTA owns a tile of 64 requests; it reads the lengths of all
// requests (batch integers, in L2) for the two prefix sums before its tile and
// the two totals, so that no CTA waits for another, then writes its tile's
// per-request tables and the row numbers of its tile's rows, one thread a row
// (a prompt's thousands of rows are spread over the CTA like any others).
// Launch latency and two dependent reads bound it (128 requests 4.6 us, 4096 with
// prompts among them 7.7).

constexpr int kTThreads = 256;
constexpr int kTile = 64;

struct TablesParams {
    const int32_t* q_lens;
    const int32_t* spec;
    const int32_t* request;
    const int32_t* slots;
    const int32_t* accepted;
    const int32_t* conv_table;
    int32_t* conv_turn;
    int32_t* cu;
    int32_t* starts;
    int32_t* indx;
    int32_t* idx;
    int32_t* acc;
    int32_t* conv_in;
    int32_t* conv_out;
    int32_t* status;
    int32_t batch, num_tokens, stride, num_requests;
};

struct Request {
    int q;            // rows of the step
    int r;            // row in the request tables (-1: none)
    bool mine;        // speculative
    int flag;
};

__device__ __forceinline__ Request request_at(const TablesParams& p, int i) {
    Request v;
    v.q = max(ld(p.q_lens + i), 0);
    v.r = p.request ? ld(p.request + i) : i;
    v.flag = 0;
    if (v.r >= p.num_requests) {
        v.flag = GDN_FLAG_SLOT_RANGE;
        v.r = -1;
    }
    v.mine = (p.spec == nullptr || ld(p.spec + i) != 0) && v.r >= 0;
    if (v.mine && v.q > p.stride) {
        v.flag |= GDN_FLAG_QLEN;
        v.mine = false;
    }
    return v;
}

__global__ void __launch_bounds__(kTThreads) gdn_step_tables_kernel(const TablesParams p) {
    __shared__ long long part[4][kTThreads / 32];
    __shared__ int start[kTile + 1], spec_start[kTile + 1];
    __shared__ bool is_mine[kTile];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int i0 = blockIdx.x * kTile, i1 = min(p.batch, i0 + kTile);
    dep_wait();

    // rows and speculative rows before the tile, and of all requests
    long long sums[4] = {0, 0, 0, 0};
    for (int i = tid; i < p.batch; i += kTThreads) {
        const Request v = request_at(p, i);
        const int m = v.mine ? v.q : 0;
        sums[2] += v.q;
        sums[3] += m;
        if (i < i0) {
            sums[0] += v.q;
            sums[1] += m;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sums[k] += __shfl_xor_sync(kFull, sums[k], o);
        if (lane == 0) part[k][warp] = sums[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        sums[k] = 0;
        for (int w = 0; w < kTThreads / 32; ++w) sums[k] += part[k][w];
    }
    const bool fits = sums[2] <= p.num_tokens;      // else an empty step
    const int before = fits ? static_cast<int>(sums[0]) : 0;
    const int spec_before = fits ? static_cast<int>(sums[1]) : 0;
    const int spec_total = fits ? static_cast<int>(sums[3]) : 0;

    // the tile's own prefix sums and per-request tables: warp 0, two requests a lane
    if (warp == 0) {
        Request v[2];
        int q[2], m[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = i0 + 2 * lane + e;
            v[e] = i < i1 ? request_at(p, i) : Request{0, -1, false, 0};
            if (v[e].flag) raise(p.status, v[e].flag);
            if (!fits) v[e].q = 0, v[e].mine = false;
            q[e] = v[e].q;
            m[e] = v[e].mine ? v[e].q : 0;
        }
        int a = q[0] + q[1], b = m[0] + m[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, a, o), y = __shfl_up_sync(kFull, b, o);
            if (lane >= o) a += x, b += y;
        }
        int sa = before + a - q[0] - q[1], sb = spec_before + b - m[0] - m[1];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            start[2 * lane + e] = sa;
            spec_start[2 * lane + e] = sb;
            is_mine[2 * lane + e] = v[e].mine;
            sa += q[e];
            sb += m[e];
        }
        if (lane == 31) start[kTile] = sa, spec_start[kTile] = sb;
        if (!fits && lane == 0 && blockIdx.x == 0) raise(p.status, GDN_FLAG_TOKEN_ROW);
    }
    __syncthreads();
    for (int k = tid; k < i1 - i0; k += kTThreads) {
        const int i = i0 + k;
        p.cu[i] = spec_start[k];
        if (p.starts) p.starts[i] = start[k];
        const int r = p.request ? ld(p.request + i) : i;
        p.acc[i] = is_mine[k] ? ld(p.accepted + r) : 0;
        if (p.conv_table) {
            int in = -1, out = -1;
            if (is_mine[k]) {
                const int c = p.conv_turn[r] & 1;
                in = ld(p.conv_table + 2 * static_cast<int64_t>(r) + c);
                out = ld(p.conv_table + 2 * static_cast<int64_t>(r) + 1 - c);
                if (start[k + 1] > start[k]) p.conv_turn[r] = 1 - c;
            }
            p.conv_in[i] = in;
            p.conv_out[i] = out;
        }
    }
    if (tid == 0 && i1 == p.batch) {
        p.cu[p.batch] = spec_start[i1 - i0];
        if (p.starts) p.starts[p.batch] = start[i1 - i0];
    }
    const int cells = (i1 - i0) * p.stride;
    for (int e = tid; e < cells; e += kTThreads) {
        const int k = e / p.stride;
        const int r = p.request ? ld(p.request + i0 + k) : i0 + k;
        p.idx[static_cast<int64_t>(i0) * p.stride + e] =
            is_mine[k] ? ld(p.slots + static_cast<int64_t>(r) * p.stride + (e - k * p.stride)) : -1;
    }
    // the rows: speculative ones first
    for (int row = start[0] + tid; row < start[i1 - i0]; row += kTThreads) {
        int lo = 0, hi = i1 - i0 - 1;               // the last request that starts at or before the row
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start[mid] <= row) lo = mid; else hi = mid - 1;
        }
        const int off = row - start[lo];
        const int at = is_mine[lo] ? spec_start[lo] + off : spec_total + (start[lo] - spec_start[lo]) + off;
        p.indx[at] = row;
    }
}

// what both entry points of the verification check and launch (request null: num_accepted in batch order)
gdn_status verify(const void* target_probs, const void* draft_probs, const int32_t* draft_tokens, const float* accept_u,
                  const float* sample_u, const int32_t* cu_seqlens, const int32_t* spec_token_indx, const int32_t* request,
                  int32_t* out_tokens, int32_t* num_accepted, const gdn_verify_dims* dims, int32_t num_requests,
                  gdn_dtype prob_dtype, int32_t* status_word, gdn_stream_t stream) {
    if (dims == nullptr) return GDN_ERR_NULL_ARG;
    if (dims->batch < 0 || dims->num_tokens < 0 || dims->vocab < 1 || dims->vocab > 0x7fff0000 || dims->max_T < 1 ||
        dims->max_T > kMaxDraftT || dims->target_stride < 0 || dims->draft_stride < 0 || dims->draft_seq < 0 ||
        dims->token_stride < 0 || dims->batch > 0x7fffffff / kMaxCluster || dims->num_tokens > kMaxRows)
        return GDN_ERR_BAD_SHAPE;
    if (num_requests < 0) return GDN_ERR_BAD_SHAPE;
    if (!is_dtype(prob_dtype)) return GDN_ERR_UNSUPPORTED;
    if (dims->batch == 0) return GDN_OK;
    if ((dims->num_tokens > 0 && !target_probs) || !sample_u || !cu_seqlens || !out_tokens || !num_accepted) return GDN_ERR_NULL_ARG;
    if (dims->max_T > 1 && (!draft_tokens || !accept_u)) return GDN_ERR_NULL_ARG;
    const uintptr_t elem = prob_dtype == GDN_F32 ? 4 : 2;
    if (!aligned(target_probs, elem) || !aligned(draft_probs, elem) || !aligned(draft_tokens, 4) ||
        !aligned(accept_u, 4) || !aligned(sample_u, 4) || !aligned(cu_seqlens, 4) || !aligned(spec_token_indx, 4) || !aligned(request, 4) ||
        !aligned(out_tokens, 4) || !aligned(num_accepted, 4) || !aligned(status_word, 4))
        return GDN_ERR_MISALIGNED;
    VerifyParams p;
    p.target = target_probs;
    p.draft = dims->max_T > 1 ? draft_probs : nullptr;
    p.tokens = draft_tokens;
    p.accept_u = accept_u;
    p.sample_u = sample_u;
    p.cu = cu_seqlens;
    p.sti = spec_token_indx;
    p.request = request;
    p.num_requests = num_requests;
    p.out = out_tokens;
    p.accepted = num_accepted;
    p.status = status_word;
    p.target_stride = dims->target_stride ? dims->target_stride : dims->vocab;
    p.draft_stride = dims->draft_stride ? dims->draft_stride : dims->vocab;
    p.draft_seq = dims->draft_seq ? dims->draft_seq : (dims->max_T - 1) * p.draft_stride;
    p.token_stride = dims->token_stride ? dims->token_stride : dims->max_T - 1;
    p.batch = dims->batch;
    p.num_tokens = dims->num_tokens;
    p.vocab = dims->vocab;
    p.max_T = dims->max_T;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = prob_dtype == GDN_F32    ? launch_verify<float>(p, s)
                            : prob_dtype == GDN_BF16 ? launch_verify<__nv_bfloat16>(p, s)
                                                     : launch_verify<__half>(p, s);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

extern "C" {

gdn_status gdn_verify_drafts(const void* target_probs, const void* draft_probs, const int32_t* draft_tokens,
                             const float* accept_u, const float* sample_u, const int32_t* cu_seqlens,
                             const int32_t* spec_token_indx, int32_t* out_tokens, int32_t* num_accepted,
                             const gdn_verify_dims* dims, gdn_dtype prob_dtype, int32_t* status_word,
                             gdn_stream_t stream) {
    return verify(target_probs, draft_probs, draft_tokens, accept_u, sample_u, cu_seqlens, spec_token_indx, nullptr, out_tokens,
                  num_accepted, dims, 0, prob_dtype, status_word, stream);
}

gdn_status gdn_verify_drafts_by_request(const void* target_probs, const void* draft_probs, const int32_t* draft_tokens,
                                        const float* accept_u, const float* sample_u, const int32_t* cu_seqlens,
                                        const int32_t* spec_token_indx, const int32_t* request, int32_t* out_tokens,
                                        int32_t* num_accepted, const gdn_verify_dims* dims, int32_t num_requests,
                                        gdn_dtype prob_dtype, int32_t* status_word, gdn_stream_t stream) {
    if (dims != nullptr && dims->batch > 0 && !request) return GDN_ERR_NULL_ARG;
    return verify(target_probs, draft_probs, draft_tokens, accept_u, sample_u, cu_seqlens, spec_token_indx, request, out_tokens,
                  num_accepted, dims, num_requests, prob_dtype, status_word, stream);
}

gdn_status gdn_step_tables(const int32_t* q_lens, const int32_t* spec, const int32_t* request,
                           const int32_t* slot_table, const int32_t* accepted, const int32_t* conv_table,
                           int32_t* conv_turn, int32_t* cu_seqlens, int32_t* row_starts, int32_t* token_indx,
                           int32_t* state_indices, int32_t* num_accepted, int32_t* conv_in, int32_t* conv_out,
                           const gdn_tables_dims* dims, int32_t* status_word, gdn_stream_t stream) {
    if (dims == nullptr) return GDN_ERR_NULL_ARG;
    if (dims->batch < 0 || dims->num_tokens < 0 || dims->spec_stride < 1 || dims->num_requests < 0 ||
        dims->batch > kMaxScanned || dims->num_tokens > kMaxRows ||
        dims->spec_stride > 0x7fffffff / kTile || (request == nullptr && dims->batch > dims->num_requests))
        return GDN_ERR_BAD_SHAPE;
    if (!cu_seqlens) return GDN_ERR_NULL_ARG;
    if (dims->batch > 0 && (!q_lens || !slot_table || !accepted || !state_indices || !num_accepted))
        return GDN_ERR_NULL_ARG;
    if (dims->num_tokens > 0 && !token_indx) return GDN_ERR_NULL_ARG;
    const bool conv = conv_table != nullptr;
    if (conv != (conv_turn != nullptr) || conv != (conv_in != nullptr) || conv != (conv_out != nullptr))
        return GDN_ERR_NULL_ARG;
    for (const void* x : {static_cast<const void*>(q_lens), static_cast<const void*>(spec),
                          static_cast<const void*>(request), static_cast<const void*>(slot_table),
                          static_cast<const void*>(accepted), static_cast<const void*>(conv_table),
                          static_cast<const void*>(conv_turn), static_cast<const void*>(cu_seqlens),
                          static_cast<const void*>(row_starts), static_cast<const void*>(token_indx),
                          static_cast<const void*>(state_indices), static_cast<const void*>(num_accepted),
                          static_cast<const void*>(conv_in), static_cast<const void*>(conv_out),
                          static_cast<const void*>(status_word)})
        if (!aligned(x, 4)) return GDN_ERR_MISALIGNED;
    const TablesParams p = {q_lens,     spec,       request,       slot_table,   accepted, conv_table,
                            conv_turn,  cu_seqlens, row_starts,    token_indx,   state_indices, num_accepted,
                            conv_in,    conv_out,   status_word,   dims->batch,  dims->num_tokens,
                            dims->spec_stride, dims->num_requests};
    // an empty batch still has its one offset, 0
    const unsigned ctas = dims->batch > 0 ? (static_cast<unsigned>(dims->batch) + kTile - 1) / kTile : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(kTThreads, 1, 1);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gdn_step_tables_kernel, p) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
