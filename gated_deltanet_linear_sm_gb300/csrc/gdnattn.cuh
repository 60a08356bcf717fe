// Internal to libgdnspec: what the two attention kernels (gdnattn_warp.cuh, gdnattn_tc.cuh) share: how a
// batch's keys are laid on one line and cut among the CTAs, loads, the references of 8-bit rows, outputs, and
// the launch that joins the parts of units that several CTAs worked on.
#pragma once

#include <cuda_fp8.h>

#include <cfloat>

#include "gdnkv.h"

namespace gdn_attn {

using namespace gdn_common;
using namespace gdn_kv;

// The reference of a row without a score yet: every finite score is above it or equal, and it is a
// reference like any other for one that is equal.
constexpr float kUnset = -FLT_MAX;
constexpr int kKeys = 16;               // a sequence's first position is rounded down to a multiple of this

// What a kernel cuts by: G::kThreads that scan, G::kPer sequences each at a time, G::kBlock keys of the line,
// G::kRows query rows of a unit, and G::kCost, what a unit costs beyond its keys, in blocks: so many places in
// front of a unit's blocks on the line have nothing to do.

// ---- the line of all units' key blocks ---------------------------------------------------

struct Span {
    int lo, hi;                         // positions that some row sees, lo rounded down to kKeys
    int n;                              // tokens
    int row0;                           // the first one's place in the order of cu_seqlens
    int blocks;                         // of G::kBlock keys
    int tiles;                          // of query rows
    int len;                            // of a unit on the line
};

template <typename G>
__device__ __forceinline__ void make_span(const AttnParams& p, int past, int n, int row0, Span& s) {
    s.n = n;
    s.row0 = row0;
    s.hi = past + n;
    s.lo = p.window > 0 && past >= p.window ? (past + 1 - p.window) & ~(kKeys - 1) : 0;
    s.blocks = (s.hi - s.lo + G::kBlock - 1) / G::kBlock;
    s.tiles = (n * p.ratio + G::kRows - 1) / G::kRows;
    s.len = s.blocks + G::kCost;
}

// A sequence's data (several are loaded before the first is looked at: their latency shows once)
struct Given {
    int a, e, past;
};
__device__ __forceinline__ Given given(const AttnParams& p, int i) {
    if (i >= p.batch) return {0, 0, 0};
    return {ld(p.cu + i), ld(p.cu + i + 1), ld(p.kv_lens + i)};
}

// A sequence's part of the line (blocks 0: nothing to do), and a flag for bad data; `end` is the last offset.
template <typename G>
__device__ __forceinline__ int span_of(const AttnParams& p, const Given& v, int end, Span& s) {
    s.blocks = 0;
    const int a = v.a, e = v.e;
    const int64_t past = v.past;
    if (e <= a) return 0;
    if (a < 0 || e > end || e > p.num_tokens) return GDN_FLAG_TOKEN_ROW;
    const int n = e - a;
    if (n > p.max_T) return GDN_FLAG_QLEN;
    if (past < 0 || past + n > static_cast<int64_t>(p.pg.cols) * p.pg.page) return GDN_FLAG_SLOT_RANGE;
    if (p.sti) {
        bool fine = true;
        for (int t = 0; t < n; ++t) {
            const int r = ld(p.sti + a + t);
            fine = fine && r >= 0 && r < p.num_tokens;
        }
        if (!fine) return GDN_FLAG_TOKEN_ROW;
    }
    make_span<G>(p, static_cast<int>(past), n, a, s);
    return 0;
}

// The line as a CTA walks it: the blocks in front of each of kT sequences at a time.
template <typename G>
struct Line {
    static constexpr int kT = G::kThreads * G::kPer;
    int64_t base;                       // blocks in front of the chunk
    int chunk;                          // first sequence of the chunk
    int64_t before[kT + 1];             // in front of each of its sequences, from base on
    int64_t warp_sum[G::kThreads / 32];
    int past[kT], n[kT], row0[kT];      // of each (where it has blocks)

    __device__ __forceinline__ void keep(int k, const Span& s) {
        past[k] = s.hi - s.n;
        n[k] = s.n;
        row0[k] = s.row0;
    }
};

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {     // (32 bits where they do: the division is part of a call's latency)
    return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

template <typename G>
__device__ __forceinline__ int64_t block_sum(Line<G>& L, int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) L.warp_sum[threadIdx.x / 32] = v;
    __syncthreads();
    int64_t sum = 0;
#pragma unroll
    for (int w = 0; w < G::kThreads / 32; ++w) sum += L.warp_sum[w];
    return sum;
}

// The blocks in front of each sequence of the chunk that begins at `first`: kPer neighbours a thread.
template <typename G>
__device__ __forceinline__ void scan_chunk(const AttnParams& p, Line<G>& L, int first, int64_t base, bool tell) {
    const int tid = threadIdx.x, lane = tid & 31;
    int64_t v[G::kPer], sum = 0;
    Given of[G::kPer];
#pragma unroll
    for (int k = 0; k < G::kPer; ++k) of[k] = given(p, first + tid * G::kPer + k);
    const int end = ld(p.cu + p.batch);
#pragma unroll
    for (int k = 0; k < G::kPer; ++k) {
        Span s;
        const int flag = span_of<G>(p, of[k], end, s);
        if (flag && tell) raise(p.status, flag);
        v[k] = 0;
        if (s.blocks > 0) {
            v[k] = static_cast<int64_t>(s.len) * s.tiles * p.groups;
            L.keep(tid * G::kPer + k, s);
        }
        sum += v[k];
    }
    const int64_t mine = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += u;
    }
    __syncthreads();
    if (lane == 31) L.warp_sum[tid / 32] = sum;
    __syncthreads();
    int64_t in = sum - mine;
#pragma unroll
    for (int w = 0; w < G::kThreads / 32; ++w)
        if (w < tid / 32) in += L.warp_sum[w];
    if (tid == 0) {
        L.before[0] = 0;
        L.chunk = first;
        L.base = base;
    }
#pragma unroll
    for (int k = 0; k < G::kPer; ++k) {
        in += v[k];
        L.before[tid * G::kPer + k + 1] = in;
    }
    __syncthreads();
}

// The whole line's length; the first chunk is scanned on the way.
template <typename G>
__device__ __forceinline__ int64_t begin_line(const AttnParams& p, Line<G>& L) {
    constexpr int kT = Line<G>::kT;
    scan_chunk<G>(p, L, 0, 0, blockIdx.x == 0);
    int64_t more = 0;
    if (p.batch > kT) {
        const int end = ld(p.cu + p.batch);
        for (int i = kT + threadIdx.x; i < p.batch; i += G::kThreads) {
            Span s;
            const int flag = span_of<G>(p, given(p, i), end, s);
            if (flag && blockIdx.x == 0) raise(p.status, flag);
            if (s.blocks > 0) more += static_cast<int64_t>(s.len) * s.tiles * p.groups;
        }
        more = block_sum<G>(L, more);
    }
    return L.before[kT] + more;
}

// The last sequence of the chunk that begins at or before block w of the line (it has blocks); a whole warp
template <typename G>
__device__ __forceinline__ int in_chunk(const Line<G>& L, int64_t w) {
    constexpr int kStep = Line<G>::kT / 32;
    static_assert(Line<G>::kT % 32 == 0 && kStep <= 32, "two looks");
    const int lane = threadIdx.x & 31;
    const int64_t x = w - L.base;
    const int near = kStep * (__popc(__ballot_sync(kFull, L.before[kStep * lane] <= x)) - 1);
    return near + __popc(__ballot_sync(kFull, lane < kStep && L.before[near + min(lane, kStep - 1)] <= x)) - 1;
}

// The sequence whose blocks contain block w of the line (0 <= w < total), chunks moving on.
template <typename G>
__device__ __forceinline__ int sequence_at(const AttnParams& p, Line<G>& L, int64_t w) {
    constexpr int kT = Line<G>::kT;
    while (w >= L.base + L.before[kT] && L.chunk + kT < p.batch) {
        const int64_t base = L.base + L.before[kT];
        const int first = L.chunk + kT;
        __syncthreads();
        scan_chunk<G>(p, L, first, base, false);
    }
    return in_chunk(L, w);
}

// The same by one warp.
template <typename G>
__device__ __forceinline__ int sequence_at_warp(const AttnParams& p, Line<G>& L, int64_t w) {
    constexpr int kT = Line<G>::kT;
    const int lane = threadIdx.x & 31;
    while (w >= L.base + L.before[kT] && L.chunk + kT < p.batch) {
        const int64_t base = L.base + L.before[kT];
        const int first = L.chunk + kT;
        __syncwarp();
        int64_t run = 0;
        const int end = ld(p.cu + p.batch);
        for (int k = 0; k < kT / 32; ++k) {
            const int i = first + 32 * k + lane;
            int64_t sum = 0;
            Span s;
            span_of<G>(p, given(p, i), end, s);
            if (s.blocks > 0) {
                sum = static_cast<int64_t>(s.len) * s.tiles * p.groups;
                L.keep(32 * k + lane, s);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(kFull, sum, o);
                if (lane >= o) sum += u;
            }
            L.before[32 * k + lane + 1] = run + sum;
            run += __shfl_sync(kFull, sum, 31);
        }
        if (lane == 0) {
            L.before[0] = 0;
            L.chunk = first;
            L.base = base;
        }
        __syncwarp();
    }
    return in_chunk(L, w);
}

// CTAs (of one member of the groups of heads) that share the line: no more than leave each `least` blocks
__device__ __forceinline__ int ctas_of(int64_t total, int grid, int least) {
    const int64_t most = (total + least - 1) / least;
    return static_cast<int>(most < grid ? (most > 0 ? most : 1) : grid);
}

// What a CTA works on next: the unit at block w of the line, up to block w1.
struct Piece {
    int seq, head, tile, rows, past, n, row0;
    int places;                         // of the line
    int b0, b1, blocks;                 // of the unit's blocks (none where b0 = b1)
    int64_t u0;                         // the line's place of the unit's first block
    int key0, key1;
};
template <typename G>
__device__ __forceinline__ Piece piece_at(const AttnParams& p, const Line<G>& L, int k, int64_t w, int64_t w1, int member) {
    Piece d;
    Span s;
    make_span<G>(p, L.past[k], L.n[k], L.row0[k], s);
    const int64_t in_seq = w - L.base - L.before[k];
    const int unit = static_cast<int>(quotient(in_seq, s.len));             // (group of heads, tile of rows)
    const int at = static_cast<int>(in_seq - static_cast<int64_t>(unit) * s.len);
    d.seq = L.chunk + k;
    d.places = static_cast<int>(w1 - w < s.len - at ? w1 - w : s.len - at);
    d.b0 = max(at - G::kCost, 0);
    d.b1 = max(at + d.places - G::kCost, 0);
    d.blocks = s.blocks;
    d.u0 = w - at + G::kCost;
    const int group = s.tiles == 1 ? unit : static_cast<int>(static_cast<uint32_t>(unit) / static_cast<uint32_t>(s.tiles));
    d.head = group * p.side + member;
    d.tile = unit - group * s.tiles;
    d.rows = min(G::kRows, s.n * p.ratio - d.tile * G::kRows);
    d.past = s.hi - s.n;
    d.n = s.n;
    d.row0 = s.row0;
    d.key0 = s.lo + d.b0 * G::kBlock;
    d.key1 = min(s.hi, s.lo + d.b1 * G::kBlock);
    return d;
}
// the record of a part that is not a whole unit (block b of the line is CTA ((b + 1) ctas - 1) / total's)
__device__ __forceinline__ void put_record(int32_t* meta, const Piece& d, int64_t total, int ctas) {
    int4* rec = reinterpret_cast<int4*>(meta) + 2 * (d.b0 > 0 ? 0 : 1);
    rec[0] = make_int4(d.seq, d.head, d.tile, static_cast<int>(quotient((d.u0 + 1) * ctas - 1, total)));
    rec[1] = make_int4(static_cast<int>(quotient((d.u0 + d.blocks) * ctas - 1, total)), d.rows, d.row0, 0);
}

// ---- instructions ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t saddr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
    const int bytes = live ? 16 : 0;    // (0: zeros, and nothing is read)
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
    const int bytes = live ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t pack_h(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_b(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- the products of weights and values' scales (8-bit caches) -----------------------------------------
//
// With P_j = 2^(s_j - m - e) |scale_j| / unit, o = sum P_j code_j and l = sum 2^(s_j - m - e), the output is
// unit o / l for any m and e of the row.  P_j goes into an operand of fp16's range, so e is kept such
// that the row's largest P is 2^kLift or more and stays below 2^(kSlack + 1): e moves as m does, by the
// products alone.  m and e are not one number: beside scores of 2^24 and more, e would be lost in it.  l is
// FP32 and needs no care: a scale counts as 2^-kFloor units at least, so 2^(s_j - m - e) stays below 2^(kFloor + kSlack),
// and scales up to 2^128 leave it 2^-104 or more.  unit = 2^16 puts the scales that have all bits at 2^-74 to 2^128
// (2^-94: half of them).
struct Product {
    static constexpr float kUnitLog2 = 16.f, kUnit = 0x1p16f, kUnitInv = 0x1p-16f, kFloor = 90.f;
    // log2 of a scale in units, rounded down (one that is no number moves nothing: it spoils the rows that see it as it is)
    __device__ __forceinline__ static float size_of(float scale) {
        const int e = static_cast<int>(__float_as_uint(scale) >> 23) & 0xff;
        return e == 255 ? -kFloor : fmaxf(static_cast<float>(e - 127) - kUnitLog2, -kFloor);
    }
    // The reference (m, e) moved to (now, ...), for products of at most 2^top beside now: the factor of what was
    // added up with the old one.
    __device__ __forceinline__ static float move(float& m, float& e, float now, float top, float lift, float slack) {
        const float old = e + (m - now), next = top > old + slack ? top - lift : old;
        m = now;
        e = next;
        return old == next ? 1.f : ex2(old - next);
    }
    // A part's sums, kept with (m, e), are joined relative to a new m: the one that makes l 1 (as far as m's own last bit
    // allows), whatever l is, since weights of values that are almost zero may be far above the products' reference.
    __device__ __forceinline__ static void settle(float& m, float& e, float l) {
        const float above = e + __log2f(l);
        if (above > 0.f) {
            const float now = m + above;
            e -= now - m;
            m = now;
        }
    }
    // The factors of l and of o then, both with 2^-16, so that sums of values up to the largest FP32 number do not
    // overflow (the joined output divides them); o's makes up for the unit.
    __device__ __forceinline__ static float of_l(float e) { return ex2(e - kUnitLog2); }
    __device__ __forceinline__ static float of_o(float e) { return ex2(e); }
};

// Lift and slack of the references of a bf16 cache: its weights have FP32's range, and this far below 1 sums
// of values up to the largest stay below infinity (4 million of them in the worst case; values down to 2^-90 keep
// their bits).
constexpr float kLiftBf = -36.f, kSlackBf = -22.f;

__device__ __forceinline__ int64_t token_row(const AttnParams& p, int i) { return p.sti ? ld(p.sti + i) : i; }

// x sigmoid(z) without a denominator that overflows: with u = e^-|z| it is x / (1 + u) or x u / (1 + u), u in two
// factors, which are normal numbers wherever the product is one
__device__ __forceinline__ float gated(float x, float z) {
    const float h = __expf(-0.5f * fabsf(z));
    return __fdividef(z < 0.f ? x * h * h : x, fmaf(h, h, 1.0f));
}

// four columns of a row, weighed: to the output, through the gate z
__device__ __forceinline__ void put_out(const AttnParams& p, int64_t at, int64_t z_at, const float (&o)[4]) {
    float x[4] = {o[0], o[1], o[2], o[3]};
    if (p.z) {
        const uint2 raw = ld(reinterpret_cast<const uint2*>(p.z + z_at));
        const float z[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u), __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u)};
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = gated(x[e], z[e]);
    }
    *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_b(x[0], x[1]), pack_b(x[2], x[3]));
}

// ---- the second launch: parts of a unit joined ------------------------------------------------------
//
// Each of the CTAs that share a unit joins some of its rows: the one at place c of c0 .. c1 of the line those whose
// number is c - c0 modulo their count, up to 16 of them to a CTA of this launch: the time is a row's chain of loads, and
// more rows than warps repeat it (units of 64 rows, 32 sequences of 8192, e4m3: the call 151 us with all rows of a CTA here,
// 143 with 32, 138 with 16, 142 with 8, when the first launch took 10 us less).  A row's parts are summed by the warps that are left over for it.

constexpr int kJThreads = 256, kJWarps = 8;
template <int kTileRows>
constexpr int kJSplit = (kTileRows + 15) / 16;      // CTAs of this launch for one of the first

template <int D, int kTileRows>
__global__ void __launch_bounds__(kJThreads) gdn_attn_join_kernel(const AttnParams p, const int grid) {
    __shared__ float sum[kJWarps][D];
    __shared__ float sum_l[kJWarps];
    dep_wait();
    dep_launch();
    const int cta = blockIdx.x / kJSplit<kTileRows>, sub_cta = blockIdx.x % kJSplit<kTileRows>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int4* const meta = reinterpret_cast<const int4*>(p.meta + static_cast<int64_t>(cta) * kMetaInts);
    const int4 rec[2][2] = {{ld(meta), ld(meta + 1)}, {ld(meta + 2), ld(meta + 3)}};
    const float* const all_ml = p.ws + static_cast<int64_t>(2 * grid) * kTileRows * D;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int4 r0 = which ? rec[1][0] : rec[0][0], r1 = which ? rec[1][1] : rec[0][1];
        if (r0.x < 0) continue;
        const int head = r0.y, tile = r0.z, c0 = r0.w, c1 = r1.x, rows = r1.y, row0 = r1.z;
        const int parts = c1 - c0 + 1, member = cta % p.side;
        const int step = parts * kJSplit<kTileRows>, mine = cta / p.side - c0 + parts * sub_cta;
        const int count = rows > mine ? (rows - mine + step - 1) / step : 0;        // rows of this CTA
        int per = 1;                                                                // warps of a row
        while (2 * per * count <= kJWarps && per < kJWarps) per *= 2;
        const int at_once = kJWarps / per;
#pragma unroll 1
        for (int base = 0; base < count; base += at_once) {
            const int j = base + warp / per, sub = warp % per;
            const int r = mine + j * step;
            constexpr int kV = D / 32;                                              // columns of a lane
            float top = -INFINITY, x[kV], l = 0.f;
#pragma unroll
            for (int e = 0; e < kV; ++e) x[e] = 0.f;
            // the first part was left by c0 as its last, the others as their first
            auto part_of = [&](int k) { return static_cast<int64_t>(2 * ((c0 + k) * p.side + member) + (k == 0 ? 1 : 0)); };
            if (j < count) {
                // every lane has the references and sums of some parts, and the first 32 of this warp in place
                float pm = -INFINITY, pl = 0.f;
                const int own = sub + lane * per;
                if (own < parts) {
                    pm = ld(all_ml + part_of(own) * 2 * kTileRows + r);
                    pl = ld(all_ml + part_of(own) * 2 * kTileRows + kTileRows + r);
                }
                for (int k = lane; k < parts; k += 32) top = fmaxf(top, ld(all_ml + part_of(k) * 2 * kTileRows + r));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
                for (int k0 = 0; sub + k0 * per < parts; k0 += 32) {
                    if (k0 > 0) {
                        const int k = sub + (k0 + lane) * per;
                        pm = k < parts ? ld(all_ml + part_of(k) * 2 * kTileRows + r) : -INFINITY;
                        pl = k < parts ? ld(all_ml + part_of(k) * 2 * kTileRows + kTileRows + r) : 0.f;
                    }
                    const float a = pm == -INFINITY ? 0.f : ex2(pm - top);
                    l += a * pl;
#pragma unroll 4
                    for (int q = 0; q < 32 && sub + (k0 + q) * per < parts; ++q) {
                        const float* src = p.ws + (part_of(sub + (k0 + q) * per) * kTileRows + r) * D;
                        const float aq = __shfl_sync(kFull, a, q);
#pragma unroll
                        for (int e = 0; e < kV; e += 2) {
                            const float2 y = ld(reinterpret_cast<const float2*>(src + 32 * e + 2 * lane));
                            x[e] += aq * y.x;                       // (a factor of 0 too: what is no number stays none)
                            x[e + 1] += aq * y.y;
                        }
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
            }
#pragma unroll
            for (int e = 0; e < kV; e += 2) *reinterpret_cast<float2*>(&sum[warp][32 * e + 2 * lane]) = make_float2(x[e], x[e + 1]);
            if (lane == 0) sum_l[warp] = l;
            __syncthreads();
            // (all rows of this pass, their columns by all threads)
            for (int id = tid; id < at_once * (D / 4); id += kJThreads) {
                const int q = id / (D / 4), col = 4 * (id - q * (D / 4));
                const int jj = base + q;
                if (jj >= count) continue;
                const int rj = mine + jj * step;
                const int rr = tile * kTileRows + rj, t = rr / p.ratio;
                const int64_t row = token_row(p, row0 + t), h = static_cast<int64_t>(head * p.ratio + rr - t * p.ratio) * D + col;
                float y[4] = {0.f, 0.f, 0.f, 0.f}, den = 0.f;
                for (int s2 = 0; s2 < per; ++s2) {
                    const float4 v = *reinterpret_cast<const float4*>(&sum[q * per + s2][col]);
                    y[0] += v.x;
                    y[1] += v.y;
                    y[2] += v.z;
                    y[3] += v.w;
                    den += sum_l[q * per + s2];
                }
                const float inv = den == 0.f ? 0.f : 1.0f / den;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] *= inv;
                put_out(p, row * p.out_stride + h, row * p.z_stride + h, y);
            }
            __syncthreads();
        }
    }
}

}  // namespace gdn_attn
