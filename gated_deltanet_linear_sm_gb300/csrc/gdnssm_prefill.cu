// libgdnspec: the state-space layer over prompts (gdn_ssm_prefill, whose C
// entry point and argument checks are in gdnssm.cu) on the sm_103a tensor cores.
//
// Chunked form (Q = 128 tokens; S the N x 64 state block at the chunk start; l_t
// the running sum of the log2-decays inside the chunk; d_t the step sizes):
//     y_t = 2^(l_t) S^T C_t + sum_{s <= t} 2^(l_t - l_s) d_s (C_t . B_s) x_s
//     S  <- 2^(l_last) S + sum_s B_s (2^(l_last - l_s) d_s x_s)^T
// the token recurrence unrolled over the chunk, the same quantities in exact
// arithmetic.  Every decay factor is 2^(non-positive), so nothing overflows.
//
// One CTA works on a (sequence, head, 64 columns of the head dim), chunk by
// chunk, with four products of 128 rows (tcgen05.mma, bf16 operands, FP32
// accumulators in tensor memory):
//     G  = C B^T          rows t, columns s     128 x 128 x N
//     Y1 = Pm X           rows t, columns p     128 x  64 x 128, Pm = G with the decays, causal,
//                                               and D on its diagonal
//     Y2 = C S            rows t, columns p     128 x  64 x N
//     dS = B^T Xw         rows n, columns p     128 x  64 x 128, Xw_s = 2^(l_last - l_s) d_s x_s
// B, C and x are bf16 and exact.  What is computed in FP32 (Pm, S, Xw) enters as
// a bf16 hi and a bf16 lo part, together within 2^-18 of its value, each part a
// product of its own in the same accumulator; the state itself stays in FP32
// registers.  With the hi parts alone an FP32 state would be off by 2^-9.
//
// x, B, C and z come by TMA (128-byte swizzle, the operand layout of the tensor
// cores), so x, B and C are operands as they land; B^T and X as the operand
// with rows and depth exchanged need no transposed copy.  Pm goes back into the
// tensor memory that G was in and is multiplied from there.
//
// Twenty warps.  0-7 keep the state: they update S, write its images and finish
// the outputs; 12-19 turn G into Pm and weigh the next chunk's x, ahead of the
// others, since neither depends on the state; one warp each issues the products,
// issues the copies, turns dt into decay factors some chunks ahead, and stores the
// outputs.  (Two warps share the 32 rows of tensor memory that the hardware lets
// them reach, and split the columns.)  In the first launch over segments 0-7 weigh.
// They meet at mbarriers only.  dS of a chunk does not depend on the state either,
// so the chain from chunk to chunk is the FP32 update of S and the product Y2.
// Arithmetic runs on pairs of columns (fma.rn.f32x2).
//
// A chunk takes 4850 cycles with every SM at work (2.6 us; N = 128, gated): G, Pm
// and Y1 one after another are 4400 of them, the state's warps are busy for 4000
// (2050 for the outputs, 1024 of which the exponentials and reciprocals of the gate
// fill their pipe), and the tensor pipe for 41 %.  16384 tokens of 64 heads take 210
// us, 38 of them in the first launch (452 MB and 113 MB of DRAM traffic: 2.7 TB/s).
// Loops that are not unrolled are so because five kinds of warps share the
// instruction cache: with all of them unrolled that case took 466 us instead of 363.
// Every wait is bounded: on a timeout the CTA sets GDN_FLAG_TIMEOUT, writes no
// state, waits (bounded) for what it has in flight and releases its tensor
// memory.
//
// With few (sequence, head) pairs the prompts are cut into segments: a first
// launch computes what the tokens before the last segment add to the state (dS
// alone: no G, Pm, Y1, Y2), by parts of a segment, two CTAs an SM, and copies the
// initial state; the second starts each segment from that copy and the parts
// before it, which it combines itself (it does not read the slot: the sequence's
// last segment may be writing it).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "gdn_internal.h"
#include "gdn_tcgen05.h"
#include "gdnssm.h"
#include "gdnssm_recur.cuh"

using namespace gdn_common;
using namespace gdn_ssm;
using namespace gdn_tc;

namespace {

constexpr int kQ = 128;                          // tokens of a chunk
constexpr int kWarps = 8;                        // that keep the state; as many make Pm
constexpr int kMma = kWarps, kLoad = kWarps + 1, kGate = kWarps + 2, kStore = kWarps + 3;   // and a warp each
constexpr int kPm = kWarps + 4;                  // the first that makes Pm (a multiple of 4)
constexpr int kSThreads = 32 * (2 * kWarps + 4);
constexpr int kStatesThreads = 32 * (kWarps + 3);
constexpr int kGates = 3;                        // chunks whose decay factors are held
constexpr float kLost = 1.0f;                    // no log2-decay: those are not positive

struct ScanParams {
    CUtensorMap x, B, C, z, out;                 // boxes of 64 elements x 128 rows
    Params p;
    float* part;                                 // segments: [part][unit] of N x 64, what a part of one adds
    float* part_decay;                           // and its log2-decay, [part][unit] (kLost: it was given up)
    int32_t seg_chunks;                          // chunks of a segment (0: whole sequences)
    int32_t parts, part_chunks;                  // parts of a segment in the first launch, and their chunks
    int32_t part_room;                           // parts that the workspace holds, initial states among them
    uint32_t wait_limit;
};

// ---- shared memory (from a 1024-byte aligned base) ------------------------------
// Tiles of 128-byte rows, 16-byte unit j of row r at r * 128 + ((j ^ (r & 7)) << 4).
// (The first launch over segments has x, B and Xw only, and room for two CTAs an SM;
// a product with 128 rows of a 64-row B^T reads on into Xw: rows that nobody uses.)
template <int N, bool kStates>
struct Lay {
    static constexpr int kTile = kQ * 128;                      // 128 rows
    static constexpr int kXStages = kStates ? 2 : 3;
    static constexpr int kX = 0;                                // kXStages tiles [s][p]
    static constexpr int kZ = kX + kXStages * kTile;            // 2 tiles [t][p]: z, then the outputs
    static constexpr int kB = kZ + (kStates ? 0 : 2 * kTile);   // N / 64 tiles [s][64 n]
    static constexpr int kC = kB + N / 64 * kTile;              // N / 64 tiles [t][64 n]
    static constexpr int kXw = kC + (kStates ? 0 : N / 64 * kTile);   // hi, lo [s][p]
    static constexpr int kS = kXw + 2 * kTile;                  // hi, lo [n][p], N rows each
    static constexpr int kMisc = kS + (kStates ? 0 : 2 * N * 128);
    static constexpr uint32_t kTmem = kStates ? 128 : 512;      // tensor-memory columns
    static constexpr uint32_t kTdS = kStates ? 0 : 384;         // dS, the hi and the lo part's product side by side
};

// Decay factors of one chunk.  The log2-decays are added up as whole multiples
// of 2^-32 in 64 bits: after a strong decay an FP32 sum is thousands with steps
// of 2^-10, and the difference of two neighbours, whose weight is near 1, would
// be off by as much.
struct alignas(16) Gates {
    float l[kQ];       // running sum of the log2-decays: its multiple of 1/16,
    float l_lo[kQ];    // and the rest
    float f[kQ];       // 2^(l at the end of the token's block of 32 - l_t) d_t
    float e[kQ];       // 2^(l_t)
    float w[kQ];       // 2^(l_last - l_t) d_t
    float d[kQ];       // step sizes
    float total;       // 2^(l_last)
    long long units;   // l_last in units of 2^-32, at least -2^43 (2^-2048 is 0 as it is)
};

struct alignas(16) Misc {
    Gates gates[kGates];
    unsigned long long x_full[3], bc_full, z_full[2];    // copies have landed
    unsigned long long gates_full[kGates];
    unsigned long long g_done, ds_done, y2_done, y1_done[2];    // products are complete
    unsigned long long ready, xw_ready, p_ready, y_free, chunk_done[2];   // the tile warps have written / read
    unsigned long long z_free[2];                               // the outputs have left their buffer
    unsigned long long drain;
    uint32_t tmem;
    int abort;
};
template <int N, bool kStates>
constexpr int scan_smem() { return Lay<N, kStates>::kMisc + static_cast<int>(sizeof(Misc)) + 1024; }
static_assert(sizeof(Gates) % 16 == 0 && Lay<64, false>::kMisc % 16 == 0 && Lay<128, true>::kMisc % 16 == 0, "float4 accesses");
static_assert(scan_smem<128, false>() <= 227 * 1024 && 2 * (scan_smem<128, true>() + 1024) <= 228 * 1024, "shared memory budget");

// tensor-memory columns
constexpr uint32_t kTG = 0;                      // G, then Pm in its place
constexpr uint32_t kTY1 = 128;                   // two Y1 of 64
constexpr uint32_t kTY2 = 256;                   // Y2, the hi and the lo part's product side by side; then dS

// ---- instructions -----------------------------------------------------------------

// MN-major operand: rows of 64 elements are the depth (K) direction; 8-row groups
// are 1024 bytes apart, the next 64 rows of the product `mn` bytes
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t mn) {
    return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(mn >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}
constexpr uint32_t kAMn = 1u << 15, kBMn = 1u << 16;            // instruction descriptor: MN-major A, B

// Products and their completion, by the lane that leads.  The whole warp runs up to
// each instruction, so that the compiler keeps the descriptors in uniform registers
// (with one lane alone in the loop every product took twice the instructions).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
        : "memory");
}
// A from tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit_to(unsigned long long* bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(saddr(bar)),
        "r"(lead)
        : "memory");
}
__device__ __forceinline__ uint32_t elect() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes;
}

__device__ __forceinline__ void tm_ld16_nowait(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void bar_init(unsigned long long* b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned long long* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(unsigned long long* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, unsigned long long* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(saddr(bar))
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Bounded wait for phase `use` of a barrier: 2^17 polls that sleep up to 20 us each,
// or, with a bound set by gdn_set_wait_limit, that many that do not sleep.  As few
// instructions as it takes: there are some twenty waits in the five kinds of warps,
// and what they add to the instruction stream shows (a bound by the clock and a look
// at the other warps' state in each poll cost 15 % of the kernel's time).
__device__ __forceinline__ bool wait(unsigned long long* bar, int use, uint32_t limit) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred P, Q;\n\t.reg .u32 n;\n\tmov.u32 n, %3;\n"
        "POLL_%=:\n\tmbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2, %4;\n\t@P bra DONE_%=;\n\t"
        "sub.u32 n, n, 1;\n\tsetp.ne.u32 Q, n, 0;\n\t@Q bra POLL_%=;\n"
        "DONE_%=:\n\tselp.u32 %0, 1, 0, P;\n\t}"
        : "=r"(done)
        : "r"(saddr(bar)), "r"(use & 1), "r"(limit ? limit : 1u << 17), "r"(limit ? 0u : 20000u)
        : "memory");
    return done != 0;
}

// Whole multiples of 2^-32 (up to 2^20 in size): from a float above -2048; their
// multiple of 1/16, exact in FP32, and the rest; and their value.  Through 32-bit
// conversions: the 64-bit ones run on a slow pipe.
__device__ __forceinline__ long long to_units(float x) {
    const int a = __float2int_rn(x * 16.0f);
    const int b = __float2int_rn((x - static_cast<float>(a) * 0.0625f) * 4294967296.0f);
    return (static_cast<long long>(a) << 28) + b;
}
__device__ __forceinline__ float units_hi(long long v) { return static_cast<float>(static_cast<int>(v >> 28)) * 0.0625f; }
__device__ __forceinline__ float units_lo(long long v) {
    return static_cast<float>(static_cast<int>(v & 0x0fffffff)) * (1.0f / 4294967296.0f);
}
__device__ __forceinline__ float from_units(long long v) { return units_hi(v) + units_lo(v); }

// x as bf16 hi and lo words: lo = bf16(x - hi), the difference exact
__device__ __forceinline__ void split_pair(u64 x, uint32_t& hi, uint32_t& lo) {
    hi = pack2(lo2(x), hi2(x));
    const u64 r = ffma2(widen(hi), dup2(-1.0f), x);
    lo = pack2(lo2(r), hi2(r));
}
__device__ __forceinline__ void split_quads(const u64* x, uint4& hi, uint4& lo) {
    split_pair(x[0], hi.x, lo.x);
    split_pair(x[1], hi.y, lo.y);
    split_pair(x[2], hi.z, lo.z);
    split_pair(x[3], hi.w, lo.w);
}
__device__ __forceinline__ u64 gate_pair(u64 o, uint32_t zw) { return fmul2(o, silu2(widen(zw))); }

__device__ __forceinline__ uint32_t unit16(int r, int j) { return static_cast<uint32_t>(r * 128 + ((j ^ (r & 7)) << 4)); }

// 32 consecutive elements of a state row <-> pairs of FP32
__device__ __forceinline__ void load_row32(const float* p, u64 (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(p) + j);
        x[2 * j] = pk2(v.x, v.y);
        x[2 * j + 1] = pk2(v.z, v.w);
    }
}
__device__ __forceinline__ u64 to_pair(uint32_t w, __nv_bfloat16) { return widen(w); }
__device__ __forceinline__ u64 to_pair(uint32_t w, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pk2(f.x, f.y);
}
__device__ __forceinline__ uint32_t from_pair(u64 x, __nv_bfloat16) { return pack2(lo2(x), hi2(x)); }
__device__ __forceinline__ uint32_t from_pair(u64 x, __half) {
    const __half2 h = __floats2half2_rn(lo2(x), hi2(x));
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void load_row32(const T* p, u64 (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + j);
        x[4 * j] = to_pair(v.x, T());
        x[4 * j + 1] = to_pair(v.y, T());
        x[4 * j + 2] = to_pair(v.z, T());
        x[4 * j + 3] = to_pair(v.w, T());
    }
}
__device__ __forceinline__ void store_row32(float* p, const u64 (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        __stcs(reinterpret_cast<float4*>(p) + j, make_float4(lo2(x[2 * j]), hi2(x[2 * j]), lo2(x[2 * j + 1]), hi2(x[2 * j + 1])));
}
template <typename T>
__device__ __forceinline__ void store_row32(T* p, const u64 (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        __stcs(reinterpret_cast<uint4*>(p) + j, make_uint4(from_pair(x[4 * j], T()), from_pair(x[4 * j + 1], T()),
                                                           from_pair(x[4 * j + 2], T()), from_pair(x[4 * j + 3], T())));
}

// A part of a segment in the workspace: the row of thread hh * N + row, 16 bytes of every
// thread in turn, so that a warp's accesses are consecutive (row by row, 32 of them
// apart, a part took 2.5 us to read).  p: where the thread's first 16 bytes are.
template <int N>
__device__ __forceinline__ void load_part(const float* p, u64 (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p) + j * 2 * N);
        x[2 * j] = pk2(v.x, v.y);
        x[2 * j + 1] = pk2(v.z, v.w);
    }
}
template <int N>
__device__ __forceinline__ void store_part(float* p, const u64 (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        __stcg(reinterpret_cast<float4*>(p) + j * 2 * N, make_float4(lo2(x[2 * j]), hi2(x[2 * j]), lo2(x[2 * j + 1]), hi2(x[2 * j + 1])));
}

// What this CTA works on.  kind 0: nothing.
struct Work {
    int kind, seq, bos, len;                     // rows of the whole sequence
    int first, chunks;                           // chunks of this CTA
    int part, parts;                             // segments: the part to write, or the first to start from and their number
    bool last;
};

// The whole-sequence form: of every 32 sequences the longest first, so that the CTAs
// of the last round are short ones.  With segments, the
// launch's index is looked up among the sequences' counts: of segments, or (the
// states alone) of the parts before each sequence's last segment.  In the
// workspace a sequence of several segments has its initial state, then those
// parts.  One warp, 32 sequences at a time; every warp does the same.  Bad data is
// reported once: by the first CTA of every 32 sequences, or, with segments, by the
// second launch's first CTA, which therefore looks at all sequences.
template <bool kStates>
__device__ Work find_work(const ScanParams& sp, int index, int lane) {
    const Params& p = sp.p;
    Work w = {};
    auto bounds = [&](int i, int& bos, int& eos) {
        bos = ld(p.cu + i);
        eos = ld(p.cu + i + 1);
        if (eos <= bos) return 0;
        if (bos < 0 || eos > p.num_tokens) return GDN_FLAG_TOKEN_ROW;
        if (ld(p.read_slots + i) >= p.num_slots || ld(p.write_slots + i) >= p.num_slots) return GDN_FLAG_SLOT_RANGE;
        return -1;
    };
    if (sp.seg_chunks == 0) {
        const int i0 = index & ~31, i = i0 + lane;
        int bos = 0, eos = 0, len = 0, rank = 0;
        if (i < p.batch) {
            const int f = bounds(i, bos, eos);
            if (f > 0 && index == i0 && threadIdx.x < 32) raise(p.status, f);
            if (f == -1) len = eos - bos;
        }
        for (int o = 0; o < min(32, p.batch - i0); ++o) {
            const int other = __shfl_sync(kFull, len, o);
            rank += other > len || (other == len && o < lane);
        }
        const unsigned hit = __ballot_sync(kFull, i < p.batch && rank == index - i0);
        const int src = __ffs(hit) - 1;
        bos = __shfl_sync(kFull, bos, src);
        len = __shfl_sync(kFull, len, src);
        if (len > 0) w = {1, i0 + src, bos, len, 0, (len + kQ - 1) / kQ, 0, 0, true};
        return w;
    }
    int base = 0, room_base = 0;
    for (int i0 = 0; i0 < p.batch; i0 += 32) {
        const int i = i0 + lane;
        int bos = 0, eos = 0, n = 0;
        if (i < p.batch) {
            const int f = bounds(i, bos, eos);
            if (!kStates && f > 0 && blockIdx.x == 0 && threadIdx.x < 32) raise(p.status, f);
            if (f == -1) n = ((eos - bos + kQ - 1) / kQ + sp.seg_chunks - 1) / sp.seg_chunks;
        }
        const int parts = n > 0 ? (n - 1) * sp.parts : 0, count = kStates ? parts : n;
        const int room = parts > 0 ? parts + 1 : 0;
        int upto = count, room_upto = room;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, upto, o), y = __shfl_up_sync(kFull, room_upto, o);
            if (lane >= o) upto += x, room_upto += y;
        }
        const int end = base + upto;
        const unsigned hit = __ballot_sync(kFull, end > index && end - count <= index);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            const int k = index - __shfl_sync(kFull, end - count, src);          // which of the sequence's
            w.kind = 1;
            w.seq = i0 + src;
            w.bos = __shfl_sync(kFull, bos, src);
            w.len = __shfl_sync(kFull, eos, src) - w.bos;
            w.part = __shfl_sync(kFull, room_base + room_upto - room, src) + (kStates ? 1 + k : 0);
            const int whole = (w.len + kQ - 1) / kQ, each = kStates ? sp.part_chunks : sp.seg_chunks;
            w.first = k * each;
            w.chunks = min(each, whole - w.first);
            const int segments = __shfl_sync(kFull, n, src);
            w.parts = kStates ? 1 : segments > 1 ? 1 + k * sp.parts : 0;
            w.last = k + 1 == segments;
            // (an initial state comes with the part behind it, whose CTA writes it)
            const int span = !kStates && w.parts == 1 ? 2 : w.parts;
            if (w.part < 0 || span > sp.part_room || w.part > sp.part_room - span) {
                // offsets that overlap (more rows than there are)
                if (threadIdx.x == 0) raise(p.status, GDN_FLAG_TOKEN_ROW);
                w.kind = 0;
            }
            if (kStates || blockIdx.x != 0) return w;
        }
        base += __shfl_sync(kFull, upto, 31);
        room_base += __shfl_sync(kFull, room_upto, 31);
    }
    return w;
}

// kStates: the first launch over segments, which only computes what each adds to the state.
template <typename StateT, int N, bool kStates>
__global__ void __launch_bounds__(kStates ? kStatesThreads : kSThreads, kStates ? 2 : 1) gdn_ssm_scan_kernel(const __grid_constant__ ScanParams sp) {
    using L = Lay<N, kStates>;
    const Params& p = sp.p;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
    Misc& ms = *reinterpret_cast<Misc*>(sm + L::kMisc);
    const uint32_t sbase = saddr(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = p.H * p.blocks;
    const int unit = static_cast<int>(blockIdx.x % units), index = static_cast<int>(blockIdx.x / units);
    const int h = unit / p.blocks, pb = unit - h * p.blocks, g = h / p.group;
    const int col = h * p.P + pb * kPB;
    if (tid == 0) {
        prefetch_map(&sp.x);
        prefetch_map(&sp.B);
        if (!kStates) {
            prefetch_map(&sp.C);
            prefetch_map(&sp.out);
            if (p.z) prefetch_map(&sp.z);
        }
    }
    dep_wait();
    dep_launch();
    const Work wk = find_work<kStates>(sp, index, lane);
    if (wk.kind == 0) return;

    if (warp == kMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&ms.tmem)),
                     "n"(L::kTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int k = 0; k < L::kXStages; ++k) bar_init(&ms.x_full[k], 1);
        for (int k = 0; k < kGates; ++k) bar_init(&ms.gates_full[k], 1);
        bar_init(&ms.bc_full, 1);
        for (int k = 0; k < 2; ++k) {
            bar_init(&ms.z_full[k], 1);
            bar_init(&ms.z_free[k], 1);
            bar_init(&ms.y1_done[k], 1);
            bar_init(&ms.chunk_done[k], kWarps);
        }
        bar_init(&ms.g_done, 1);
        bar_init(&ms.ds_done, 1);
        bar_init(&ms.y2_done, 1);
        bar_init(&ms.ready, kWarps);
        bar_init(&ms.xw_ready, kWarps);
        bar_init(&ms.y_free, kWarps);
        bar_init(&ms.p_ready, kWarps);
        bar_init(&ms.drain, 1);
        ms.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = ms.tmem;
    const uint32_t limit = sp.wait_limit;
    const bool gated = p.z != nullptr;
    volatile int* abort = &ms.abort;
    const int row0 = wk.bos + wk.first * kQ;                     // first row of this CTA
    const int left = wk.len - wk.first * kQ;                     // rows from there to the end of the sequence
    auto rows_of = [&](int c) { return min(kQ, left - c * kQ); };
    // Phase `use` of a barrier.  A role never waits for a phase that the barrier
    // may have left behind by two (the parity would stand for the later one): who
    // completes phase use + 1 waits, itself or through others, for what the
    // waiter does after phase use.  need_warp: the whole warp takes one answer.
    bool ok = true;
    auto need = [&](unsigned long long* bar, int use) {
        if (ok && !wait(bar, use, limit)) {
            ok = false;
            *abort = 1;
        }
        return ok;
    };
    auto need_warp = [&](unsigned long long* bar, int use) {
        if (ok && !__all_sync(kFull, wait(bar, use, limit))) {
            ok = false;
            *abort = 1;
        }
        return ok;
    };

    // Xw of chunk c, and the rows past the sequence's end cleared
    auto weigh = [&](int c, int row, int hh) {
        if (!need_warp(&ms.gates_full[c % kGates], c / kGates) || !need_warp(&ms.x_full[c % L::kXStages], c / L::kXStages)) return;
        const int n = rows_of(c);
        unsigned char* X = sm + L::kX + c % L::kXStages * L::kTile;
        const u64 w2 = dup2(ms.gates[c % kGates].w[row]);
        if (n < kQ) {
            if (!need_warp(kStates ? &ms.bc_full : &ms.g_done, c)) return;     // (G has read B)
            if (row >= n) {
                const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(X + unit16(row, 4 * hh + j)) = zero;
#pragma unroll
                for (int j = 0; j < N / 16; ++j) {           // this half of the row's N / 8 units
                    const int u = hh * (N / 16) + j;
                    *reinterpret_cast<uint4*>(sm + L::kB + (u >> 3) * L::kTile + unit16(row, u & 7)) = zero;
                }
            }
        }
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
            const uint32_t at = unit16(row, 4 * hh + j);
            const uint4 v = *reinterpret_cast<const uint4*>(X + at);
            const u64 x[4] = {fmul2(widen(v.x), w2), fmul2(widen(v.y), w2), fmul2(widen(v.z), w2), fmul2(widen(v.w), w2)};
            uint4 hi, lo;
            split_quads(x, hi, lo);
            *reinterpret_cast<uint4*>(sm + L::kXw + at) = hi;
            *reinterpret_cast<uint4*>(sm + L::kXw + L::kTile + at) = lo;
        }
    };

    if (warp == kMma) {
        // ---- products ----
        {
            const uint32_t lead = elect();
            constexpr uint32_t id_g = (1u << 4) | (1u << 7) | (1u << 10) | (128u >> 3 << 17) | (128u >> 4 << 24);
            constexpr uint32_t id_y2 = id_g | kBMn, id_ds = id_g | kAMn | kBMn;
            constexpr uint32_t id_y1 = (1u << 4) | (1u << 7) | (1u << 10) | (64u >> 3 << 17) | (128u >> 4 << 24) | kBMn;
            // operands as their descriptors, formed once; a step along the depth adds its bytes / 16.
            // The hi and lo tiles of Xw and of S are one operand of 128 columns: a product of 64 takes as long.
            const uint64_t c_km = desc_sw128(sbase + L::kC), b_km = desc_sw128(sbase + L::kB);
            const uint64_t b_mn = desc_mn(sbase + L::kB, L::kTile), xw_mn = desc_mn(sbase + L::kXw, L::kTile);
            const uint64_t s_mn = desc_mn(sbase + L::kS, N * 128), x_mn0 = desc_mn(sbase + L::kX, L::kTile);
            for (int c = 0; c < wk.chunks; ++c) {
                // (G of a last chunk reads what lies behind the sequence too: columns that Pm leaves out)
                if (!need_warp(&ms.bc_full, c)) break;
                fence_after();
                if (!kStates) {
                    if (c > 0 && !need_warp(&ms.y1_done[(c - 1) & 1], (c - 1) >> 1)) break;   // Pm has been used
#pragma unroll
                    for (int ks = 0; ks < N / 16; ++ks) {
                        const uint64_t o = (ks >> 2) * (L::kTile / 16) + (ks & 3) * 2;
                        mma_ss(tm + kTG, c_km + o, b_km + o, id_g, ks > 0, lead);
                    }
                    commit_to(&ms.g_done, lead);
                }
                // Xw is there; and S is, so dS of c - 1 has been read
                if (!kStates && !need_warp(&ms.xw_ready, c)) break;
                if (!need_warp(&ms.ready, c)) break;
                fence_after();
#pragma unroll
                for (int ks = 0; ks < kQ / 16; ++ks)
                    mma_ss(tm + L::kTdS, b_mn + ks * 128, xw_mn + ks * 128, id_ds, ks > 0, lead);
                commit_to(&ms.ds_done, lead);
                if (!kStates) {
                    // Y2 of chunk c - 1 has been read (so has Y1 of c - 2, before `ready`)
                    if (c > 0 && !need_warp(&ms.y_free, c - 1)) break;
                    fence_after();
#pragma unroll
                    for (int ks = 0; ks < N / 16; ++ks)
                        mma_ss(tm + kTY2, c_km + (ks >> 2) * (L::kTile / 16) + (ks & 3) * 2, s_mn + ks * 128, id_y2, ks > 0, lead);
                    commit_to(&ms.y2_done, lead);
                    if (!need_warp(&ms.p_ready, c)) break;
                    fence_after();
                    const uint64_t x_mn = x_mn0 + c % L::kXStages * (L::kTile / 16);
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int ks = 0; ks < kQ / 16; ++ks)
                            mma_ts(tm + kTY1 + (c & 1) * 64, tm + kTG + ks * 16 + part * 8, x_mn + ks * 128, id_y1, part + ks > 0, lead);
                    commit_to(&ms.y1_done[c & 1], lead);
                }
            }
            // every product issued has to finish before tensor memory goes (with the default
            // bound; long complete, unless some warp gave up)
            commit_to(&ms.drain, lead);
            if (!wait(&ms.drain, 0, 0) && lead) raise(p.status, GDN_FLAG_DRAIN);
        }
        __syncwarp();
    } else if (warp == kLoad) {
        // ---- copies, each once what it overwrites has been read ----
        if (lane == 0) {
            auto load_x = [&](int c) {
                unsigned long long* bar = &ms.x_full[c % L::kXStages];
                bar_expect(bar, L::kTile);
                tma_load(sbase + L::kX + c % L::kXStages * L::kTile, &sp.x, col, row0 + c * kQ, bar);
            };
            auto load_bc = [&](int c) {
                bar_expect(&ms.bc_full, (kStates ? 1 : 2) * (N / 64) * L::kTile);
#pragma unroll
                for (int k = 0; k < N / 64; ++k) {
                    tma_load(sbase + L::kB + k * L::kTile, &sp.B, g * N + 64 * k, row0 + c * kQ, &ms.bc_full);
                    if (!kStates) tma_load(sbase + L::kC + k * L::kTile, &sp.C, g * N + 64 * k, row0 + c * kQ, &ms.bc_full);
                }
            };
            auto load_z = [&](int c) {
                bar_expect(&ms.z_full[c & 1], L::kTile);
                tma_load(sbase + L::kZ + (c & 1) * L::kTile, &sp.z, col, row0 + c * kQ, &ms.z_full[c & 1]);
            };
            load_bc(0);
            load_x(0);
            if (wk.chunks > 1) load_x(1);
            if (!kStates && gated) load_z(0);
            int x_loads = wk.chunks > 1 ? 2 : 1, bc_loads = 1, z_loads = 1;
            for (int c = 0; c + 1 < wk.chunks; ++c) {
                if (kStates && !need(&ms.ds_done, c)) break;     // (so x of chunk c has been weighed)
                if (c + 2 < wk.chunks) {                         // into the stage of chunk c - 1, or of c
                    if (!kStates && c > 0 && !need(&ms.chunk_done[(c - 1) & 1], (c - 1) >> 1)) break;
                    load_x(c + 2);
                    ++x_loads;
                }
                if (!kStates && (!need(&ms.g_done, c) || !need(&ms.y2_done, c))) break;
                if (!kStates && !need(&ms.ds_done, c)) break;
                load_bc(c + 1);
                ++bc_loads;
                if (!kStates && gated) {
                    if (c > 0 && !need(&ms.z_free[(c + 1) & 1], (c - 1) >> 1)) break;
                    load_z(c + 1);
                    ++z_loads;
                }
            }
            // and every copy before shared memory goes
            bool landed = true;
#pragma unroll 1
            for (int k = 0; k < L::kXStages; ++k) {
                const int n = (x_loads - k + L::kXStages - 1) / L::kXStages;       // copies into this stage
                if (n > 0) landed &= wait(&ms.x_full[k], n - 1, 0);
            }
            landed &= wait(&ms.bc_full, bc_loads - 1, 0);
            if (!kStates && gated)
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    const int n = (z_loads - k + 1) / 2;
                    if (n > 0) landed &= wait(&ms.z_full[k], n - 1, 0);
                }
            if (!landed) raise(p.status, GDN_FLAG_DRAIN);
        }
        __syncwarp();
    } else if (warp == kGate) {
        // ---- decay factors ----
        const float rate = -expf(ld(p.A_log + h)) * kLog2e, bias = __bfloat162float(p.dt_bias[h]);
        __nv_bfloat16 raw[4] = {};                               // dt of four neighbouring tokens
        auto fetch = [&](int c) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = 4 * lane + k;
                if (t < rows_of(c)) raw[k] = p.dt[(static_cast<int64_t>(row0) + c * kQ + t) * p.dt_stride + h];
            }
        };
        fetch(0);
        for (int c = 0; c < wk.chunks; ++c) {
            const int n = rows_of(c);
            float d[4];
            long long l[4], up = 0;                              // sums up to and with a token
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                d[k] = 4 * lane + k < n ? softplus(__bfloat162float(raw[k]) + bias) : 0.f;
                l[k] = up += to_units(fmaxf(rate * d[k], -2048.0f));   // 2^-2048 is 0 as it is
            }
            if (c + 1 < wk.chunks) fetch(c + 1);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long a = __shfl_up_sync(kFull, up, o);
                if (lane >= o) up += a;
            }
            const long long before = up - l[3];
            const long long all = __shfl_sync(kFull, up, 31), block_end = __shfl_sync(kFull, up, lane | 7);
            float hi[4], lo[4], f[4], e[4], w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                l[k] += before;
                hi[k] = units_hi(l[k]);
                lo[k] = units_lo(l[k]);
                f[k] = ex2(from_units(block_end - l[k])) * d[k];
                e[k] = ex2(hi[k] + lo[k]);
                w[k] = ex2(from_units(all - l[k])) * d[k];
            }
            if (c >= kGates && !need_warp(&ms.chunk_done[(c - kGates) & 1], (c - kGates) >> 1)) break;   // the buffer's last readers
            Gates& gt = ms.gates[c % kGates];
            *reinterpret_cast<float4*>(gt.l + 4 * lane) = make_float4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<float4*>(gt.l_lo + 4 * lane) = make_float4(lo[0], lo[1], lo[2], lo[3]);
            *reinterpret_cast<float4*>(gt.f + 4 * lane) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(gt.e + 4 * lane) = make_float4(e[0], e[1], e[2], e[3]);
            *reinterpret_cast<float4*>(gt.w + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<float4*>(gt.d + 4 * lane) = make_float4(d[0], d[1], d[2], d[3]);
            if (lane == 0) {
                gt.total = ex2(from_units(all));
                gt.units = max(all, -(1LL << 43));
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&ms.gates_full[c % kGates]);
        }
    } else if (warp < kWarps) {
        // ---- the state, and the outputs ----
        const int quad = warp & 3, hh = warp >> 2;
        const int row = quad * 32 + lane;                        // token t or s, or state row n: this thread's lane
        const uint32_t lanes = tm + (static_cast<uint32_t>(quad * 32) << 16);
        const bool state_row = row < N;                          // whole warps
        u64 S[16];                                               // state row `row`, columns 32 hh ..
#pragma unroll
        for (int j = 0; j < 16; ++j) S[j] = 0;
        long long run = 0;                                       // the log2-decay of the part (at most 512 chunks: 2^52)
        auto part_at = [&](int part) { return static_cast<int64_t>(part) * units + unit; };
        auto part_of = [&](int part) { return sp.part + part_at(part) * N * kPB + 4 * (hh * N + row); };
        if (state_row && (kStates ? wk.first == 0 : wk.parts == 0)) {
            const long long rs = ld(p.read_slots + wk.seq);
            if (rs >= 0)
                load_row32(static_cast<const StateT*>(p.pool) + ((rs * p.H + h) * N + row) * static_cast<int64_t>(p.P) + pb * kPB +
                               32 * hh,
                           S);
        }
        if (kStates && wk.first == 0 && state_row) {             // the initial state, kept for the second launch
            store_part<N>(part_of(wk.part - 1), S);
            if (row == 0 && hh == 0) sp.part_decay[part_at(wk.part - 1)] = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) S[j] = 0;
        }
        if (!kStates) {
            // segments: the initial state, and what lies before this one
            for (int k0 = 0; k0 < wk.parts && ok; k0 += 32) {
                const int n = min(32, wk.parts - k0);            // their decays come together
                const float decay = lane < n ? ld(sp.part_decay + part_at(wk.part + k0 + lane)) : 0.f;
                if (__any_sync(kFull, decay == kLost)) {
                    ok = false;
                    *abort = 1;
                    break;
                }
                const float scale = exp2f(decay);
                for (int k = 0; k < n && state_row; ++k) {
                    const u64 a2 = dup2(__shfl_sync(kFull, scale, k));
                    u64 x[16];
                    load_part<N>(part_of(wk.part + k0 + k), x);
#pragma unroll
                    for (int j = 0; j < 16; ++j) S[j] = ffma2(a2, S[j], x[j]);
                }
            }
        }
        // the state's hi and lo images for the next chunk
        auto image = [&]() {
            if (state_row) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint4 hi, lo;
                    split_quads(S + 4 * j, hi, lo);
                    *reinterpret_cast<uint4*>(sm + L::kS + unit16(row, 4 * hh + j)) = hi;
                    *reinterpret_cast<uint4*>(sm + L::kS + N * 128 + unit16(row, 4 * hh + j)) = lo;
                }
            }
        };
        auto publish = [&]() {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(&ms.ready);
        };
        if (kStates) weigh(0, row, hh);
        else image();
        if (ok) publish();
        if (!kStates) need_warp(&ms.gates_full[0], 0);
        for (int c = 0; c < wk.chunks && ok; ++c) {
            const Gates& gt = ms.gates[c % kGates];
            // the state after this chunk
            if (!need_warp(&ms.ds_done, c)) break;
            fence_after();
            if (kStates) run += gt.units;
            if (state_row) {
                const u64 a2 = dup2(gt.total);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t x[16], y[16];
                    tm_ld16_nowait(lanes + L::kTdS + 32 * hh + 16 * half, x);
                    tm_ld16_nowait(lanes + L::kTdS + 64 + 32 * hh + 16 * half, y);
                    tm_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        S[8 * half + j] = ffma2(a2, S[8 * half + j], add2(raw2(x[2 * j], x[2 * j + 1]), raw2(y[2 * j], y[2 * j + 1])));
                }
            }
            fence_before();
            if (kStates) {
                if (c + 1 < wk.chunks) {
                    weigh(c + 1, row, hh);
                    if (!ok) break;
                    publish();
                }
            } else {
                if (!need_warp(&ms.y2_done, c)) break;           // the images may be overwritten
                if (c + 1 < wk.chunks) {
                    // (here, so that the gates are never two rounds ahead of a wait for chunk_done)
                    if (!need_warp(&ms.gates_full[(c + 1) % kGates], (c + 1) / kGates)) break;
                    image();
                    publish();
                }
                // the outputs: (2^(l_t) Y2 + Y1) silu(z); Y2 first, so that the next may be made
                fence_after();
                u64 o[16];
                const u64 et2 = dup2(gt.e[row]);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t y2[16], y3[16];
                    tm_ld16_nowait(lanes + kTY2 + 32 * hh + 16 * half, y2);
                    tm_ld16_nowait(lanes + kTY2 + 64 + 32 * hh + 16 * half, y3);
                    tm_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        o[8 * half + j] = fmul2(et2, add2(raw2(y2[2 * j], y2[2 * j + 1]), raw2(y3[2 * j], y3[2 * j + 1])));
                }
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&ms.y_free);
                if (!need_warp(&ms.y1_done[c & 1], c >> 1)) break;
                // z has landed; without it the buffer's last outputs have left
                if (gated ? !need_warp(&ms.z_full[c & 1], c >> 1) : c >= 2 && !need_warp(&ms.z_free[c & 1], (c - 2) >> 1)) break;
                fence_after();
                unsigned char* Z = sm + L::kZ + (c & 1) * L::kTile;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t y1[16];
                    tm_ld16_nowait(lanes + kTY1 + (c & 1) * 64 + 32 * hh + 16 * half, y1);
                    tm_wait_ld();
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t at = unit16(row, 4 * hh + 2 * half + j);
                        u64 v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = 8 * j + 2 * e;
                            v[e] = add2(o[8 * half + 4 * j + e], raw2(y1[k], y1[k + 1]));
                        }
                        if (gated) {
                            const uint4 z = *reinterpret_cast<const uint4*>(Z + at);
                            v[0] = gate_pair(v[0], z.x);
                            v[1] = gate_pair(v[1], z.y);
                            v[2] = gate_pair(v[2], z.z);
                            v[3] = gate_pair(v[3], z.w);
                        }
                        *reinterpret_cast<uint4*>(Z + at) = make_uint4(pack2(lo2(v[0]), hi2(v[0])), pack2(lo2(v[1]), hi2(v[1])),
                                                                       pack2(lo2(v[2]), hi2(v[2])), pack2(lo2(v[3]), hi2(v[3])));
                    }
                }
                fence_before();
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(&ms.chunk_done[c & 1]);
        }
        // what this CTA leaves, unless a warp gave up: its segment's part, or the sequence's last
        // state, rounded once
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
        if (kStates) {
            if (state_row) store_part<N>(part_of(wk.part), S);
            if (tid == 0) sp.part_decay[part_at(wk.part)] = *abort == 0 ? from_units(run) : kLost;
        } else if (*abort == 0 && state_row) {
            if (wk.last) {
                const long long ws = ld(p.write_slots + wk.seq);
                if (ws >= 0)
                    store_row32(static_cast<StateT*>(p.pool) + ((ws * p.H + h) * N + row) * static_cast<int64_t>(p.P) + pb * kPB +
                                    32 * hh,
                                S);
            }
        }
    } else if (kStates) {
        // (not launched)
    } else if (warp == kStore) {
        // ---- the outputs to memory: whole tiles by TMA (it is not the state's warps that store: their
        //      proxy fences would wait for the stores), the last rows of a sequence one by one ----
        for (int c = 0; c < wk.chunks; ++c) {
            if (!need_warp(&ms.chunk_done[c & 1], c >> 1)) break;
            const int n = rows_of(c);
            if (n == kQ) {
                if (lane == 0) {
                    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                                     reinterpret_cast<uint64_t>(&sp.out)),
                                 "r"(sbase + L::kZ + (c & 1) * L::kTile), "r"(col), "r"(row0 + c * kQ)
                                 : "memory");
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                }
            } else {
                const unsigned char* Z = sm + L::kZ + (c & 1) * L::kTile;
                for (int t = lane >> 3; t < n; t += 4)
                    *reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(row0) + c * kQ + t) * p.out_stride + col +
                                              8 * (lane & 7)) = *reinterpret_cast<const uint4*>(Z + unit16(t, lane & 7));
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&ms.z_free[c & 1]);
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    } else {
        // ---- Pm = G with the decays, causal, hi and lo, into the columns that the warp read ----
        const int quad = warp & 3, hh = (warp - kPm) >> 2;
        const int row = quad * 32 + lane;
        const float D = p.D ? ld(p.D + h) : 0.f;
        auto publish = [&]() {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(&ms.xw_ready);
        };
        weigh(0, row, hh);
        if (ok) publish();
        for (int c = 0; c < wk.chunks && ok; ++c) {
            if (!need_warp(&ms.gates_full[c % kGates], c / kGates) || !need_warp(&ms.g_done, c)) break;
            fence_after();
            const Gates& gt = ms.gates[c % kGates];
            const uint32_t G = tm + (static_cast<uint32_t>(quad * 32) << 16) + kTG + 16 * hh;
            const float lt = gt.l[row], lt_lo = gt.l_lo[row];
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {                        // this warp's 16 columns s of block j of 32
                const int s0 = 32 * j + 16 * hh;
                uint32_t hi[8], lo[8];
                if (j > quad) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) hi[k] = lo[k] = 0;
                } else {
                    uint32_t r[16];
                    tm_ld16_nowait(G + 32 * j, r);
                    tm_wait_ld();
                    if (j < quad) {
                        // 2^(l_t - l_s) d_s through the end of the block of s: both factors at most 1 (times d_s)
                        const u64 e2 = dup2(ex2((lt - gt.l[32 * j + 31]) + (lt_lo - gt.l_lo[32 * j + 31])));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(gt.f + s0 + 4 * k);
                            split_pair(fmul2(raw2(r[4 * k], r[4 * k + 1]), fmul2(e2, f.x)), hi[2 * k], lo[2 * k]);
                            split_pair(fmul2(raw2(r[4 * k + 2], r[4 * k + 3]), fmul2(e2, f.y)), hi[2 * k + 1], lo[2 * k + 1]);
                        }
                    } else {
                        const u64 lt2 = dup2(lt), lo_t2 = dup2(lt_lo), neg = dup2(-1.0f);
                        const int last = lane - 16 * hh;         // columns up to this one count; it is the diagonal
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const ulonglong2 ls = *reinterpret_cast<const ulonglong2*>(gt.l + s0 + 4 * k);
                            const ulonglong2 lo_s = *reinterpret_cast<const ulonglong2*>(gt.l_lo + s0 + 4 * k);
                            const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(gt.d + s0 + 4 * k);
                            const u64 l_s[2] = {ls.x, ls.y}, l_o[2] = {lo_s.x, lo_s.y}, d_s[2] = {d.x, d.y};
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const int s = 4 * k + 2 * q;
                                const u64 x = ffma2(l_s[q], neg, lt2), y = ffma2(l_o[q], neg, lo_t2);
                                const float x0 = ex2(lo2(x) + lo2(y)), x1 = ex2(hi2(x) + hi2(y));   // (unused beyond the diagonal)
                                const u64 v = fmul2(raw2(r[s], r[s + 1]), fmul2(pk2(x0, x1), d_s[q]));
                                float v0 = lo2(v) + (s == last ? D : 0.f), v1 = hi2(v) + (s + 1 == last ? D : 0.f);
                                v0 = s <= last ? v0 : 0.f;
                                v1 = s + 1 <= last ? v1 : 0.f;
                                split_pair(pk2(v0, v1), hi[2 * k + q], lo[2 * k + q]);
                            }
                        }
                    }
                }
                tm_st8(G + 32 * j, hi);
                tm_st8(G + 32 * j + 8, lo);
            }
            tm_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&ms.p_ready);
            if (c + 1 < wk.chunks) {
                if (!need_warp(&ms.ds_done, c)) break;           // Xw may be overwritten
                weigh(c + 1, row, hh);
                if (ok) publish();
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (tid == 0 && *abort != 0) raise(p.status, GDN_FLAG_TIMEOUT);
    if (warp == kMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(L::kTmem));
}

// ---- host side ----------------------------------------------------------------------

// rows x cols bf16, rows `stride` elements apart, read in boxes of 64 x 128
bool encode_map(CUtensorMap& map, const void* base, int64_t cols, int64_t rows, int64_t stride) {
    using Encode = PFN_cuTensorMapEncodeTiled_v12000;
    static const Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<Encode>(fn);
    }();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[2] = {64, kQ};
    const cuuint32_t estr[2] = {1, 1};
    return encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename StateT, int N, bool kStates>
cudaError_t launch_kernel(const ScanParams& sp, int64_t ctas, cudaStream_t stream) {
    auto kernel = gdn_ssm_scan_kernel<StateT, N, kStates>;
    static bool done[64] = {false};                              // shared-memory opt-in, once per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !__atomic_load_n(&done[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, scan_smem<N, kStates>());
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) __atomic_store_n(&done[dev], true, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(kStates ? kStatesThreads : kSThreads, 1, 1);
    cfg.dynamicSmemBytes = scan_smem<N, kStates>();
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, sp);
}

// How the prompts are cut: chunks of a segment (0: whole sequences) and parts of a
// segment in the first launch, whichever an estimate of the time says is shorter.
// The host knows the rows and the sequences but not their lengths; with several it
// takes the longest for twice as long as the mean (four prompts of 4096 tokens in all, 16
// heads, us whole and cut at 6 chunks: 44 and 33 with lengths far apart, 28 and 33 alike),
// and cuts all or none.  The estimate's constants, in us, are measured: a chunk takes kChunk, or kAlone while every SM pair runs one CTA; a
// chunk of the first launch kState with two CTAs an SM; a CTA's start and end kStart
// or kStateStart, and kPart for every part that it starts from; the first launch kLaunch.
// (Whole and cut: one prompt of 16384 tokens and 64 heads 312 and 210 us, of 4096 and 32
// heads 83 and 45, of 2000 and 64 heads 47 and 43, of 1000 and 16 heads 25 and 17, of 600
// and 16 heads 18.6 and 19.7; below that whole is shorter.)
struct Cut {
    int chunks, parts;
};
Cut cut(int batch, int num_tokens, int units) {
    constexpr double kChunk = 2.6, kAlone = 2.25, kState = 1.75, kStart = 5.5, kStateStart = 4.0, kPart = 0.6, kLaunch = 3.0;
    const double sms = sm_count() ? sm_count() : 148;
    const double chunks = static_cast<double>((static_cast<int64_t>(num_tokens) + kQ - 1) / kQ);
    const double mean = chunks / batch, longest = batch > 1 ? 2 * mean : mean, whole = static_cast<double>(batch) * units;
    const double c0 = 2 * whole <= sms ? kAlone : kChunk;
    // CTAs that are resident at once take as long as the longest; more, their sum and half of one
    auto several = [&](double ctas, double sum, double each, double most) {
        return ctas <= sms ? most : std::max(most, sum / sms + 0.5 * each);
    };
    double best = batch > 1 ? several(whole, (chunks * c0 + batch * kStart) * units, mean * c0 + kStart, longest * c0 + kStart)
                            : std::ceil(whole / sms) * (chunks * c0 + kStart);
    Cut take = {0, 1};
    for (int parts = 1; parts <= 4; parts *= 2)
        for (int k = parts; k < longest && k <= 512; k += parts) {
            double cost = kLaunch;
            if (batch > 1) {
                const double segments = chunks / k + 0.5 * batch, before = std::max(chunks / k - 0.5 * batch, 0.0);
                const double c = 2 * segments * units <= sms ? kAlone : kChunk, start = kStart + kPart * 0.5 * parts * longest / k;
                cost += several(segments * units, (chunks * c + segments * start) * units, k * c + start, k * c + start) +
                        std::max(std::ceil(before * parts * units / (2 * sms)), 1.0) * (k / parts * kState + kStateStart);
            } else {
                // units * before segments of k chunks, then as many shorter ones as there are units
                const double before = std::ceil(chunks / k) - 1, rest = chunks - before * k;
                const double c = 2 * (before + 1) * units <= sms ? kAlone : kChunk, start = kStart + kPart * (1 + parts * before);
                const double full = k * c + start, last = rest * c + start;
                const double rounds = std::floor(before * units / sms), busy = before * units - rounds * sms, idle = sms - busy;
                const double beside = busy > 0 ? idle * std::floor(full / last) : 0;     // that run beside the last long ones
                cost += rounds * full + (busy == 0           ? std::ceil(units / sms) * last
                                         : beside >= units ? full
                                                           : std::min(std::ceil(units / idle) * last,
                                                                      full + std::ceil((units - beside) / sms) * last)) +
                        std::ceil(before * parts * units / (2 * sms)) * (k / parts * kState + kStateStart);
            }
            if (cost < best) {
                best = cost;
                take = {k, parts};
            }
        }
    return take;
}

// At most this many segments that are not a sequence's last; and what the workspace
// holds: their parts, and an initial state for each sequence that has some.
int64_t segments_before(int num_tokens, Cut c) { return num_tokens / (static_cast<int64_t>(c.chunks) * kQ); }
int64_t part_room(int batch, int num_tokens, Cut c) {
    const int64_t n = segments_before(num_tokens, c);
    return n * c.parts + std::min<int64_t>(n, batch);
}

template <typename StateT, int N>
cudaError_t launch(ScanParams& sp, int units, void* workspace, cudaStream_t stream) {
    const Params& p = sp.p;
    const Cut c = cut(p.batch, p.num_tokens, units);
    sp.seg_chunks = c.chunks;
    sp.parts = c.parts;
    if (sp.seg_chunks == 0) return launch_kernel<StateT, N, false>(sp, static_cast<int64_t>(p.batch) * units, stream);
    sp.part_chunks = c.chunks / c.parts;
    const int64_t before = segments_before(p.num_tokens, c), room = part_room(p.batch, p.num_tokens, c);
    if (std::max(before + p.batch, room) * units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    sp.part_room = static_cast<int32_t>(room);
    sp.part = static_cast<float*>(workspace);
    sp.part_decay = sp.part + room * units * N * kPB;
    if (before > 0) {
        // (some more than there are parts, so that every part in the workspace is written whatever the offsets)
        const cudaError_t e = launch_kernel<StateT, N, true>(sp, room * units, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel<StateT, N, false>(sp, (before + p.batch) * units, stream);
}

template <int N>
cudaError_t launch_n(ScanParams& sp, gdn_dtype t, int units, void* ws, cudaStream_t s) {
    return t == GDN_F32    ? launch<float, N>(sp, units, ws, s)
           : t == GDN_BF16 ? launch<__nv_bfloat16, N>(sp, units, ws, s)
                           : launch<__half, N>(sp, units, ws, s);
}

}  // namespace

namespace gdn_ssm {

int64_t prefill_workspace(int batch, int num_tokens, int units, int N) {
    const Cut c = cut(batch, num_tokens, units);
    return c.chunks == 0 ? 0 : part_room(batch, num_tokens, c) * units * (static_cast<int64_t>(N) * kPB + 1) * 4;
}

cudaError_t launch_prefill(const Params& p, int N, gdn_dtype state_dtype, void* workspace, cudaStream_t stream) {
    ScanParams sp = {};
    sp.p = p;
    sp.wait_limit = __atomic_load_n(&gdn_internal::g_wait_limit, __ATOMIC_RELAXED);
    const int64_t HP = static_cast<int64_t>(p.H) * p.P, GN = static_cast<int64_t>(p.G) * N;
    if (!encode_map(sp.x, p.x, HP, p.num_tokens, p.x_stride) || !encode_map(sp.B, p.B, GN, p.num_tokens, p.b_stride) ||
        !encode_map(sp.C, p.C, GN, p.num_tokens, p.c_stride) ||
        (p.z && !encode_map(sp.z, p.z, HP, p.num_tokens, p.z_stride)) || !encode_map(sp.out, p.out, HP, p.num_tokens, p.out_stride))
        return cudaErrorInvalidValue;
    const int units = p.H * p.blocks;
    return N == 64 ? launch_n<64>(sp, state_dtype, units, workspace, stream)
                   : launch_n<128>(sp, state_dtype, units, workspace, stream);
}

}  // namespace gdn_ssm
