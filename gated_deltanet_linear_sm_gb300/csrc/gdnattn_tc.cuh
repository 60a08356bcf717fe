// Internal to libgdnspec: the attention of a step's tokens over the paged key-value cache on the
// tcgen05 tensor cores, for bf16, fp16 and e4m3 caches (gdnattn_bf16.cu and its like instantiate it; gdnattn.cu
// has the mathematics, the line that the work is cut from, the kernel for what does not run here, and
// the choice between the two).
//
// A unit's rows (heads of a group times tokens) are 64 at most, its keys come in tiles of 128:
//     S^T[128 keys][64 rows] = K Q^T        O^T[D][64 rows] += V^T P^T
// so the tensor core's 128 rows are always full and its columns are what is cheap: with the
// query rows as the 128 rows of S, one token of a group of 4 would use 4 of them.  K is the
// left operand as it lies in shared memory, V^T the same tile read the other way (MN-major).
// A thread has one key of a tile, so the softmax needs no exchange between threads at all
// as long as the rows' references stand (one vote a tile); sums over keys are made once
// per unit.
//
// Warps: softmax and output (a quarter of the keys each, and a half or quarter of the rows), helpers
// (what goes with a tile's keys, q, and values that are not to be taken as they lie), loads, products, the
// line.  All run over the same sequence of tiles, units behind one another, through rings: the loads are
// up to a ring ahead whatever unit that is, the scores of the next tile are made while the weights of this
// one are.  TMA brings boxes of positions that lie in one page, from a tensor of pages, heads, positions
// and elements.  What a page holds behind a unit's keys may be NaN: the helpers clear those values before
// the products take them (a score is masked; 0 times NaN is not).
//
// What bounds it: with few bytes and many rows the softmax (32 sequences of 8192, head dim 128, 64 rows, e4m3:
// 149 us, 1.9 TB/s; the time stays when the products, the exponentials, the stores or the loads are left out
// one at a time: it is the chain of a tile's steps in 4 warps a quarter), with more bytes a row
// the ring's four places (beside q and weights laid out for 64 rows, whatever the call has) and the call's start and end (2 of 65535, head dim 256, 64 rows, bf16: 62 us, 4.3 TB/s),
// and with short sequences a unit's own chain (first tile, its edge, output: 11 us with nothing beside it).
//
// bf16: weights as two bf16 parts (16 significant bits), two products.  fp16: one.  e4m3: the
// codes are operands as they are; q is the sum of three e5m2 parts (3 bits each, with its signs its 8 bits; the row's
// largest element is 2^14 to 2^15, so elements down to 2^-24 of it are exact), a weight times the
// value's scale is an fp16 number cut into four e5m2 ones of 3 bits each.  e5m2 has fp16's largest value, but no
// bits below 2^-16: the third and fourth part are of 64 times the rest, in columns of their own that
// the output adds up divided by that, so the four hold the number up to 2^-23, 2^-31 of the row's largest.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_internal.h"
#include "gdn_pairs.h"
#include "gdn_tcgen05.h"
#include "gdnattn.cuh"

namespace gdn_attn_tc {

using namespace gdn_attn;
using gdn_tc::desc_sw128;
using gdn_tc::fence_after;
using gdn_tc::fence_async_smem;
using gdn_tc::fence_before;

enum Kind { kBf16, kF16, kE4m3 };

constexpr int kTile = 128, kRowsT = 64;
constexpr int kUnits = 4;               // units known at a time
constexpr int kKeyRing = 8;             // tiles whose keys' scales and presence are known at a time
constexpr int kHelp = 4;

// Roles by warp: softmax and output, helpers, loads, products, the line.  16 softmax warps of at most two chunks of 8
// rows do better than 8 of four where a weight takes most work (32 sequences of 8192, head dim 128, 64 rows, e4m3: 6 % less
// time), 8 with twice the registers where it takes less (16 of up to 16384, head dim 256, 32 rows, bf16: 5 % less).
template <int kKind>
struct Warps {
    static constexpr int kSoft = kKind == kE4m3 ? 16 : 8;
    static constexpr int kLoad = kSoft + kHelp, kMma = kLoad + 1, kLine = kMma + 1;
    static constexpr int kThreads = (kLine + 1) * 32;
    static constexpr int kMine = kRowsT / 8 / (kSoft / 4);      // chunks of 8 rows of a softmax warp, at most
};

template <int kKind>
struct Cut {                            // (gdnattn.cuh)
    static constexpr int kThreads = Warps<kKind>::kThreads;
    static constexpr int kPer = 1, kCost = 1;
    static constexpr int kBlock = kTile;
    static constexpr int kRows = kRowsT;
};

// weights are 2^(s - m) with m = (largest score when it was set) - kLift; m moves when a weight would
// pass 2^kSlack.  8 bits: 2^(s - m - e), and e keeps weight times scale there (gdnattn.cuh: Product)
// (fp16: beside a score of 2^27, whose last bit is 16, m is rounded, and 8 below it would be 16)
constexpr float kLiftH = 7.f, kLiftQ = 8.f, kSlackH = 14.f;

template <int kKind, int D>
struct Lay {
    static constexpr bool kQuantised = kKind == kE4m3;
    static constexpr int kBytes = kQuantised ? 1 : 2;
    static constexpr int kBlocks = (D + 127) / 128;                         // of a head dim: products of 128 rows of O^T
    static constexpr int kAtoms = kQuantised || D == 64 ? 1 : 2;            // columns of 128 bytes of an item
    static constexpr int kItem = kAtoms * kTile * 128;                      // K or V of a tile, one block of the head dim
    static constexpr int kPAtoms = kKind == kF16 ? 1 : 2;
    static constexpr int kP = kPAtoms * kTile * 128;
    static constexpr int kQTerm = (kQuantised ? (D + 127) / 128 : D / 64) * kRowsT * 128;
    static constexpr int kQ = kQTerm * (kQuantised ? 3 : 1);
    static constexpr int kBudget = 198 * 1024;
    static constexpr int kQs = kQTerm <= (kQuantised ? 8 : 16) * 1024 ? 2 : 1;  // buffers of q
    static constexpr int kRing0 = (kBudget - kP - kQs * kQ) / kItem;
    static constexpr int kRing = kRing0 > 9 ? 9 : kRing0;
    // (the weights behind the ring: the products of a head dim of 64 read 64 rows of V^T more than there are, the next item's)
    static constexpr int kORing = 0, kOP = kRing * kItem, kOQ = kOP + kP, kOMisc = kOQ + kQs * kQ;
    // tensor memory: two S^T, then O^T of one or two units
    static constexpr int kOCols = kQuantised ? 128 : 64;                    // of a block
    static constexpr int kOs = kBlocks * kOCols <= 128 ? 2 : (kBlocks * kOCols * 2 + 128 <= 512 ? 2 : 1);
    static constexpr uint32_t kTO = 128;
    static_assert(kRing >= 4, "K and V of two tiles");
    static_assert(kTO + kOs * kBlocks * kOCols <= 512, "tensor memory");
};

struct TcParams {
    uint32_t limit;                     // of waits (gdn_set_wait_limit)
    int parts;                          // softmax warps of a quarter of the keys that have rows
    int chunks;                         // chunks of 8 rows of each
    int box, box_log2;                  // positions that one TMA copy brings: they divide a page
};

struct Desc {                           // a unit's part of one CTA
    int seq, head, tile, rows, past, n, row0;
    int key0, key1, tiles;              // tiles 0: no more units
    int part;                           // of the workspace, -1: finish here
    int poison;                         // a value that is no number was taken out of its tiles
};

template <int kKind>
struct Misc {
    Line<Cut<kKind>> line;
    unsigned long long full[9], empty[9], s_full[2], s_free[2], p_full, p_free, q_full[2], q_free[2], o_full[2], o_free[2];
    unsigned long long keys_full[kKeyRing], keys_free[kKeyRing], edge_full[8], fixed[8], u_full[kUnits], u_free[kUnits], qs_full[kUnits], drain;
    Desc desc[kUnits];
    uint32_t live[kKeyRing][4];                // per tile and quarter: keys that are there
    float2 scales[kKeyRing][kTile];            // of keys and values (8 bits)
    alignas(16) float q_scale[kUnits][kRowsT];
    alignas(16) float ref[2][kRowsT];      // minus the references m
    alignas(16) float shift[2][kRowsT];    // minus their e (8 bits)
    alignas(16) float alpha[kRowsT], zero[kRowsT];
    alignas(16) float col[4][kRowsT], size[4][kRowsT];
    float inv[kRowsT];
    int first[kRowsT], last[kRowsT];
    int64_t out_at[kRowsT], z_at[kRowsT];
    uint32_t tmem;
    int abort;
};

template <int kKind, int D>
constexpr int smem_of() { return Lay<kKind, D>::kOMisc + static_cast<int>(sizeof(Misc<kKind>)) + 1024; }

// ---- instructions -------------------------------------------------------------------------

__device__ __forceinline__ void bar_init(unsigned long long* b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned long long* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}
// Bounded wait for phase `use` of a barrier, as in the scan over prompts: polls that sleep up to 20 us each,
// or, with a bound set by gdn_set_wait_limit, that many that do not sleep.
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
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t mn) {
    return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(mn >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
template <bool kF8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
    if constexpr (kF8)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
            : "memory");
}
__device__ __forceinline__ void commit_to(unsigned long long* bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(saddr(bar)), "r"(lead)
        : "memory");
}
__device__ __forceinline__ uint32_t elect() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes;
}
__device__ __forceinline__ void tm_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tm_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void bar_expect(unsigned long long* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(bytes) : "memory");
}
// a box of a cache: element x, row y of a page, head, page
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int head, int page, unsigned long long* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(head), "r"(page), "r"(saddr(bar))
        : "memory");
}
// the softmax warps among themselves
__device__ __forceinline__ void soft_sync(int parts) { asm volatile("bar.sync 1, %0;" ::"r"(parts * 128) : "memory"); }
__device__ __forceinline__ bool soft_any(bool x, int parts) {
    uint32_t y;
    asm volatile("{\n\t.reg .pred P, Q;\n\tsetp.ne.u32 P, %1, 0;\n\tbar.red.or.pred Q, 1, %2, P;\n\tselp.u32 %0, 1, 0, Q;\n\t}"
                 : "=r"(y) : "r"(x ? 1u : 0u), "r"(parts * 128) : "memory");
    return y != 0;
}
__device__ __forceinline__ void st16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void st8(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// an arrival once this thread's copies so far are there
__device__ __forceinline__ void arrive_when_copied(unsigned long long* b) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(saddr(b)) : "memory");
}
// 16-byte chunk c of row r of a tile of 128-byte rows (SWIZZLE_128B)
__device__ __forceinline__ uint32_t unit16(int r, int c) { return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4)); }

// fp16 pairs as e5m2 parts: the upper byte of an fp16 number is the e5m2 one below it (towards zero).  Of a number
// below 2^15 two parts leave less than 2^9, which times 64 is below 2^15 again.
constexpr float kUp = 64.f;
__device__ __forceinline__ uint32_t upper_bytes(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7531); }
__device__ __forceinline__ uint32_t rest_of(uint32_t h) {               // exact
    const uint32_t hi = h & 0xff00ff00u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&hi));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t times_up(uint32_t h) {              // exact
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&h), __floats2half2_rn(kUp, kUp));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// A value of sequence `seq` at position x, column d, that is no number (0 if it is one)
template <int kKind>
__device__ __noinline__ float no_number(const AttnParams& p, int seq, int head, int x, int d) {
    const int page = ld(p.pg.table + static_cast<int64_t>(seq) * p.pg.table_stride + p.pg.page_of(x));
    if (page < 0 || page >= p.pg.num_pages) return 0.f;
    const int64_t at = page * p.pg.page_stride + static_cast<int64_t>(x - p.pg.page_of(x) * p.pg.page) * p.pg.token_stride + head * p.pg.head_stride + d;
    if constexpr (kKind == kE4m3) {
        return (static_cast<const uint8_t*>(p.v)[at] & 0x7f) == 0x7f ? __uint_as_float(0x7fc00000u) : 0.f;
    } else {
        const float v = kKind == kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.v)[at]) : __half2float(static_cast<const __half*>(p.v)[at]);
        return fabsf(v) < INFINITY ? 0.f : v;
    }
}

// Whether the tile at position x0 has values that its products must not take as they lie: behind the unit's keys, or
// seen by some rows only.
__device__ __forceinline__ bool is_edge(int x0, int key1, int all_lo, int all_hi) {
    return x0 < all_lo || x0 + kTile > min(key1, all_hi);
}

// column d of the values that the unit's tiles left out, added to 8 rows that see them
template <int kKind>
__device__ __noinline__ void add_no_numbers(const AttnParams& p, const Desc& d, const int* first, const int* last, int all_lo, int all_hi,
                                            int dcol, float* y) {
    for (int x = d.key0; x < d.key1; ++x) {
        if (x >= all_lo && x < all_hi) {
            x = all_hi - 1;
            continue;
        }
        const float v = no_number<kKind>(p, d.seq, d.head, x, dcol);
        for (int e = 0; e < 8; ++e)
            if (v != 0.f && x >= first[e] && x <= last[e]) y[e] += v;
    }
}

// Each of N columns joined over the 32 lanes: lane c gets column c mod N.  Halves of the columns change places
// between halves of the lanes, so it takes about N exchanges instead of 5 N.
template <int N, typename Op>
__device__ __forceinline__ float over_lanes(float (&v)[N], int lane, Op op) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < o; ++k) {
            const float mine = lane & o ? v[k + o] : v[k], other = lane & o ? v[k] : v[k + o];
            v[k] = op(mine, __shfl_xor_sync(kFull, other, o));
        }
#pragma unroll
    for (int o = 16; o >= N; o >>= 1) v[0] = op(v[0], __shfl_xor_sync(kFull, v[0], o));
    return v[0];
}

template <int kKind, int D>
__global__ void __launch_bounds__(Warps<kKind>::kThreads, 1) gdn_attn_tc_kernel(const AttnParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const TcParams tc) {
    const uint32_t limit = tc.limit;
    const int parts = tc.parts;
    using L = Lay<kKind, D>;
    using G = Cut<kKind>;
    constexpr int kSoft = Warps<kKind>::kSoft, kLoadWarp = Warps<kKind>::kLoad, kMmaWarp = Warps<kKind>::kMma, kLineWarp = Warps<kKind>::kLine;
    constexpr int kMine = Warps<kKind>::kMine;
    constexpr bool kQ8 = L::kQuantised, kB = kKind == kBf16;
    constexpr float kLift = kB ? kLiftBf : kQ8 ? kLiftQ : kLiftH, kSlack = kB ? kSlackBf : kSlackH;
    extern __shared__ unsigned char raw_smem[];
    unsigned char* const sm = raw_smem + ((1024 - (saddr(raw_smem) & 1023)) & 1023);
    Misc<kKind>& ms = *reinterpret_cast<Misc<kKind>*>(sm + L::kOMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int k = 0; k < L::kRing; ++k) {
            bar_init(&ms.full[k], 1);
            bar_init(&ms.empty[k], 1);
        }
        for (int k = 0; k < 2; ++k) {
            bar_init(&ms.s_full[k], 2);
            bar_init(&ms.s_free[k], 4 * parts);
            bar_init(&ms.q_full[k], 32 * kHelp);
            bar_init(&ms.q_free[k], 1);
            bar_init(&ms.o_full[k], 1);
            bar_init(&ms.o_free[k], 4 * parts);
        }
        bar_init(&ms.p_full, 4 * parts);
        bar_init(&ms.p_free, 1);
        bar_init(&ms.drain, 1);
        for (int k = 0; k < kKeyRing; ++k) {
            bar_init(&ms.keys_full[k], kHelp + (kQ8 ? 32 * kHelp : 0));
            bar_init(&ms.edge_full[k], L::kBlocks);
            bar_init(&ms.fixed[k], kHelp);
            bar_init(&ms.keys_free[k], 4 * parts);
        }
        for (int k = 0; k < kUnits; ++k) {
            bar_init(&ms.u_full[k], 1);
            bar_init(&ms.u_free[k], 4 * parts + kHelp + 2);
            bar_init(&ms.qs_full[k], 32 * kHelp);
        }
        ms.abort = 0;
        for (int k = 0; k < kRowsT; ++k) ms.zero[k] = 0.f;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    dep_wait();
    // (behind the wait: a predecessor that still runs may need its tensor memory on this SM, and in front of
    // dep_launch: a successor must not take it first)
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&ms.tmem)), "n"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    const int64_t total = begin_line<G>(p, ms.line);
    dep_launch();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = ms.tmem;
    const int ctas = ctas_of(total, gridDim.x / p.side, 1 + G::kCost);
    const int cta = blockIdx.x, place = cta / p.side, member = cta - place * p.side;
    volatile int* const abort = &ms.abort;
    int it = 0, edges = 0;                          // items of the ring that this role is past; edge tiles that were loaded
    const uint32_t ring = saddr(sm + L::kORing), pbuf = saddr(sm + L::kOP), qbuf = saddr(sm + L::kOQ);

    // A role never waits for a phase that the barrier may have left behind by two (the parity would stand for the
    // later one): who completes phase use + 1 waits, itself or through others, for what the waiter does after phase use.
    if (warp == kLineWarp) {
        // ---- the line: which unit comes next ----
        int32_t* const meta = p.meta + static_cast<int64_t>(cta) * kMetaInts;
        if (lane == 0) meta[0] = meta[8] = -1;
        __syncwarp();
        const int64_t w0 = place < ctas ? quotient(total * place, ctas) : 0, w1 = place < ctas ? quotient(total * (place + 1), ctas) : 0;
        int64_t w = w0;
        for (int u = 0;; ++u) {
            if (!__all_sync(kFull, wait(&ms.u_free[u % kUnits], u / kUnits + 1, limit))) {
                *abort = 1;
                break;
            }
            Desc d = {};
            Piece pc = {};
            while (w < w1) {                        // (places that have nothing to do are passed by)
                const int k = sequence_at_warp<G>(p, ms.line, w);
                pc = piece_at<G>(p, ms.line, k, w, w1, member);
                w += pc.places;
                if (pc.b0 == pc.b1) continue;
                d.seq = pc.seq;
                d.head = pc.head;
                d.tile = pc.tile;
                d.rows = pc.rows;
                d.past = pc.past;
                d.n = pc.n;
                d.row0 = pc.row0;
                d.key0 = pc.key0;
                d.key1 = pc.key1;
                d.tiles = pc.b1 - pc.b0;
                d.part = pc.b0 == 0 && pc.b1 == pc.blocks ? -1 : pc.b0 > 0 ? 2 * cta : 2 * cta + 1;
                break;
            }
            if (lane == 0) {
                ms.desc[u % kUnits] = d;
                bar_arrive(&ms.u_full[u % kUnits]);
                if (d.tiles > 0 && d.part >= 0) put_record(meta, pc, total, ctas);
            }
            __syncwarp();
            if (d.tiles == 0) break;
        }
    } else if (warp == kLoadWarp) {
        // ---- loads: K of tile t, then V of tile t - 1, in boxes of positions that lie in one page ----
        int t = 0, u = 0, j = 0;                    // tile, unit, tile of the unit
        bool ok = true;
        auto need = [&](unsigned long long* bar, int use) {
            if (ok && !__all_sync(kFull, wait(bar, use, limit))) {
                ok = false;
                *abort = 1;
            }
            return ok;
        };
        int begun = 0;                              // blocks loaded of an edge tile's V whose others are not yet
        const int boxes = kTile >> tc.box_log2;     // of a tile and 128-byte column; lane b has box b's place
        Desc d = {};
        const int32_t* table = nullptr;
        int x0 = 0, page = -1;
        int v_page = 0, v_row = 0, v_live = 0, v_head = 0;          // the previous tile's
        bool v_edge = false;
        auto page_at = [&](int x) { return lane < boxes && x < d.key1 ? ld(table + p.pg.page_of(x)) : -1; };
        // (one pass of this loop a tile, and one more for the last tile's V; each thing in one place only: the
        // instructions of a launch are fetched while it runs)
        for (bool more = true; ok;) {
            if (j == d.tiles) {                     // the next unit
                if (u > 0 && lane == 0) bar_arrive(&ms.u_free[(u - 1) % kUnits]);
                if (!need(&ms.u_full[u % kUnits], u / kUnits)) break;
                d = ms.desc[u % kUnits];
                j = 0;
                ++u;
                more = d.tiles > 0;
                if (more) {
                    table = p.pg.table + static_cast<int64_t>(d.seq) * p.pg.table_stride;
                    x0 = d.key0;
                    page = page_at(x0 + (lane << tc.box_log2));
                }
            }
            // (a page that is none: one behind the last, which reads as zeros)
            const int x = x0 + (lane << tc.box_log2);
            const int k_row = x - p.pg.page_of(x) * p.pg.page;
            const int k_page = page >= 0 && page < p.pg.num_pages ? page : static_cast<int>(p.pg.num_pages);
            const int k_live = more ? min(boxes, (d.key1 - x0 + tc.box - 1) >> tc.box_log2) : 0;
            const int k_head = d.head;
            if (more) {
                x0 += kTile;
                page = j + 1 < d.tiles ? page_at(x0 + (lane << tc.box_log2)) : -1;
            }
#pragma unroll 1
            for (int k = more ? 0 : L::kBlocks; k < (t > 0 ? 2 * L::kBlocks : L::kBlocks); ++k) {
                const bool is_k = k < L::kBlocks;
                const int block = is_k ? k : k - L::kBlocks;
                const int slot = it % L::kRing;
                if (!need(&ms.empty[slot], it / L::kRing + 1)) break;
                const int atoms = D == 192 && block == 1 ? 1 : L::kAtoms;       // (its second half is not there)
                const int live = is_k ? k_live : v_live;
                // (values that the helpers work on first land for them; the products wait for these)
                const bool to_fix = !is_k && v_edge;
                unsigned long long* const bar = to_fix ? &ms.edge_full[edges & 7] : &ms.full[slot];
                if (lane == 0) {
                    bar_expect(bar, live * atoms * tc.box * 128);
                    if (to_fix) bar_arrive(&ms.full[slot]);
                }
                __syncwarp();
                const uint32_t dst = ring + slot * L::kItem;
                for (int i = 0; i < boxes * atoms; i += 32) {
                    const int col = (i + lane) >> (7 - tc.box_log2), b = (i + lane) & (boxes - 1);
                    const int row = __shfl_sync(kFull, is_k ? k_row : v_row, b), pg = __shfl_sync(kFull, is_k ? k_page : v_page, b);
                    if (col < atoms && b < live)
                        tma_load(dst + col * kTile * 128 + b * tc.box * 128, is_k ? &k_map : &v_map, block * 128 + col * 64, row, is_k ? k_head : v_head, pg, bar);
                }
                ++it;
                if (to_fix) {
                    begun = block + 1 < L::kBlocks ? block + 1 : 0;
                    if (begun == 0) ++edges;
                }
            }
            if (!more) break;
            v_page = k_page;
            v_row = k_row;
            v_live = k_live;
            v_head = k_head;
            v_edge = is_edge(x0 - kTile, d.key1, p.window > 0 ? max(0, d.past + d.n - p.window) : 0, d.past + 1);
            ++j;
            ++t;
        }
        // (given up between an edge tile's blocks: its barrier is told not to expect the others, so that what was loaded
        // can be waited for like the rest)
        if (begun > 0) {
            if (lane == 0)
                for (int k = begun; k < L::kBlocks; ++k) bar_arrive(&ms.edge_full[edges & 7]);
            ++edges;
        }
    } else if (warp >= kSoft && warp < kSoft + kHelp) {
        // ---- what goes with a tile: its keys' presence and scales (a thread each), q of its unit, and its values where
        // they are not to be taken as they lie; 32 positions of a tile a warp ----
        const int cw = warp - kSoft, ct = tid - kSoft * 32;
        bool ok = true;
        auto need = [&](unsigned long long* bar, int use) {
            if (ok && !__all_sync(kFull, wait(bar, use, limit))) {
                ok = false;
                *abort = 1;
            }
            return ok;
        };
        int t = 0, u = 0, j = 0, fixes = 0;
        bool v_edge = false;                        // the previous tile's
        uint32_t v_partly = 0, v_lives = 0;
        int v_unit = 0;
        Desc d = {};
        const int32_t* table = nullptr;
        int all_lo = 0, all_hi = 0, x = 0, page = -1;
        constexpr int kPer = 2;                     // threads of a row of q
        constexpr int kN = D / 8 / kPer;            // 16-byte pieces of each
        const int qr = ct / kPer, qj = ct % kPer;
        auto page_at = [&](int x) { return x < d.key1 ? ld(table + p.pg.page_of(x)) : -1; };
        for (bool more = true; ok;) {
            if (j == d.tiles) {
                if (u > 0) {
                    __syncwarp();
                    if (lane == 0) bar_arrive(&ms.u_free[(u - 1) % kUnits]);
                }
                if (!need(&ms.u_full[u % kUnits], u / kUnits)) break;
                d = ms.desc[u % kUnits];
                j = 0;
                ++u;
                more = d.tiles > 0;
                if (more) {
                    table = p.pg.table + static_cast<int64_t>(d.seq) * p.pg.table_stride;
                    all_lo = p.window > 0 ? max(0, d.past + d.n - p.window) : 0;
                    all_hi = d.past + 1;
                    x = d.key0 + 32 * cw + lane;
                    page = page_at(x);
                }
            }
            if (more && j == 0) {
                // q: bf16 as it is; else its row's largest element becomes 2^14 to 2^15 (in fp16 elements down to 2^-31
                // of that are exact, in e5m2 parts to 2^-24)
                const int rr = d.tile * kRowsT + qr, tok = rr / p.ratio;
                const bool has = qr < d.rows;
                const uint4* src = reinterpret_cast<const uint4*>(p.q);
                if (has) src = reinterpret_cast<const uint4*>(p.q + token_row(p, d.row0 + tok) * p.q_stride + static_cast<int64_t>(d.head * p.ratio + rr - tok * p.ratio) * D);
                float down = 1.f, up = 1.f;
                uint4 raw[kN];
#pragma unroll
                for (int k = 0; k < kN; ++k) {
                    raw[k] = make_uint4(0, 0, 0, 0);
                    if (has) raw[k] = ld(src + qj + kPer * k);
                }
                if constexpr (!kB) {
                    uint32_t big = 0;
#pragma unroll
                    for (int k = 0; k < kN; ++k) {
                        const uint32_t w4[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) big = max(big, max(w4[e] & 0x7fffu, (w4[e] >> 16) & 0x7fffu));
                    }
                    big = max(big, __shfl_xor_sync(kFull, big, 1));
                    constexpr int kTop = 14;
                    const int e = max(static_cast<int>(big >> 7), 1 + kTop);
                    if ((big >> 7) != 255) {
                        down = __uint_as_float(static_cast<uint32_t>(254 + kTop - e) << 23);
                        up = __uint_as_float(static_cast<uint32_t>(e - kTop) << 23);
                    } else if constexpr (kQ8) {
                        up = __uint_as_float(0x7fc00000u);      // (the parts saturate: the row's scores are NaN)
                    }
                }
                const int qb = (u - 1) % L::kQs;
                if (!need(&ms.q_free[qb], (u - 1) / L::kQs + 1)) break;
                if (qj == 0) ms.q_scale[(u - 1) % kUnits][qr] = p.scale * up;
                const uint32_t q0 = qbuf + qb * L::kQ;
#pragma unroll
                for (int k = 0; k < kN; ++k) {
                    const int c = qj + kPer * k;    // elements 8 c ..
                    const uint32_t w4[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
                    if constexpr (kB) {
                        st16(q0 + (c >> 3) * kRowsT * 128 + unit16(qr, c & 7), w4[0], w4[1], w4[2], w4[3]);
                    } else {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            f[2 * e] = __uint_as_float(w4[e] << 16) * down;
                            f[2 * e + 1] = __uint_as_float(w4[e] & 0xffff0000u) * down;
                        }
                        if constexpr (kKind == kF16) {
                            st16(q0 + (c >> 3) * kRowsT * 128 + unit16(qr, c & 7), pack_h(f[0], f[1]), pack_h(f[2], f[3]), pack_h(f[4], f[5]), pack_h(f[6], f[7]));
                        } else {
                            // three parts, each the nearest e5m2 value of what is left
                            const uint32_t a = q0 + (c >> 4) * kRowsT * 128 + unit16(qr, (c >> 1) & 7) + 8 * (c & 1);
#pragma unroll
                            for (int term = 0; term < 3; ++term) {
                                uint32_t part[2] = {0, 0};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * e], f[2 * e + 1]), __NV_SATFINITE, __NV_E5M2);
                                    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(h, __NV_E5M2);
                                    const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hr));
                                    f[2 * e] -= hf.x;
                                    f[2 * e + 1] -= hf.y;
                                    part[e >> 1] |= static_cast<uint32_t>(h) << (16 * (e & 1));
                                }
                                st8(a + term * L::kQTerm, part[0], part[1]);
                            }
                        }
                    }
                }
                fence_async_smem();
                bar_arrive(&ms.q_full[qb]);
                bar_arrive(&ms.qs_full[(u - 1) % kUnits]);
            }
            bool edge = false;
            uint32_t partly = 0, lives = 0;
            if (more) {
                const bool live = page >= 0 && page < p.pg.num_pages;
                if (page >= p.pg.num_pages) raise(p.status, GDN_FLAG_SLOT_RANGE);
                edge = is_edge(d.key0 + j * kTile, d.key1, all_lo, all_hi);
                partly = __ballot_sync(kFull, live && (x < all_lo || x >= all_hi));
                lives = __ballot_sync(kFull, live);
                if (!need(&ms.keys_free[t % kKeyRing], t / kKeyRing + 1)) break;
                if (lane == 0) {
                    ms.live[t % kKeyRing][cw] = lives;
                    bar_arrive(&ms.keys_full[t % kKeyRing]);
                }
                if constexpr (kQ8) {
                    const int64_t sat = live ? page * p.pg.s_page + static_cast<int64_t>(x - p.pg.page_of(x) * p.pg.page) * p.pg.s_token + d.head * p.pg.s_head : 0;
                    const uint32_t to = saddr(&ms.scales[t % kKeyRing][32 * cw + lane]);
                    copy4(to, p.k_scale + sat, live);
                    copy4(to + 4, p.v_scale + sat, live);
                    arrive_when_copied(&ms.keys_full[t % kKeyRing]);
                }
                x += kTile;
                page = j + 1 < d.tiles ? page_at(x) : -1;
            }
            if (more) it += L::kBlocks;
            if (t > 0) {
                it += L::kBlocks;
                if (v_edge) {
                    if (!need(&ms.edge_full[fixes & 7], fixes >> 3)) break;
                    // Values behind the unit's keys are cleared (a page holds anything there).  Those that are no numbers and
                    // that some rows see and some do not would reach the others as 0 * NaN: out of the tile, the output
                    // adds them where they are seen.
                    bool bad = false;
#pragma unroll 1
                    for (int b = 0; b < L::kBlocks; ++b) {
                        const int slot = (it - L::kBlocks + b) % L::kRing;
                        const uint32_t dst = ring + slot * L::kItem;
#pragma unroll 1
                        for (uint32_t rows = ~v_lives | v_partly; rows != 0; rows &= rows - 1) {
                            const int bit = __ffs(rows) - 1, r = 32 * cw + bit;
                            const bool clear = !((v_lives >> bit) & 1u);
#pragma unroll
                            for (int k = 0; k < L::kAtoms; ++k) {
                                const uint32_t at4 = dst + k * kTile * 128 + r * 128 + lane * 4;
                                uint32_t x4 = 0, keep = 0;
                                if (!clear) {
                                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x4) : "r"(at4) : "memory");
                                    keep = 0xffffffffu;
                                    if constexpr (kQ8) {
#pragma unroll
                                        for (int e = 0; e < 4; ++e)
                                            if (((x4 >> (8 * e)) & 0x7fu) == 0x7fu) keep &= ~(0xffu << (8 * e));
                                    } else {
                                        constexpr uint32_t kExp = kB ? 0x7f80u : 0x7c00u;
                                        if ((x4 & kExp) == kExp) keep &= 0xffff0000u;
                                        if (((x4 >> 16) & kExp) == kExp) keep &= 0xffffu;
                                    }
                                    bad = bad || keep != 0xffffffffu;
                                }
                                if (keep != 0xffffffffu) asm volatile("st.shared.u32 [%0], %1;" ::"r"(at4), "r"(x4 & keep) : "memory");
                            }
                        }
                    }
                    if (bad) ms.desc[v_unit % kUnits].poison = 1;
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&ms.fixed[fixes & 7]);
                    ++fixes;
                }
            }
            if (!more) break;
            v_edge = edge;
            v_partly = partly;
            v_lives = lives;
            v_unit = u - 1;
            ++j;
            ++t;
        }
        copies_wait_all();
    } else if (warp == kMmaWarp) {
        // ---- products: S of tile t, then O of tile t - 1 ----
        const uint32_t lead = elect();
        bool ok = true;
        auto need = [&](unsigned long long* bar, int use) {
            if (ok && !__all_sync(kFull, wait(bar, use, limit))) {
                ok = false;
                *abort = 1;
            }
            return ok;
        };
        constexpr uint32_t kS16 = (1u << 4) | (kB ? (1u << 7) | (1u << 10) : 0u) | (static_cast<uint32_t>(kRowsT >> 3) << 17) | (8u << 24);
        constexpr uint32_t kMn = (1u << 15) | (1u << 16);
        constexpr uint32_t kIS = kQ8 ? (1u << 4) | (1u << 10) | (static_cast<uint32_t>(kRowsT >> 3) << 17) | (8u << 24) : kS16;
        constexpr uint32_t kIO = kQ8 ? (1u << 4) | (1u << 10) | kMn | (16u << 17) | (8u << 24) : kS16 | kMn;
        int t = 0, fixes = 0;
        int pv_unit = 0;
        bool pv_first = false, pv_last = false, pv_edge = false, more = false;
        auto weigh = [&](int tile) {                // O of tile `tile`
            const int ob = pv_unit % L::kOs;
            if (pv_first && !need(&ms.o_free[ob], pv_unit / L::kOs + 1)) return;
            if (!need(&ms.p_full, tile)) return;
            if (pv_edge) {
                if (!need(&ms.fixed[fixes & 7], fixes >> 3)) return;
                ++fixes;
            }
            fence_after();
#pragma unroll
            for (int b = 0; b < L::kBlocks; ++b) {
                const int slot = it % L::kRing;
                if (!need(&ms.full[slot], it / L::kRing)) return;
                fence_after();
                const uint32_t o = tm + L::kTO + (ob * L::kBlocks + b) * L::kOCols;
                const uint32_t v = ring + slot * L::kItem;
                constexpr int kSteps = kQ8 ? 4 : 8;         // of 32 or 16 keys
#pragma unroll
                for (int term = 0; term < L::kPAtoms; ++term)
#pragma unroll
                    for (int ks = 0; ks < kSteps; ++ks)
                        mma_ss<kQ8>(o, desc_mn(v + ks * (16384 / kSteps), kTile * 128), desc_mn(pbuf + term * kTile * 128 + ks * (16384 / kSteps), kTile * 128),
                                    kIO, (pv_first && term == 0 && ks == 0) ? 0u : 1u, lead);
                commit_to(&ms.empty[slot], lead);
                ++it;
            }
            commit_to(&ms.p_free, lead);
            if (pv_last) commit_to(&ms.o_full[ob], lead);
        };
        for (int u = 0; ok; ++u) {
            if (!need(&ms.u_full[u % kUnits], u / kUnits)) break;
            const Desc& d = ms.desc[u % kUnits];
            const int tiles = d.tiles, key0 = d.key0, key1 = d.key1;
            if (tiles == 0) break;
            const int all_lo = p.window > 0 ? max(0, d.past + d.n - p.window) : 0, all_hi = d.past + 1;
            const int qb = u % L::kQs;
            for (int j = 0; j < tiles && ok; ++j, ++t) {
                if (!need(&ms.s_free[t & 1], t / 2 + 1)) break;
                if (j == 0 && !need(&ms.q_full[qb], u / L::kQs)) break;
                const uint32_t s = tm + 64 * (t & 1);
#pragma unroll
                for (int b = 0; b < L::kBlocks; ++b) {
                    const int slot = it % L::kRing;
                    if (!need(&ms.full[slot], it / L::kRing)) break;
                    fence_after();
                    const uint32_t k = ring + slot * L::kItem, q = qbuf + qb * L::kQ + b * L::kAtoms * kRowsT * 128;
                    const int steps = (min(128, D - 128 * b)) * L::kBytes / 32;
#pragma unroll
                    for (int term = 0; term < (kQ8 ? 3 : 1); ++term)
#pragma unroll
                        for (int ks = 0; ks < steps; ++ks)
                            mma_ss<kQ8>(s, desc_sw128(k + (ks >> 2) * kTile * 128 + (ks & 3) * 32),
                                        desc_sw128(q + term * L::kQTerm + (ks >> 2) * kRowsT * 128 + (ks & 3) * 32), kIS,
                                        (b == 0 && term == 0 && ks == 0) ? 0u : 1u, lead);
                    commit_to(&ms.empty[slot], lead);
                    ++it;
                }
                if (!ok) break;
                commit_to(&ms.s_full[t & 1], lead);
                if (!need(&ms.keys_full[t % kKeyRing], t / kKeyRing)) break;
                if (lane == 0) bar_arrive(&ms.s_full[t & 1]);
                if (j == tiles - 1) commit_to(&ms.q_free[qb], lead);
                if (more) weigh(t - 1);
                pv_unit = u;
                pv_first = j == 0;
                pv_last = j == tiles - 1;
                pv_edge = is_edge(key0 + j * kTile, key1, all_lo, all_hi);
                more = true;
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&ms.u_free[u % kUnits]);
        }
        if (more && ok) weigh(t - 1);
        // Products still in flight: after a timeout of any warp's nothing else waits for them (a softmax warp may have
        // given up on the output while this warp's own waits all ended); else the wait is over at once.
        commit_to(&ms.drain, lead);
        if (!__all_sync(kFull, wait(&ms.drain, 0, 0)) && lane == 0) raise(p.status, GDN_FLAG_DRAIN);
    } else if (warp < 4 * parts) {
        // ---- weights and outputs: this thread's key of a tile, chunks of 8 rows ----
        const int quad = warp & 3, part = warp >> 2, key = quad * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        bool fail = false;
        auto need = [&](unsigned long long* bar, int use) {
            if (!fail && !wait(bar, use, limit)) {
                fail = true;
                *abort = 1;
            }
        };
        int t = 0;
        for (int u = 0;; ++u) {
            need(&ms.u_full[u % kUnits], u / kUnits);
            need(&ms.qs_full[u % kUnits], fail ? 0 : (ms.desc[u % kUnits].tiles == 0 ? u / kUnits - 1 : u / kUnits));
            if (soft_any(fail, parts)) break;              // (and the last unit's rows are read)
            const Desc d = ms.desc[u % kUnits];
            if (d.tiles == 0) break;
            if (tid < kRowsT) {
                const int rr = d.tile * kRowsT + tid, tok = min(rr / p.ratio, d.n - 1);
                ms.ref[0][tid] = tid < d.rows ? -kUnset : kUnset;   // (rows that are not there score 0: no weight)
                ms.shift[0][tid] = 0.f;
                ms.last[tid] = d.past + tok;
                ms.first[tid] = p.window > 0 ? max(0, d.past + tok - p.window + 1) : 0;
                if (tid < d.rows) {
                    const int64_t row = token_row(p, d.row0 + tok);
                    const int64_t h = static_cast<int64_t>(d.head * p.ratio + rr - tok * p.ratio) * D;
                    ms.out_at[tid] = row * p.out_stride + h;
                    ms.z_at[tid] = row * p.z_stride + h;
                }
            }
            soft_sync(parts);
            // chunks of 8 rows of this warp, rows 8 (parts i + part) ..: by what the call may have, the same in all units (rows that
            // are not there score 0 and go nowhere)
            const int chunks = tc.chunks;
            const int all_lo = p.window > 0 ? max(0, d.past + d.n - p.window) : 0, all_hi = d.past + 1;
            const float* const qs = ms.q_scale[u % kUnits];
            // (a zero that the compiler does not know: it makes one instruction of a product and a sum on pairs)
            const u64 nothing = *reinterpret_cast<const u64*>(ms.zero);
            u64 l[kMine][4];
#pragma unroll
            for (int i = 0; i < kMine; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) l[i][e] = 0;
            int cur = 0;                            // which of the two ref (and shift) arrays
            bool stop = false;
            for (int j = 0; j < d.tiles; ++j, ++t) {
                need(&ms.s_full[t & 1], t / 2);     // (and what the helpers know of the keys)
                fence_after();
                const uint32_t S = tm + 64 * (t & 1) + lanes;
                const int x0 = d.key0 + j * kTile, x = x0 + key;
                const uint32_t lives = ms.live[t % kKeyRing][quad];
                const bool all = (ms.live[t % kKeyRing][0] & ms.live[t % kKeyRing][1] & ms.live[t % kKeyRing][2] & ms.live[t % kKeyRing][3]) == 0xffffffffu;
                float ks = 1.f, vs = 1.f;
                if constexpr (kQ8) {
                    const float2 f = ms.scales[t % kKeyRing][key];
                    ks = f.x;
                    vs = f.y;
                }
                const bool plain = all && x0 >= all_lo && x0 + kTile <= all_hi;
                const bool live = (lives >> lane) & 1u;
                // scores (in units of log2 e) less the references of `ref`; those that a row does not see are -infinity
                auto unseen = [&](int c) { return !live || x < ms.first[c] || x > ms.last[c]; };
                uint32_t s[kMine][8];
                auto score = [&](uint32_t (&y)[8], int c0, const float* ref, const float* shift) {      // one chunk, in place
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float4 r = *reinterpret_cast<const float4*>(ref + c0 + 4 * h);
                        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                        if constexpr (!kB) f = *reinterpret_cast<const float4*>(qs + c0 + 4 * h);
                        u64 f0 = dup2(p.scale), f1 = f0;
                        if constexpr (!kB) f0 = pk2(f.x, f.y), f1 = pk2(f.z, f.w);
                        if constexpr (kQ8) f0 = fmul2(f0, dup2(ks)), f1 = fmul2(f1, dup2(ks));
                        // (the product rounds before the reference is taken off: that came from such products, and one step
                        // would leave half a last bit of the score between the two, 2^32 for a score of 10^9)
                        u64 a = add2(ffma2(raw2(y[4 * h], y[4 * h + 1]), f0, nothing), pk2(r.x, r.y));
                        u64 b = add2(ffma2(raw2(y[4 * h + 2], y[4 * h + 3]), f1, nothing), pk2(r.z, r.w));
                        if constexpr (kQ8) {
                            const float4 e4 = *reinterpret_cast<const float4*>(shift + c0 + 4 * h);
                            a = add2(a, pk2(e4.x, e4.y));
                            b = add2(b, pk2(e4.z, e4.w));
                        }
                        y[4 * h] = __float_as_uint(lo2(a));
                        y[4 * h + 1] = __float_as_uint(hi2(a));
                        y[4 * h + 2] = __float_as_uint(lo2(b));
                        y[4 * h + 3] = __float_as_uint(hi2(b));
                    }
                    if (!plain) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (unseen(c0 + e)) y[e] = 0xff800000u;
                    }
                };
                const float size = kQ8 ? Product::size_of(vs) : 0.f;
                // 0: scores less the references, and whether one has to move; 1: the scores themselves, for new references;
                // 2: scores less those.  (In a loop, so that the instructions are there once.)
                int mode = j == 0 ? 1 : 0;
                for (;; ++mode) {
                    const float* const ref = mode == 1 ? ms.zero : ms.ref[cur];
                    const float* const shift = mode == 1 ? ms.zero : ms.shift[cur];
#pragma unroll
                    for (int i = 0; i < kMine; ++i)
                        if (i < chunks) tm_ld8(S + 8 * (parts * i + part), s[i]);
                    tm_wait_ld();
#pragma unroll
                    for (int i = 0; i < kMine; ++i)
                        if (i < chunks) score(s[i], 8 * (parts * i + part), ref, shift);
                    if (mode == 0) {
                        float most[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < kMine; ++i)
                            if (i < chunks) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) most[e & 3] = fmaxf(most[e & 3], __uint_as_float(s[i][e]));
                            }
                        const bool grow = fail || fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])) + size > kSlack;
                        if (!soft_any(grow, parts)) break;
                        if (soft_any(fail, parts)) {
                            stop = true;
                            break;
                        }
                    } else if (mode == 1) {
                        // each row's largest score over the tile's keys, and its largest product beside that
                        float v[8 * kMine];
#pragma unroll
                        for (int e = 0; e < 8 * kMine; ++e) v[e] = __uint_as_float(s[e >> 3][e & 7]);
                        const float mx = over_lanes(v, lane, [](float x, float y) { return fmaxf(x, y); });
                        if ((lane >> 3) < chunks) ms.col[quad][8 * (parts * (lane >> 3) + part) + (lane & 7)] = mx;
                        if constexpr (kQ8) {
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < kMine; ++i)
                                if (i < chunks) {
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        v[8 * i + e] = __uint_as_float(s[i][e]) - ms.col[quad][8 * (parts * i + part) + e] + size;
                                }
                            const float top = over_lanes(v, lane, [](float x, float y) { return fmaxf(x, y); });
                            if ((lane >> 3) < chunks) ms.size[quad][8 * (parts * (lane >> 3) + part) + (lane & 7)] = top;
                        }
                        soft_sync(parts);
                        if (tid < kRowsT) {
                            const float m = -ms.ref[cur][tid];
                            float mx = -INFINITY;
                            if (tid < d.rows) mx = fmaxf(fmaxf(ms.col[0][tid], ms.col[1][tid]), fmaxf(ms.col[2][tid], ms.col[3][tid]));
                            if constexpr (kQ8) {
                                float m2 = m, e2 = -ms.shift[cur][tid], top = -INFINITY;
                                const float now = fmaxf(m, mx);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (tid < d.rows && ms.col[k][tid] > -INFINITY) top = fmaxf(top, ms.size[k][tid] + (ms.col[k][tid] - now));
                                ms.alpha[tid] = Product::move(m2, e2, now, top, kLift, kSlack);
                                ms.ref[cur ^ 1][tid] = -m2;
                                ms.shift[cur ^ 1][tid] = -e2;
                            } else {
                                const float now = mx > m + kSlack ? mx - kLift : m;
                                ms.ref[cur ^ 1][tid] = -now;
                                ms.alpha[tid] = now == m ? 1.f : ex2(m - now);
                            }
                        }
                        soft_sync(parts);
                        cur ^= 1;
                    } else {
                        if (j == 0) break;
#pragma unroll
                        for (int i = 0; i < kMine; ++i)
                            if (i < chunks) {
                                const float4* const a = reinterpret_cast<const float4*>(ms.alpha + 8 * (parts * i + part));
                                l[i][0] = fmul2(l[i][0], pk2(a[0].x, a[0].y));
                                l[i][1] = fmul2(l[i][1], pk2(a[0].z, a[0].w));
                                l[i][2] = fmul2(l[i][2], pk2(a[1].x, a[1].y));
                                l[i][3] = fmul2(l[i][3], pk2(a[1].z, a[1].w));
                            }
                        need(&ms.p_free, t - 1);    // the products of the tile before are done
                        fence_after();
                        const int ob = u % L::kOs;
#pragma unroll 1
                        for (int i = 0; i < chunks; ++i) {
                            const int c0 = 8 * (parts * i + part);
#pragma unroll 1
                            for (int k = 0; k < L::kBlocks * (kQ8 ? 2 : 1); ++k) {
                                const uint32_t o = tm + L::kTO + ob * L::kBlocks * L::kOCols + 64 * k + c0 + lanes;
                                uint32_t y[8];
                                tm_ld8(o, y);
                                tm_wait_ld();
#pragma unroll
                                for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * ms.alpha[c0 + e]);
                                tm_st8(o, y);
                            }
                        }
                        tm_wait_st();
                        break;
                    }
                }
                if (stop) break;
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(&ms.s_free[t & 1]);
                    bar_arrive(&ms.keys_free[t % kKeyRing]);
                }
                // weights
                u64 vu = dup2(1.f);
                if constexpr (kQ8) vu = dup2(vs * Product::kUnitInv);
                uint32_t w[kMine][4], w2[kMine][4];
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (i < chunks) {
                        u64 pe[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            pe[e] = pk2(ex2(__uint_as_float(s[i][2 * e])), ex2(__uint_as_float(s[i][2 * e + 1])));
                            l[i][e] = add2(l[i][e], pe[e]);
                            if constexpr (kQ8) pe[e] = fmul2(pe[e], vu);
                        }
                        if constexpr (kQ8) {
                            if (!plain) {                   // (a value that a row does not see may have the scale NaN)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    pe[e] = pk2(unseen(8 * (parts * i + part) + 2 * e) ? 0.f : lo2(pe[e]), unseen(8 * (parts * i + part) + 2 * e + 1) ? 0.f : hi2(pe[e]));
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if constexpr (kB) {
                                w[i][e] = pack_b(lo2(pe[e]), hi2(pe[e]));
                                const u64 rest = ffma2(widen(w[i][e]), dup2(-1.0f), pe[e]);
                                w2[i][e] = pack_b(lo2(rest), hi2(rest));
                            } else {
                                w[i][e] = pack_h(lo2(pe[e]), hi2(pe[e]));
                            }
                        }
                    }
                if (t > 0) need(&ms.p_free, t - 1);
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (i < chunks) {
                        const int c = parts * i + part;     // chunk of 8 rows
                        if constexpr (!kQ8) {
                            const uint32_t a = pbuf + unit16(key, c);
                            st16(a, w[i][0], w[i][1], w[i][2], w[i][3]);
                            if constexpr (kB) st16(a + kTile * 128, w2[i][0], w2[i][1], w2[i][2], w2[i][3]);
                        } else {
#pragma unroll
                            for (int b8 = 0; b8 < 4; ++b8) {        // the four parts in columns 0 | 2, then 1 | 3
                                st8(pbuf + (b8 & 1) * kTile * 128 + unit16(key, 4 * (b8 >> 1) + (c >> 1)) + 8 * (c & 1), upper_bytes(w[i][0], w[i][1]),
                                    upper_bytes(w[i][2], w[i][3]));
                                if (b8 < 3)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) w[i][e] = rest_of(w[i][e]);
                                if (b8 == 1)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) w[i][e] = times_up(w[i][e]);
                                if (b8 == 2)                        // (the last one is rounded: half of its last bit)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) w[i][e] += 0x00800080u;
                            }
                        }
                    }
                fence_async_smem();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&ms.p_full);
            }
            if (stop) break;
            // ---- the unit's output ----
            {
                float v[8 * kMine];
#pragma unroll
                for (int e = 0; e < 8 * kMine; ++e) v[e] = e & 1 ? hi2(l[e >> 3][(e >> 1) & 3]) : lo2(l[e >> 3][(e >> 1) & 3]);
                const float sum = over_lanes(v, lane, [](float x, float y) { return x + y; });
                if ((lane >> 3) < chunks) ms.col[quad][8 * (parts * (lane >> 3) + part) + (lane & 7)] = sum;
            }
            const int ob = u % L::kOs;
            need(&ms.o_full[ob], u / L::kOs);
            if (soft_any(fail, parts)) break;
            fence_after();
            if (tid < kRowsT) {
                const float sum = ms.col[0][tid] + ms.col[1][tid] + ms.col[2][tid] + ms.col[3][tid];
                ms.inv[tid] = sum == 0.f ? 0.f : (kQ8 ? Product::kUnit : 1.f) / sum;
                if (d.part >= 0) {
                    float m = -ms.ref[cur][tid], e = -ms.shift[cur][tid];
                    if constexpr (kQ8) Product::settle(m, e, sum);
                    ms.inv[tid] = kQ8 ? Product::of_o(e) : 1.f;
                    if (tid < d.rows) {
                        float* ml = p.ws + static_cast<int64_t>(2 * gridDim.x) * kRowsT * D + static_cast<int64_t>(d.part) * 2 * kRowsT;
                        ml[tid] = m;
                        ml[kRowsT + tid] = kQ8 ? sum * Product::of_l(e) : sum;
                    }
                }
            }
            soft_sync(parts);
            const bool poison = *const_cast<volatile int*>(&ms.desc[u % kUnits].poison) != 0;
#pragma unroll 1
            for (int k = 0; k < L::kBlocks * chunks; ++k) {
                const int i = k / L::kBlocks, b2 = k - i * L::kBlocks;
                const int dcol = 128 * b2 + key, c0 = 8 * (parts * i + part);
                const uint32_t o = tm + L::kTO + (ob * L::kBlocks + b2) * L::kOCols + c0 + lanes;
                float y[8];
                uint32_t y1[8], y2[8];
                tm_ld8(o, y1);
                if constexpr (kQ8) tm_ld8(o + 64, y2);
                tm_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = kQ8 ? fmaf(__uint_as_float(y2[e]), 1.f / kUp, __uint_as_float(y1[e])) : __uint_as_float(y1[e]);
                    y[e] *= ms.inv[c0 + e];
                }
                if (dcol >= D) continue;
                if (poison) add_no_numbers<kKind>(p, d, ms.first + c0, ms.last + c0, all_lo, all_hi, dcol, y);
                if (d.part >= 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c0 + e < d.rows) p.ws[(static_cast<int64_t>(d.part) * kRowsT + c0 + e) * D + dcol] = y[e];
                } else {
                    if (p.z) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (c0 + e < d.rows) y[e] = gated(y[e], __bfloat162float(ld(p.z + ms.z_at[c0 + e] + dcol)));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c0 + e < d.rows) p.out[ms.out_at[c0 + e] + dcol] = __float2bfloat16_rn(y[e]);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) {
                bar_arrive(&ms.o_free[ob]);
                bar_arrive(&ms.u_free[u % kUnits]);
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (*abort != 0) {
        if (tid == 0) raise(p.status, GDN_FLAG_TIMEOUT);
        if (warp == kLoadWarp) {                    // loads still on their way end before this shared memory is another's
            bool landed = true;
            for (int k = max(0, it - L::kRing); k < it; ++k) landed = wait(&ms.full[k % L::kRing], k / L::kRing, 0) && landed;
            for (int k = max(0, edges - 8); k < edges; ++k) landed = wait(&ms.edge_full[k & 7], k >> 3, 0) && landed;
            if (!landed && lane == 0) raise(p.status, GDN_FLAG_DRAIN);
        }
    }
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(512));
}

// A cache as [pages][heads][positions of a page][D], read in boxes of 128 bytes by `box` positions.
inline bool encode_map(CUtensorMap& map, const void* base, const AttnParams& p, int D, int kind, int box) {
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
    const int bytes = kind == kE4m3 ? 1 : 2;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.pg.page), static_cast<cuuint64_t>(p.heads),
                                static_cast<cuuint64_t>(p.pg.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(p.pg.token_stride) * bytes, static_cast<cuuint64_t>(p.pg.head_stride) * bytes,
                                   static_cast<cuuint64_t>(p.pg.page_stride) * bytes};
    const cuuint32_t boxes[4] = {128u / bytes, static_cast<cuuint32_t>(box), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = kind == kE4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : kind == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode(&map, type, 4, const_cast<void*>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kKind, int D>
cudaError_t launch(const AttnParams& p, bool joins, int grid, cudaStream_t stream) {
    auto kernel = gdn_attn_tc_kernel<kKind, D>;
    static bool ready_on[64] = {false};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 64 || !__atomic_load_n(&ready_on[dev], __ATOMIC_ACQUIRE)) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of<kKind, D>());
        if (err != cudaSuccess) return err;
        if (dev < 64) __atomic_store_n(&ready_on[dev], true, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(Warps<kKind>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_of<kKind, D>();
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static_assert(smem_of<kKind, D>() <= 227 * 1024, "shared memory");
    TcParams tc;
    tc.limit = __atomic_load_n(&gdn_internal::g_wait_limit, __ATOMIC_RELAXED);
    const int rows = p.ratio * p.max_T < kRowsT ? p.ratio * p.max_T : kRowsT;
    constexpr int kMost = Warps<kKind>::kSoft / 4;
    tc.parts = (rows + 7) / 8 < kMost ? (rows + 7) / 8 : kMost;
    tc.chunks = ((rows + 7) / 8 + tc.parts - 1) / tc.parts;
    // positions of a box: a power of two that divides a page, and 16 at most where a window may begin a unit at any multiple of 16
    tc.box_log2 = 3;
    while (tc.box_log2 < (p.window > 0 ? 4 : 7) && p.pg.page % (2 << tc.box_log2) == 0) ++tc.box_log2;
    tc.box = 1 << tc.box_log2;
    CUtensorMap k_map, v_map;
    if (!encode_map(k_map, p.k, p, D, kKind, tc.box) || !encode_map(v_map, p.v, p, D, kKind, tc.box)) return cudaErrorInvalidValue;
    err = cudaLaunchKernelEx(&cfg, kernel, p, k_map, v_map, tc);
    if (err != cudaSuccess || !joins) return err;
    cfg.gridDim = dim3(static_cast<unsigned>(grid * kJSplit<kRowsT>), 1, 1);
    cfg.blockDim = dim3(kJThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, gdn_attn_join_kernel<D, kRowsT>, p, grid);
}

inline int grid_of() {
    const int sms = sm_count() ? sm_count() : 148;
    return sms < kMaxCtas ? sms : kMaxCtas;
}

// the launch for one type of cache (a translation unit each)
template <int kKind>
cudaError_t launch_kind(AttnParams p, int D, void* workspace, cudaStream_t s) {
    const int grid = grid_of();
    p.meta = static_cast<int32_t*>(workspace);
    p.ws = reinterpret_cast<float*>(p.meta + static_cast<int64_t>(grid) * kMetaInts);
    p.stand_side_by_side();
    // a unit of one block has nothing to join
    const bool joins = static_cast<int64_t>(p.pg.cols) * p.pg.page + kKeys > kTile;
    return D == 64    ? launch<kKind, 64>(p, joins, grid, s)
           : D == 128 ? launch<kKind, 128>(p, joins, grid, s)
           : D == 192 ? launch<kKind, 192>(p, joins, grid, s)
                      : launch<kKind, 256>(p, joins, grid, s);
}

inline int64_t workspace_of(int D) {
    const int64_t grid = grid_of();
    return grid * kMetaInts * 4 + 2 * grid * kRowsT * (D + 2) * 4;
}

}  // namespace gdn_attn_tc
