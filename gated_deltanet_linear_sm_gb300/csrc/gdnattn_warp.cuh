// Internal to libgdnspec: the attention of a step's tokens over the paged key-value cache for few query
// rows, with every warp on keys of its own (gdnattn_*.cu instantiate it; gdnattn.cu has the mathematics
// and the choice of kernel).
//
// A unit is one (sequence, cache head, tile of 8 kOct query rows: heads of the group times tokens).  A
// warp takes 16 keys at a time, from a ring of asynchronous copies that no other warp touches (K and V
// of 16 keys are an item each), and runs
//     S^T[16 keys][8 rows] = K Q^T,        O^T[D][8 rows] += V^T P^T
// on the tensor cores (m16n8k16): the keys and the head dim are the 16 rows, so 8 query rows cost no more
// than they are (with the query rows as the 16 rows, 4 of them took twice the products, the accumulators
// and the registers: 32 sequences of up to 4096 66 us, 4 of 131072 in e4m3 303).  The weights come out
// transposed for the second product; movmatrix turns them.
//
// What bounds it: with 8 rows or fewer the bytes (32 of up to 4096, head dim 128, bf16 64 us, 5.4 TB/s; 4 of
// 131072, e4m3 185 us, 6.0 TB/s); with more rows the instructions of the widening and the softmax in the 8
// warps of an SM that the accumulators leave room for (64 x 3 tokens x window 1024, 18 rows, int8 38.5 us: 1000 instructions for
// 16 keys with a unit's start and end, 0.45 a cycle and scheduler); with short sequences a unit's chain of start and end, about 2.5 us.
//
// A row's reference m is kUnset until it has a score; it moves when a score passes it by more than
// 2^kSlack, and only then do the lanes compare: a block's vote is one instruction.  kLift keeps weights
// far from the end of fp16's range (bf16: gdnattn.cuh).
//
// fp16 and 8-bit caches run on fp16 operands: codes are exact in fp16, a key's scale multiplies its score
// and a value's scale its weight.  What has to fit fp16 is then weight times scale, so an 8-bit row has its
// reference in two parts: m, its largest score when it moved, and e (gdnattn.cuh: Product), from the largest product
// of a weight and a scale among the keys that the row itself sees.  A scale that other rows see, or that has
// no weight, takes no bits from a row's other products.  q becomes fp16 by a power of two of its
// row, which goes into the row's scale.  A bf16 cache runs on bf16 operands, and a weight is the sum of two
// bf16 parts: one has 8 bits only.
#pragma once

#include "gdnattn.cuh"

namespace gdn_attn_warp {

using namespace gdn_attn;

enum Kind { kBf16, kF16, kE4m3, kI8 };

constexpr float kLiftH = 6.f, kSlackH = 14.f;

// ---- instructions -----------------------------------------------------------------------------

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t turn(uint32_t x) {      // an 8 x 8 matrix of 16-bit elements, transposed
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// C[16][8] += A[16][16] B[16][8]; bf16 or fp16 operands
template <bool kBf>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// four 8-bit codes as fp16 pairs: bytes 0 and 1, bytes 2 and 3 (exact for either type)
template <int kKind>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& ab, uint32_t& cd) {
    if constexpr (kKind == kE4m3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(ab), "=r"(cd) : "r"(w));
    } else {
        // 0x6400 + u is 1024 + u in fp16; u = code + 128
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 c = __floats2half2_rn(1152.f, 1152.f);
        const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&x), c), b = __hsub2(*reinterpret_cast<const __half2*>(&y), c);
        ab = *reinterpret_cast<const uint32_t*>(&a);
        cd = *reinterpret_cast<const uint32_t*>(&b);
    }
}
__device__ __forceinline__ float lds(uint32_t a) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
    return x;
}

// ---- shapes -------------------------------------------------------------------------------------

constexpr int kCutKeys = 64, kWarps = 4, kThreads = kWarps * 32;
template <int kOct, int kRow>
struct Cut {                            // (gdnattn.cuh)
    static constexpr int kThreads = gdn_attn_warp::kThreads;
    static constexpr int kPer = 2;
    static constexpr int kBlock = kCutKeys;
    static constexpr int kRows = 8 * kOct;
    static constexpr int kCost = 384 / kRow > 1 ? 384 / kRow : 1;   // (about 10000 cycles: 3 blocks of 16 KB, 1 of 64 KB)
};

template <int kKind, int D, int kOct>
struct Shape {
    static constexpr int kBytes = kKind <= kF16 ? 2 : 1;
    static constexpr int kRow = D * kBytes;                     // bytes of a key
    static constexpr int kItem = kKeys * kRow + (kBytes == 1 ? 4 * kKeys : 0);      // K or V of 16 keys, with their scales
    // CTAs of an SM: short rows (64 x 16 bits, 128 x 8) leave room for three with long rings, whose units' starts and
    // ends overlap (256 sequences of up to 500, head dim 64: 59 us with two or four, 49 with three, 45 as it is now); with more bytes a
    // row two long rings do better than four short ones (32 of up to 4096, head dim 128, bf16: 64 us, 69 with three, 78 with four)
    static constexpr int kCtas = kRow <= 128 && kOct == 1 ? 3 : 2;
    static constexpr int kQ = 8 * kOct * D * 2;
    static constexpr int kStatic = 8 * 1024;                    // (the line and what the warps exchange)
    static constexpr int kRing0 = (227 * 1024 / kCtas - 1024 - kStatic - kQ) / (kWarps * kItem);
    static constexpr int kRing = kRing0 > 8 ? 8 : kRing0;       // items of a warp, on their way or in use
    static constexpr int kRingBytes = kWarps * kRing * kItem;
    static constexpr int kJoinBytes = kWarps * 8 * kOct * D * 4;    // the warps' O, in the ring's place
    static constexpr int kSmem = kQ + (kRingBytes > kJoinBytes ? kRingBytes : kJoinBytes);
    static constexpr bool kHoldQ = kOct * D <= 256;             // q's fragments in registers
    static_assert(kRing >= 3, "a ring of K, V and one more");
    static_assert(kCtas * (kSmem + kStatic + 1024) <= 228 * 1024, "shared memory");
};

// byte of 16-byte chunk c of key r in an item: the chunks of a row in an order that depends on the
// row, so that neither ldmatrix (8 rows, one chunk) nor an 8-bit K fragment's load (2 rows, 4 chunks)
// meets a bank twice
template <int kKind, int D, bool kIsK>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    constexpr int kRow = D * (kKind <= kF16 ? 2 : 1);
    if constexpr (kKind <= kF16) return r * kRow + 16 * (c ^ (r & 7));
    else if constexpr (kRow % 128 != 0) return r * kRow + 16 * (kIsK ? c : c ^ ((r >> 1) & 3));
    else return r * kRow + 16 * (kIsK ? c ^ ((r & 1) << 2) : c ^ (r & 7));
}

// An infinity or NaN among values that some rows see and some do not: its products would reach the
// others as 0 * NaN.  It is added to the rows that see it (whatever its weight: the sum is no number
// then) and taken out of the tile.  (16-bit caches; in the others it is a scale, which stays with its weight.)
template <int kKind, int D, int kOct>
__device__ __noinline__ void take_out(float* o, uint32_t vs0, int x0, const int* first, const int* last, uint32_t live, int lane) {
    constexpr uint32_t kExp = kKind == kBf16 ? 0x7f80u : 0x7c00u;
    const int g = lane >> 2, tq = lane & 3;
    for (int dn = 0; dn < D / 16; ++dn)
        for (int h = 0; h < 2; ++h)
            for (int kk = 0; kk < kKeys; ++kk) {
                uint32_t raw;
                const int d = 16 * dn + 8 * h + g;
                const uint32_t at = vs0 + chunk_at<kKind, D, false>(kk, d / 8) + 2 * (d % 8 & ~1);
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(raw) : "r"(at) : "memory");
                const uint32_t x = (raw >> (16 * (d & 1))) & 0xffffu;
                if ((x & kExp) != kExp || !((live >> kk) & 1u)) continue;
                const __half_raw hr = {static_cast<unsigned short>(x)};
                const float v = kKind == kBf16 ? __uint_as_float(x << 16) : __half2float(__half(hr));
                for (int n = 0; n < kOct; ++n)
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * n + 2 * tq + e;
                        if (x0 + kk >= first[row] && x0 + kk <= last[row]) o[(dn * kOct + n) * 4 + 2 * h + e] += v;
                    }
            }
    __syncwarp();
    for (int id = lane; id < kKeys * D / 2; id += 32) {
        const uint32_t at = vs0 + 4 * id;
        uint32_t raw;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(raw) : "r"(at) : "memory");
        if ((raw & kExp) == kExp) raw &= 0xffff0000u;
        if (((raw >> 16) & kExp) == kExp) raw &= 0xffffu;
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(raw) : "memory");
    }
    __syncwarp();
}

template <int kKind, int D, int kOct>
__global__ void __launch_bounds__(kThreads, Shape<kKind, D, kOct>::kCtas) gdn_attn_decode_kernel(const AttnParams p) {
    using S = Shape<kKind, D, kOct>;
    using G = Cut<kOct, S::kRow>;
    constexpr int kRowsU = 8 * kOct;
    constexpr bool kQuantised = S::kBytes == 1;
    constexpr bool kB = kKind == kBf16;
    constexpr float kLift = kB ? kLiftBf : kLiftH, kSlack = kB ? kSlackBf : kSlackH;
    constexpr int kSteps = D / 16;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Line<G> line;
    __shared__ float row_m[kWarps][kRowsU], row_l[kWarps][kRowsU];
    __shared__ float q_scale[kRowsU], row_inv[kRowsU];
    __shared__ int row_first[kRowsU], row_last[kRowsU];
    __shared__ int64_t row_out[kRowsU], row_z[kRowsU];
    __shared__ uint32_t live_keys[kWarps][S::kRing];
    unsigned char* const sq = smem;
    unsigned char* const ring0 = smem + S::kQ;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    dep_wait();
    const int64_t total = begin_line<G>(p, line);
    dep_launch();
    const int ctas = ctas_of(total, gridDim.x / p.side, 1 + G::kCost);
    const int cta = blockIdx.x, place = cta / p.side, member = cta - place * p.side;
    int32_t* const meta = p.meta + static_cast<int64_t>(cta) * kMetaInts;
    if (tid == 0) meta[0] = meta[8] = -1;           // (no part yet)
    if (place >= ctas) return;
    const int64_t w0 = quotient(total * place, ctas), w1 = quotient(total * (place + 1), ctas);
    const uint32_t my_ring = saddr(ring0) + warp * S::kRing * S::kItem;
    const bool aligned_pages = p.pg.page % kKeys == 0;          // 16 keys lie in one page

    for (int64_t w = w0; w < w1;) {
        const int k = sequence_at<G>(p, line, w);
        const Piece d = piece_at<G>(p, line, k, w, w1, member);
        w += d.places;
        if (d.b0 == d.b1) continue;
        const bool whole = d.b0 == 0 && d.b1 == d.blocks;
        const int part = whole ? -1 : d.b0 > 0 ? 2 * cta : 2 * cta + 1;
        const int items = 2 * max(0, ((d.key1 - d.key0 + kKeys - 1) / kKeys - warp + kWarps - 1) / kWarps);

        // ---- the ring ----
        const char* const kc = static_cast<const char*>(p.k) + d.head * p.pg.head_stride * S::kBytes;
        const char* const vc = static_cast<const char*>(p.v) + d.head * p.pg.head_stride * S::kBytes;
        const int32_t* const table = p.pg.table + static_cast<int64_t>(d.seq) * p.pg.table_stride;
        // Pages: where 16 keys lie in one, lane l knows that of this warp's block l of the present 32 (and of the next
        // 32), so that a lookup's latency shows once a unit; else each lane that of its key of the next block.
        const int my_key = lane & 15;
        auto page_at = [&](int x) { return x < d.key1 ? ld(table + p.pg.page_of(x)) : -1; };
        auto block_at = [&](int block) { return d.key0 + (warp + block * kWarps) * kKeys; };
        int pages = aligned_pages ? page_at(block_at(lane)) : page_at(block_at(0) + my_key);
        int pages_next = aligned_pages && items > 64 ? page_at(block_at(32 + lane)) : -1;
        int64_t at = 0;                             // bytes: this lane's key, or the first of the 16
        int64_t sat = 0;
        uint32_t live = 0;
        int issued = 0;
        auto issue = [&]() {
            if (issued < items) {
                const int slot = issued % S::kRing;
                const uint32_t dst = my_ring + slot * S::kItem;
                const bool is_k = (issued & 1) == 0;
                if (is_k) {
                    const int block = issued >> 1, x0 = block_at(block), x = aligned_pages ? x0 : x0 + my_key;
                    if (aligned_pages && block > 0 && (block & 31) == 0) {
                        pages = pages_next;
                        pages_next = page_at(block_at(block + 32 + lane));
                    }
                    const int page = aligned_pages ? __shfl_sync(kFull, pages, block & 31) : pages;
                    const bool has = page >= 0 && page < p.pg.num_pages;
                    if (page >= p.pg.num_pages) raise(p.status, GDN_FLAG_SLOT_RANGE);
                    const int64_t in = x - p.pg.page_of(x) * p.pg.page;
                    at = has ? (page * p.pg.page_stride + in * p.pg.token_stride) * S::kBytes : 0;
                    if constexpr (kQuantised) sat = has ? page * p.pg.s_page + in * p.pg.s_token + d.head * p.pg.s_head : 0;
                    if (aligned_pages) {
                        const int n = has ? min(kKeys, d.key1 - x0) : 0;
                        live = (1u << n) - 1;
                    } else {
                        live = __ballot_sync(kFull, has) & 0xffffu;
                    }
                    if (lane == 0) live_keys[warp][slot] = live;
                    if (!aligned_pages) pages = page_at(block_at(block + 1) + my_key);
                }
                const char* const src = (is_k ? kc : vc);
                constexpr int kChunks = S::kRow / 16;               // of a key
                if (aligned_pages) {
                    const char* const from = src + at;
                    const int64_t step = p.pg.token_stride * S::kBytes;
#pragma unroll
                    for (int it = 0; it < kChunks / 2; ++it) {
                        const int id = it * 32 + lane;
                        const int r = id / kChunks, c = id - r * kChunks;
                        copy16(dst + (is_k ? chunk_at<kKind, D, true>(r, c) : chunk_at<kKind, D, false>(r, c)), from + r * step + 16 * c, (live >> r) & 1u);
                    }
                } else {
#pragma unroll 2
                    for (int it = 0; it < kChunks / 2; ++it) {
                        const int id = it * 32 + lane;
                        const int r = id / kChunks, c = id - r * kChunks;
                        const int64_t from = __shfl_sync(kFull, at, r);
                        copy16(dst + (is_k ? chunk_at<kKind, D, true>(r, c) : chunk_at<kKind, D, false>(r, c)), src + from + 16 * c, (live >> r) & 1u);
                    }
                }
                if constexpr (kQuantised) {
                    if (lane < kKeys)
                        copy4(dst + kKeys * S::kRow + 4 * lane, (is_k ? p.k_scale : p.v_scale) + sat + (aligned_pages ? lane * p.pg.s_token : 0), (live >> lane) & 1u);
                }
            }
            copies_commit();
            ++issued;
        };

        // ---- q: [rows][D] in shared memory, fp16 with a power of two per row, or bf16 as it is; the rows' places ----
        {
            constexpr int kPer = kThreads / (kRowsU > 16 ? 32 : kRowsU);        // threads of a row
            constexpr int kN = (D / 8 + kPer - 1) / kPer;           // 16-byte pieces of each
            const int r = tid / kPer, j = tid % kPer;
            const bool in = r < kRowsU;
            const int rr = d.tile * kRowsU + r, t = min(rr / p.ratio, d.n - 1);
            const bool has = r < d.rows;
            const int64_t row = token_row(p, d.row0 + t);
            const int64_t hq = static_cast<int64_t>(d.head * p.ratio + rr - t * p.ratio) * D;
            const __nv_bfloat16* src = has ? p.q + row * p.q_stride + hq : p.q;
            uint4 raw[kN];
            uint32_t big = 0;
#pragma unroll
            for (int u = 0; u < kN; ++u) {
                const int c = j + u * kPer;
                raw[u] = make_uint4(0, 0, 0, 0);
                if (has && c < D / 8) raw[u] = ld(reinterpret_cast<const uint4*>(src) + c);
            }
            // (q is on its way while the first keys are asked for)
#pragma unroll 1
            for (int u = 0; u < S::kRing - 1; ++u) issue();
#pragma unroll
            for (int u = 0; u < kN; ++u) {
                const uint32_t x[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) big = max(big, max(x[e] & 0x7fffu, (x[e] >> 16) & 0x7fffu));
            }
            float down = 1.f, up = 1.f;
            if constexpr (!kB) {
#pragma unroll
                for (int o = kPer / 2; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(kFull, big, o, kPer));
                // exponent: the row's largest becomes 2^14 to 2^15, so that elements down to 2^-31 of it are exact
                constexpr int kTop = 14;
                const int e = max(static_cast<int>(big >> 7), 1 + kTop);
                if ((big >> 7) != 255) {                                        // (an infinity or NaN stays what it is)
                    down = __uint_as_float(static_cast<uint32_t>(254 + kTop - e) << 23);
                    up = __uint_as_float(static_cast<uint32_t>(e - kTop) << 23);
                }
            }
            if (j == 0 && in) {
                q_scale[r] = p.scale * up;
                row_last[r] = d.past + t;
                row_first[r] = p.window > 0 ? max(0, d.past + t - p.window + 1) : 0;
                row_out[r] = row * p.out_stride + hq;
                row_z[r] = row * p.z_stride + hq;
            }
#pragma unroll
            for (int u = 0; u < kN; ++u) {
                const int c = j + u * kPer;
                if (c < D / 8 && in) {
                    uint4 y = raw[u];
                    if constexpr (!kB) {
                        uint32_t* w2 = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w2[e] = pack_h(__uint_as_float(w2[e] << 16) * down, __uint_as_float(w2[e] & 0xffff0000u) * down);
                    }
                    *reinterpret_cast<uint4*>(sq + r * D * 2 + 16 * (c ^ (r & 7))) = y;
                }
            }
        }
        __syncthreads();
        // q as right operand: k is the head dim, n the row.  8-bit caches have their elements in the order of a K
        // fragment, 16 neighbouring ones per lane of a quad.
        auto q_frag = [&](int n, int ks, uint32_t& b0, uint32_t& b1) {
            if constexpr (!kQuantised) {
                const uint2 x = make_uint2(*reinterpret_cast<const uint32_t*>(sq + (8 * n + g) * D * 2 + 16 * ((2 * ks) ^ g) + 4 * tq),
                                           *reinterpret_cast<const uint32_t*>(sq + (8 * n + g) * D * 2 + 16 * ((2 * ks + 1) ^ g) + 4 * tq));
                b0 = x.x;
                b1 = x.y;
            } else {
                const int e = (ks >> 2) * 64 + tq * 16 + 4 * (ks & 3);
                const uint2 x = *reinterpret_cast<const uint2*>(sq + (8 * n + g) * D * 2 + 16 * ((e / 8) ^ g) + (e % 8) * 2);
                b0 = x.x;
                b1 = x.y;
            }
        };
        uint32_t qf[S::kHoldQ ? kOct : 1][S::kHoldQ ? kSteps : 1][2];
        if constexpr (S::kHoldQ) {
#pragma unroll
            for (int n = 0; n < kOct; ++n)
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks) q_frag(n, ks, qf[n][ks][0], qf[n][ks][1]);
        }
        // this thread's rows 8 n + 2 tq and the next: their scale, reference (pe: e of the products) and sum
        float qs[kOct][2], m[kOct][2], pe[kOct][2], l[kOct][2];
#pragma unroll
        for (int n = 0; n < kOct; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qs[n][e] = q_scale[8 * n + 2 * tq + e];
                m[n][e] = 8 * n + 2 * tq + e < d.rows ? kUnset : -kUnset;   // (rows that are not there score 0: no weight)
                pe[n][e] = l[n][e] = 0.f;
            }
        const int all_lo = p.window > 0 ? max(0, d.past + d.n - p.window) : 0, all_hi = d.past + 1;     // seen by every row
        float o[D / 16][kOct][4];
#pragma unroll
        for (int dn = 0; dn < D / 16; ++dn)
#pragma unroll
            for (int n = 0; n < kOct; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[dn][n][e] = 0.f;

        // ---- the keys ----
#pragma unroll 1
        for (int i = 0; i < items; i += 2) {
            copies_wait<S::kRing - 2>();
            __syncwarp();
            issue();
            const uint32_t ks0 = my_ring + (i % S::kRing) * S::kItem;
            const uint32_t vs0 = my_ring + ((i + 1) % S::kRing) * S::kItem;
            float s[kOct][4];                       // keys g and g + 8, rows 2 tq and 2 tq + 1: key of e is e >> 1, row e & 1
            {
                float c0[kOct][4], c1[kOct][4];     // (two chains of products)
#pragma unroll
                for (int n = 0; n < kOct; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c0[n][e] = c1[n][e] = 0.f;
                auto product = [&](int ks, const uint32_t (&a)[4]) {
#pragma unroll
                    for (int n = 0; n < kOct; ++n) {
                        uint32_t b0, b1;
                        if constexpr (S::kHoldQ) b0 = qf[n][ks][0], b1 = qf[n][ks][1];
                        else q_frag(n, ks, b0, b1);
                        mma<kB>(ks & 1 ? c1[n] : c0[n], a, b0, b1);
                    }
                };
                if constexpr (!kQuantised) {
#pragma unroll
                    for (int ks = 0; ks < kSteps; ++ks) {
                        uint32_t a[4];
                        ldsm4(a, ks0 + chunk_at<kKind, D, true>(lane & 15, 2 * ks + (lane >> 4)));
                        product(ks, a);
                    }
                } else {
#pragma unroll
                    for (int seg = 0; seg < D / 64; ++seg) {
                        uint32_t x[2][4];           // 16 codes of keys g and g + 8
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(x[h][0]), "=r"(x[h][1]), "=r"(x[h][2]), "=r"(x[h][3])
                                         : "r"(ks0 + chunk_at<kKind, D, true>(8 * h + g, 4 * seg + tq)) : "memory");
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            uint32_t a[4];
                            widen4<kKind>(x[0][ks], a[0], a[2]);
                            widen4<kKind>(x[1][ks], a[1], a[3]);
                            product(4 * seg + ks, a);
                        }
                    }
                }
                float f[2] = {1.f, 1.f};
                if constexpr (kQuantised) f[0] = lds(ks0 + kKeys * S::kRow + 4 * g), f[1] = lds(ks0 + kKeys * S::kRow + 4 * g + 32);
#pragma unroll
                for (int n = 0; n < kOct; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // (rounded before the reference is taken off, which comes from such scores)
                        const float x = __fmul_rn(c0[n][e] + c1[n][e], qs[n][e & 1]);
                        s[n][e] = kQuantised ? __fmul_rn(x, f[e >> 1]) : x;
                    }
            }
            const int x0 = d.key0 + (warp + (i >> 1) * kWarps) * kKeys;
            const uint32_t there = live_keys[warp][i % S::kRing];
            const bool partly = x0 < all_lo || x0 + kKeys > all_hi;
            const bool plain = !partly && there == 0xffffu;
            if (!plain) {
#pragma unroll
                for (int n = 0; n < kOct; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int kk = g + 8 * (e >> 1), x = x0 + kk, row = 8 * n + 2 * tq + (e & 1);
                        if (x < row_first[row] || x > row_last[row] || !((there >> kk) & 1u)) s[n][e] = -INFINITY;
                    }
            }
            copies_wait<S::kRing - 2>();            // (V: its scales are wanted now)
            __syncwarp();
            issue();
            // ---- the softmax's references and weights ----
            float f[2] = {1.f, 1.f}, size[2] = {0.f, 0.f};
            if constexpr (kQuantised) {
                f[0] = lds(vs0 + kKeys * S::kRow + 4 * g);
                f[1] = lds(vs0 + kKeys * S::kRow + 4 * g + 32);
                size[0] = Product::size_of(f[0]);
                size[1] = Product::size_of(f[1]);
            }
            float y[kOct][4];                       // scores less their references
            auto less = [&]() {
#pragma unroll
                for (int n = 0; n < kOct; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[n][e] = s[n][e] - m[n][e & 1];
                        if constexpr (kQuantised) y[n][e] -= pe[n][e & 1];
                    }
            };
            less();
            bool grow = false;
#pragma unroll
            for (int n = 0; n < kOct; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    grow = grow || (kQuantised ? fmaxf(y[n][e] + size[0], y[n][e + 2] + size[1]) : fmaxf(y[n][e], y[n][e + 2])) > kSlack;
            if (__any_sync(kFull, grow)) {
#pragma unroll
                for (int n = 0; n < kOct; ++n) {
                    float a[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(s[n][e], s[n][e + 2]);
#pragma unroll
                        for (int q = 4; q < 32; q <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, q));
                        if constexpr (kQuantised) {
                            const float now = fmaxf(m[n][e], mx);
                            float top = fmaxf(s[n][e] - now + size[0], s[n][e + 2] - now + size[1]);
#pragma unroll
                            for (int q = 4; q < 32; q <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, q));
                            a[e] = Product::move(m[n][e], pe[n][e], now, top, kLift, kSlack);
                        } else {
                            const float now = mx > m[n][e] + kSlack ? mx - kLift : m[n][e];
                            a[e] = m[n][e] == now ? 1.f : ex2(m[n][e] - now);
                            m[n][e] = now;
                        }
                        l[n][e] *= a[e];
                    }
#pragma unroll
                    for (int dn = 0; dn < D / 16; ++dn)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[dn][n][e] *= a[e & 1];
                }
                less();
            }
            if constexpr (kQuantised) {
                f[0] *= Product::kUnitInv;
                f[1] *= Product::kUnitInv;
            }
            uint32_t pf[kOct][2], pl[kOct][2];      // right operand: k is the key, n the row
#pragma unroll
            for (int n = 0; n < kOct; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float w2[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        w2[e] = ex2(y[n][2 * h + e]);
                        l[n][e] += w2[e];
                        if constexpr (kQuantised) {                 // (a value that a row does not see may have the scale NaN)
                            w2[e] *= f[h];
                            if (!plain) w2[e] = s[n][2 * h + e] == -INFINITY ? 0.f : w2[e];
                        }
                    }
                    if constexpr (kB) {
                        const uint32_t hi = pack_b(w2[0], w2[1]);
                        pf[n][h] = turn(hi);
                        pl[n][h] = turn(pack_b(w2[0] - __uint_as_float(hi << 16), w2[1] - __uint_as_float(hi & 0xffff0000u)));
                    } else {
                        pf[n][h] = turn(pack_h(w2[0], w2[1]));
                    }
                }
            if constexpr (!kQuantised) {
                if (partly) {
                    constexpr uint32_t kExp = kB ? 0x7f80u : 0x7c00u;
                    bool bad = false;
#pragma unroll 1
                    for (int id = lane; id < kKeys * D / 2; id += 32) {
                        uint32_t raw;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(raw) : "r"(vs0 + 4 * id) : "memory");
                        bad = bad || (raw & kExp) == kExp || ((raw >> 16) & kExp) == kExp;
                    }
                    if (__any_sync(kFull, bad)) {
                        float copy[D / 16 * kOct * 4];
#pragma unroll
                        for (int dn = 0; dn < D / 16; ++dn)
#pragma unroll
                            for (int e = 0; e < 4 * kOct; ++e) copy[dn * kOct * 4 + e] = o[dn][e >> 2][e & 3];
                        take_out<kKind, D, kOct>(copy, vs0, x0, row_first, row_last, there, lane);
#pragma unroll
                        for (int dn = 0; dn < D / 16; ++dn)
#pragma unroll
                            for (int e = 0; e < 4 * kOct; ++e) o[dn][e >> 2][e & 3] = copy[dn * kOct * 4 + e];
                    }
                }
            }
            // ---- O^T += V^T P^T ----
            if constexpr (!kQuantised) {
                const int r = (lane & 7) + ((lane >> 4) << 3), c = (lane >> 3) & 1;
#pragma unroll
                for (int dn = 0; dn < D / 16; ++dn) {
                    uint32_t a[4];
                    ldsm4t(a, vs0 + chunk_at<kKind, D, false>(r, 2 * dn + c));
#pragma unroll
                    for (int n = 0; n < kOct; ++n) {
                        mma<kB>(o[dn][n], a, pf[n][0], pf[n][1]);
                        if constexpr (kB) mma<kB>(o[dn][n], a, pl[n][0], pl[n][1]);
                    }
                }
            } else {
                // 16 columns are a tile, the even ones its rows 0 to 7 and the odd ones 8 to 15: neighbouring columns of
                // two keys come in one register
                const int r = lane & 15, c = lane >> 4;
#pragma unroll
                for (int dd = 0; dd < D / 32; ++dd) {
                    uint32_t b[4];
                    ldsm4t(b, vs0 + chunk_at<kKind, D, false>(r, 2 * dd + c));
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        uint32_t a[4];
                        widen4<kKind>(__byte_perm(b[2 * cc], 0, 0x3120), a[0], a[1]);
                        widen4<kKind>(__byte_perm(b[2 * cc + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                        for (int n = 0; n < kOct; ++n) mma<false>(o[2 * dd + cc][n], a, pf[n][0], pf[n][1]);
                    }
                }
            }
        }
        copies_wait<0>();

        // ---- the warps' parts ----
#pragma unroll
        for (int n = 0; n < kOct; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int q = 4; q < 32; q <<= 1) l[n][e] += __shfl_xor_sync(kFull, l[n][e], q);
                if constexpr (kQuantised) {
                    Product::settle(m[n][e], pe[n][e], l[n][e]);
                    l[n][e] *= Product::of_l(pe[n][e]);
                }
                if (g == 0) {
                    row_m[warp][8 * n + 2 * tq + e] = m[n][e];
                    row_l[warp][8 * n + 2 * tq + e] = l[n][e];
                }
            }
        __syncthreads();                                    // (every warp has read its ring)
        float* const ow = reinterpret_cast<float*>(ring0);  // [warp][row][D]
        auto top_of = [&](int row) {
            float top = row_m[0][row];
#pragma unroll
            for (int w2 = 1; w2 < kWarps; ++w2) top = fmaxf(top, row_m[w2][row]);
            return top;
        };
        if (tid < kRowsU) {
            const float top = top_of(tid);
            float sum = 0.f;
#pragma unroll
            for (int w2 = 0; w2 < kWarps; ++w2) sum += ex2(row_m[w2][tid] - top) * row_l[w2][tid];
            row_inv[tid] = part >= 0 ? 1.f : sum == 0.f ? 0.f : 1.0f / sum;
            if (part >= 0) {
                float* ml = p.ws + static_cast<int64_t>(2 * gridDim.x) * kRowsU * D + static_cast<int64_t>(part) * 2 * kRowsU;
                ml[tid] = top;
                ml[kRowsU + tid] = sum;
            }
        }
        float a[kOct][2];
#pragma unroll
        for (int n = 0; n < kOct; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                a[n][e] = m[n][e] - top_of(8 * n + 2 * tq + e);
                a[n][e] = kQuantised ? Product::of_o(a[n][e] + pe[n][e]) : ex2(a[n][e]);
            }
#pragma unroll
        for (int n = 0; n < kOct; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * n + 2 * tq + e;
                if (row >= d.rows) continue;
                float* const to = ow + (warp * kRowsU + row) * D;
#pragma unroll
                for (int dn = 0; dn < D / 16; ++dn) {
                    // (a factor of 0 is a product too: what is no number stays none, whichever warp took it)
                    const float x = o[dn][n][e] * a[n][e], y = o[dn][n][e + 2] * a[n][e];
                    // (columns exchanged by the row, so that the rows of a store lie in different banks)
                    if constexpr (kQuantised) {
                        *reinterpret_cast<float2*>(to + ((16 * dn + 2 * g) ^ ((row & 2) << 3))) = make_float2(x, y);
                    } else {
                        to[(16 * dn + g) ^ ((row & 6) << 2)] = x;
                        to[(16 * dn + g + 8) ^ ((row & 6) << 2)] = y;
                    }
                }
            }
        __syncthreads();
#pragma unroll 1
        for (int id = tid; id < d.rows * (D / 4); id += kThreads) {
            const int r = id / (D / 4), col = 4 * (id - r * (D / 4));
            const int at4 = kQuantised ? col ^ ((r & 2) << 3) : col ^ ((r & 6) << 2);
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w2 = 0; w2 < kWarps; ++w2) {
                const float4 y = *reinterpret_cast<const float4*>(ow + (w2 * kRowsU + r) * D + at4);
                x[0] += y.x;
                x[1] += y.y;
                x[2] += y.z;
                x[3] += y.w;
            }
            if (part < 0) {
                const float inv = row_inv[r];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] *= inv;
                put_out(p, row_out[r] + col, row_z[r] + col, x);
            } else {
                *reinterpret_cast<float4*>(p.ws + (static_cast<int64_t>(part) * kRowsU + r) * D + col) = make_float4(x[0], x[1], x[2], x[3]);
            }
        }
        if (!whole && tid == 0) put_record(meta, d, total, ctas);
        __syncthreads();
    }
}

template <int kKind, int D, int kOct>
cudaError_t launch(const AttnParams& p, bool joins, int grid, cudaStream_t stream) {
    using S = Shape<kKind, D, kOct>;
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 64 || !__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE)) {
        err = cudaFuncSetAttribute(gdn_attn_decode_kernel<kKind, D, kOct>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (err != cudaSuccess) return err;
        if (dev < 64) __atomic_store_n(&ready[dev], true, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, gdn_attn_decode_kernel<kKind, D, kOct>, p);
    if (err != cudaSuccess || !joins) return err;
    cfg.gridDim = dim3(static_cast<unsigned>(grid * kJSplit<8 * kOct>), 1, 1);
    cfg.blockDim = dim3(kJThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, gdn_attn_join_kernel<D, 8 * kOct>, p, grid);
}

// the launch for one type of cache (a translation unit each), and its CTAs: what is resident at once
template <int kKind, int kOct>
cudaError_t by_dim(const AttnParams& p, int D, bool joins, int grid, cudaStream_t s) {
    if constexpr (kOct <= 2) {
        if (D == 192) return launch<kKind, 192, kOct>(p, joins, grid, s);
        if (D == 256) return launch<kKind, 256, kOct>(p, joins, grid, s);
    }
    return D == 64 ? launch<kKind, 64, kOct>(p, joins, grid, s) : launch<kKind, 128, kOct>(p, joins, grid, s);
}
template <int kKind, int kOct>
int ctas_of_sm(int D) {
    if constexpr (kOct <= 2) {
        if (D == 192) return Shape<kKind, 192, kOct>::kCtas;
        if (D == 256) return Shape<kKind, 256, kOct>::kCtas;
    }
    return D == 64 ? Shape<kKind, 64, kOct>::kCtas : Shape<kKind, 128, kOct>::kCtas;
}
template <int kKind, int kOct>
int grid_of(int D) {
    const int n = (sm_count() ? sm_count() : 148) * ctas_of_sm<kKind, kOct>(D);
    return n < kMaxCtas ? n : kMaxCtas;
}
template <int kKind, int kOct>
int64_t workspace_of(int D) {
    const int64_t grid = grid_of<kKind, kOct>(D);
    return grid * kMetaInts * 4 + 2 * grid * 8 * kOct * (D + 2) * 4;
}
template <int kKind, int kOct>
cudaError_t launch_oct(AttnParams p, int D, void* workspace, cudaStream_t s) {
    const int grid = grid_of<kKind, kOct>(D);
    p.meta = static_cast<int32_t*>(workspace);
    p.ws = reinterpret_cast<float*>(p.meta + static_cast<int64_t>(grid) * kMetaInts);
    p.stand_side_by_side();
    // a unit of one block has nothing to join
    const bool joins = static_cast<int64_t>(p.pg.cols) * p.pg.page + kKeys > kCutKeys;
    return by_dim<kKind, kOct>(p, D, joins, grid, s);
}
// Units of up to 32 rows where the accumulators fit, else 16: with two tiles of 16 the cache is read twice
// (24 rows of 32 sequences of up to 4096, head dim 128: 64 us against 50 in bf16, 57 and 45 in e4m3; 32 rows: 65
// and 59, 57 and 53).
constexpr int octets(int rows, int D) { return rows <= 8 ? 1 : rows <= 16 || D > 128 ? 2 : rows <= 24 ? 3 : 4; }
template <int kKind>
int64_t workspace_kind(int rows, int D) {
    const int n = octets(rows, D);
    return n == 1 ? workspace_of<kKind, 1>(D) : n == 2 ? workspace_of<kKind, 2>(D) : n == 3 ? workspace_of<kKind, 3>(D) : workspace_of<kKind, 4>(D);
}
template <int kKind>
cudaError_t launch_kind(const AttnParams& p, int rows, int D, void* workspace, cudaStream_t s) {
    const int n = octets(rows, D);
    return n == 1   ? launch_oct<kKind, 1>(p, D, workspace, s)
           : n == 2 ? launch_oct<kKind, 2>(p, D, workspace, s)
           : n == 3 ? launch_oct<kKind, 3>(p, D, workspace, s)
                    : launch_oct<kKind, 4>(p, D, workspace, s);
}

}  // namespace gdn_attn_warp
