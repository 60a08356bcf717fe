// libgdnspec: the attention of a step's tokens over the paged key-value cache
// (gdn_attn_decode; its C entry point is in gdnkv.cu).  Declared in include/gdnspec.h.
//
// For a row of scores s_j over keys, with any reference m and weights p_j = 2^(s_j - m)
// (log2 e is in the scale), the output is (sum p_j v_j) / (sum p_j): keys may come in any
// pieces, each with its own m, and (m, sum p, sum p v) of two pieces add up after a factor
// 2^(m - m') on one of them.  So one pass over the cache does, in three levels: a warp over
// its keys, the warps of a CTA, and the CTAs that share a sequence.
//
// A unit is one (sequence, cache head, tile of 16 query rows); its rows are the heads of the
// group times the tokens.  All units' keys, in blocks of 64, form one line that is cut evenly
// among the CTAs, whatever the lengths; a CTA computes from the lengths alone where its part
// begins.  A part that is a whole unit is finished where it is; the others go to the workspace
// and a second launch joins them in order.
#include "gdnattn.cuh"

using namespace gdn_attn;

namespace {

constexpr int kTileRows = 16, kCutKeys = 64;
template <int kT>
struct Cut {                            // (gdnattn.cuh)
    static constexpr int kThreads = kT;
    static constexpr int kBlock = kCutKeys;
    static constexpr int kRows = kTileRows;
};

// ---- instructions ---------------------------------------------------------------------------

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// C[16][8] += A[16][16] B[16][8]; bf16 or fp16 operands
template <bool kBf16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBf16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// ---- what the cache's types differ in -------------------------------------------------------

enum Kind { kBf16, kF16, kE4m3, kI8 };

// two 8-bit codes, in the low and high half of w's selected bytes, as fp16 (exact for either type)
template <int kKind>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& ab, uint32_t& cd) {
    if constexpr (kKind == kE4m3) {
        const __half2_raw x = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3);
        const __half2_raw y = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
        ab = static_cast<uint32_t>(x.x) | (static_cast<uint32_t>(x.y) << 16);
        cd = static_cast<uint32_t>(y.x) | (static_cast<uint32_t>(y.y) << 16);
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

// ---- the kernel ---------------------------------------------------------------------------------
//
// Each warp has keys of its own, 16 at a time, through a ring of asynchronous copies that no other
// warp touches: K and V of 16 keys are an item each.  S = Q K^T and O += P V run on the tensor cores
// (m16n8k16, 16 query rows); the scores' layout is that of the weights as left operand.
// The reference m of a row only moves when a score passes it by more than 2^kSlack: then
// O and the sums are scaled down.  kLift keeps weights far from the end of fp16's range.
//
// fp16 and 8-bit caches run on fp16 operands: codes are exact in fp16, a key's scale multiplies its
// score and a value's scale its weight.  So that weight times scale fits fp16, scales count in
// units of a power of two that a warp keeps for all its values, the largest yet.  q becomes fp16 by
// a power of two of its row, which goes into the row's scale.  A bf16 cache runs on bf16 operands,
// and a weight is the sum of two bf16 parts: one has 8 bits only.

constexpr float kLift = 6.f, kSlack = 14.f;

template <int kKind, int D>
struct Shape {
    static constexpr int kBytes = kKind <= kF16 ? 2 : 1;
    static constexpr int kRow = D * kBytes;                     // bytes of a key
    static constexpr int kScales = kBytes == 1 ? 4 * kKeys : 0;
    static constexpr int kItem = kKeys * kRow + kScales;        // K or V of 16 keys
    static constexpr int kWarps = D * kBytes > 256 ? 8 : 4;
    static constexpr int kCtas = kWarps == 8 ? 1 : 2;           // an SM
    static constexpr int kRing0 = (kCtas == 1 ? 200 * 1024 : 96 * 1024) / (kWarps * kItem);
    static constexpr int kRing = kRing0 > 12 ? 12 : kRing0;     // items of a warp, on their way or in use
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRingBytes = kWarps * kRing * kItem;
    static constexpr int kJoinBytes = kWarps * kTileRows * D * 4;   // the warps' O, in the ring's place
    static constexpr int kQ = kTileRows * D * 2;
    static constexpr int kSmem = kQ + (kRingBytes > kJoinBytes ? kRingBytes : kJoinBytes);
    static_assert(kRing >= 3, "a ring of K, V and one more");
};

// byte of 16-byte chunk c of key r in an item: the chunks of a row in an order that depends on the
// row, so that neither ldmatrix (8 rows, one chunk) nor a K fragment's load (2 rows, 4 chunks)
// meets a bank twice
template <int kKind, int D, bool kIsK>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    constexpr int kRow = Shape<kKind, D>::kRow;
    if constexpr (kKind <= kF16) return r * kRow + 16 * (c ^ (r & 7));
    else if constexpr (kRow % 128 != 0) return r * kRow + 16 * (kIsK ? c : c ^ ((r >> 1) & 3));
    else return r * kRow + 16 * (kIsK ? c ^ ((r & 1) << 2) : c ^ (r & 7));
}

// column of a row in the warps' parts, so that the rows of a store lie in different banks
template <bool kQuantised>
__device__ __forceinline__ int join_col(int r, int col) {
    return kQuantised ? col ^ ((r & 1) << 4) : col ^ ((r & 3) << 3);
}

// An infinity or NaN among values that some rows see and some do not: its products would reach the
// others as 0 * NaN.  It is added to the rows that see it (whatever its weight: the sum is no number
// then) and taken out of the tile.
template <int kKind, int D>
__device__ __noinline__ void add_unseen_cold(float (*o)[4], uint32_t vs0, int x0, int first0, int first1, int last0, int last1,
                                             uint32_t live, int lane) {
    constexpr uint32_t kExp = kKind == kBf16 ? 0x7f80u : 0x7c00u;
    const int tq = lane & 3;
    for (int n = 0; n < D / 8; ++n)
        for (int kk = 0; kk < kKeys; ++kk) {
            uint32_t raw;                       // columns 8 n + 2 tq and the next
            const uint32_t at = vs0 + chunk_at<kKind, D, false>(kk, n) + 4 * tq;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(raw) : "r"(at) : "memory");
            for (int e = 0; e < 2; ++e) {
                const uint32_t x = (raw >> (16 * e)) & 0xffffu;
                if ((x & kExp) != kExp || !((live >> kk) & 1u)) continue;
                const __half_raw hr = {static_cast<unsigned short>(x)};
                const float v = kKind == kBf16 ? __uint_as_float(x << 16) : __half2float(__half(hr));
                if (x0 + kk >= first0 && x0 + kk <= last0) o[n][e] += v;
                if (x0 + kk >= first1 && x0 + kk <= last1) o[n][2 + e] += v;
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
template <int kKind, int D>
__device__ __forceinline__ void add_unseen(float (&o)[D / 8][4], uint32_t vs0, int x0, const int (&first)[2], const int (&last)[2],
                                           uint32_t live, int lane) {
    constexpr uint32_t kExp = kKind == kBf16 ? 0x7f80u : 0x7c00u;
    bool bad = false;
    for (int id = lane; id < kKeys * D / 2; id += 32) {
        uint32_t raw;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(raw) : "r"(vs0 + 4 * id) : "memory");
        bad = bad || (raw & kExp) == kExp || ((raw >> 16) & kExp) == kExp;
    }
    if (__any_sync(kFull, bad)) {
        float copy[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) copy[n][e] = o[n][e];
        add_unseen_cold<kKind, D>(copy, vs0, x0, first[0], first[1], last[0], last[1], live, lane);
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = copy[n][e];
    }
}

template <int kKind, int D>
__global__ void __launch_bounds__(Shape<kKind, D>::kThreads, Shape<kKind, D>::kCtas) gdn_attn_decode_kernel(const AttnParams p) {
    using S = Shape<kKind, D>;
    constexpr int kT = S::kThreads;
    using G = Cut<kT>;
    constexpr bool kQuantised = S::kBytes == 1;
    constexpr bool kB = kKind == kBf16;
    constexpr int kSteps = D / 16;                  // of the products over D
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Line<G> line;
    __shared__ float row_m[S::kWarps][kTileRows], row_l[S::kWarps][kTileRows];
    __shared__ float q_scale[kTileRows];
    __shared__ float join_m[kTileRows], join_l[kTileRows];
    __shared__ uint32_t live_keys[S::kWarps][S::kRing];
    unsigned char* const sq = smem;
    unsigned char* const ring0 = smem + S::kQ;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    dep_wait();
    begin_line<G>(p, line);
    dep_launch();
    const int64_t total = line.total;
    const int ctas = ctas_of(total, gridDim.x, 2);
    const int cta = blockIdx.x;
    int32_t* const meta = p.meta + static_cast<int64_t>(cta) * kMetaInts;
    if (tid == 0) meta[0] = meta[8] = -1;           // (no part yet)
    if (cta >= ctas) return;
    const int64_t w0 = quotient(total * cta, ctas), w1 = quotient(total * (cta + 1), ctas);
    const uint32_t my_ring = saddr(ring0) + warp * S::kRing * S::kItem;

    for (int64_t w = w0; w < w1;) {
        // ---- the unit at block w of the line ----
        const int k = sequence_at<G>(p, line, w);
        const Piece d = piece_at<G>(p, line, k, w, w1);
        const int seq = d.seq, head = d.head, tile = d.tile, past = d.past, row0 = d.row0, rows = d.rows, key0 = d.key0, key1 = d.key1;
        const int b0 = d.b0, b1 = d.b1;
        const bool whole = b0 == 0 && b1 == d.blocks;
        const int part = whole ? -1 : b0 > 0 ? 2 * cta : 2 * cta + 1;
        if (!whole && tid == 0) put_record(meta, d, w, total, ctas);
        const int items = 2 * max(0, ((key1 - key0 + kKeys - 1) / kKeys - warp + S::kWarps - 1) / S::kWarps);

        // ---- the ring ----
        const char* const kc = static_cast<const char*>(p.k) + head * p.pg.head_stride * S::kBytes;
        const char* const vc = static_cast<const char*>(p.v) + head * p.pg.head_stride * S::kBytes;
        const int32_t* const table = p.pg.table + static_cast<int64_t>(seq) * p.pg.table_stride;
        const int my_key = lane & 15;
        int next_page = -1;                         // of this lane's key in the next block
        auto look_up = [&](int block) {
            const int x = key0 + (warp + block * S::kWarps) * kKeys + my_key;
            next_page = x < key1 ? ld(table + p.pg.page_of(x)) : -1;
        };
        int64_t at = 0, sat = 0;                    // this lane's key of the block on its way
        bool live = false;
        int issued = 0;
        auto issue = [&]() {
            if (issued < items) {
                const int slot = issued % S::kRing;
                const uint32_t dst = my_ring + slot * S::kItem;
                const bool is_k = (issued & 1) == 0;
                if (is_k) {
                    const int block = issued >> 1;
                    const int x = key0 + (warp + block * S::kWarps) * kKeys + my_key;
                    live = next_page >= 0 && next_page < p.pg.num_pages;
                    if (next_page >= p.pg.num_pages) raise(p.status, GDN_FLAG_SLOT_RANGE);
                    const int64_t in = x - p.pg.page_of(x) * p.pg.page;
                    at = live ? next_page * p.pg.page_stride + in * p.pg.token_stride : 0;
                    sat = live ? next_page * p.pg.s_page + in * p.pg.s_token + head * p.pg.s_head : 0;
                    const uint32_t mask = __ballot_sync(kFull, live) & 0xffffu;
                    if (lane == 0) live_keys[warp][slot] = mask;
                    look_up(block + 1);
                }
                const char* const src = is_k ? kc : vc;
                constexpr int kChunks = S::kRow / 16;               // of a key
#pragma unroll
                for (int it = 0; it < kChunks / 2; ++it) {
                    const int id = it * 32 + lane;
                    const int r = id / kChunks, c = id - r * kChunks;
                    const int64_t from = __shfl_sync(kFull, at, r);
                    const bool has = __shfl_sync(kFull, live ? 1 : 0, r) != 0;
                    copy16(dst + (is_k ? chunk_at<kKind, D, true>(r, c) : chunk_at<kKind, D, false>(r, c)), src + from * S::kBytes + 16 * c, has);
                }
                if constexpr (kQuantised) {
                    if (lane < kKeys) copy4(dst + kKeys * S::kRow + 4 * lane, (is_k ? p.k_scale : p.v_scale) + sat, live);
                }
            }
            copies_commit();
            ++issued;
        };
        look_up(0);
#pragma unroll
        for (int u = 0; u < S::kRing - 1; ++u) issue();

        // ---- q: [16][D] in shared memory, fp16 with a power of two per row, or bf16 as it is ----
        {
            constexpr int kPer = kT / kTileRows;                    // threads of a row
            const int r = tid / kPer, j = tid % kPer;
            const int rr = tile * kTileRows + r;
            const bool has = r < rows;
            const int t = rr / p.ratio, hq = head * p.ratio + rr - t * p.ratio;
            const __nv_bfloat16* src = has ? p.q + token_row(p, row0 + t) * p.q_stride + static_cast<int64_t>(hq) * D : p.q;
            uint4 raw[(D / 8 + kPer - 1) / kPer];
            uint32_t big = 0;
#pragma unroll
            for (int u = 0; u < (D / 8 + kPer - 1) / kPer; ++u) {
                const int c = j + u * kPer;
                raw[u] = make_uint4(0, 0, 0, 0);
                if (has && c < D / 8) raw[u] = ld(reinterpret_cast<const uint4*>(src) + c);
                const uint32_t x[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) big = max(big, max(x[e] & 0x7fffu, (x[e] >> 16) & 0x7fffu));
            }
            float down = 1.f, up = 1.f;
            if constexpr (!kB) {
#pragma unroll
                for (int o = kPer / 2; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(kFull, big, o, kPer));
                const int e = min(max(static_cast<int>(big >> 7), 1), 253);     // exponent: the row's largest becomes 1 to 2
                if ((big >> 7) != 255) {                                        // (an infinity or NaN stays what it is)
                    down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                    up = __uint_as_float(static_cast<uint32_t>(e) << 23);
                }
            }
            if (j == 0) q_scale[r] = p.scale * up;
#pragma unroll
            for (int u = 0; u < (D / 8 + kPer - 1) / kPer; ++u) {
                const int c = j + u * kPer;
                if (c < D / 8) {
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
        uint32_t qf[kSteps][4];
        if constexpr (!kQuantised) {
            const int r = lane & 15, c = lane >> 4;
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) ldsm4(qf[ks], saddr(sq) + r * D * 2 + 16 * ((2 * ks + c) ^ (r & 7)));
        } else {
            // the elements in the order that a K fragment has them: 16 neighbouring ones per lane of a quad
#pragma unroll
            for (int seg = 0; seg < D / 64; ++seg)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const int d = seg * 64 + tq * 16 + 4 * ks;
                    const uint2 x = *reinterpret_cast<const uint2*>(sq + g * D * 2 + 16 * ((d / 8) ^ (g & 7)) + (d % 8) * 2);
                    const uint2 y = *reinterpret_cast<const uint2*>(sq + (g + 8) * D * 2 + 16 * ((d / 8) ^ (g & 7)) + (d % 8) * 2);
                    qf[4 * seg + ks][0] = x.x;
                    qf[4 * seg + ks][1] = y.x;
                    qf[4 * seg + ks][2] = x.y;
                    qf[4 * seg + ks][3] = y.y;
                }
        }
        // this thread's rows g and g + 8: their scale, and the positions that they see
        float qs[2], m[2], l[2];
        int last[2], first[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = min((tile * kTileRows + g + 8 * h) / p.ratio, d.n - 1);
            qs[h] = q_scale[g + 8 * h];
            last[h] = past + t;
            first[h] = p.window > 0 ? max(0, last[h] - p.window + 1) : 0;
            m[h] = -INFINITY;
            l[h] = 0.f;
        }
        const int all_lo = p.window > 0 ? max(0, past + d.n - p.window) : 0, all_hi = past + 1;      // seen by every row
        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        int unit_e = 1;                             // exponent (biased) of the values' scale unit

        // ---- the keys ----
        for (int i = 0; i < items; i += 2) {
            copies_wait<S::kRing - 2>();
            __syncwarp();
            issue();
            const uint32_t ks0 = my_ring + (i % S::kRing) * S::kItem;
            const uint32_t vs0 = my_ring + ((i + 1) % S::kRing) * S::kItem;
            float s[2][4];
            {
                float c0[2][4], c1[2][4];           // (two chains of products)
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c0[nt][e] = c1[nt][e] = 0.f;
                if constexpr (!kQuantised) {
                    const int r = (lane & 7) + ((lane >> 4) << 3), c = (lane >> 3) & 1;
#pragma unroll
                    for (int ks = 0; ks < kSteps; ++ks) {
                        uint32_t b[4];
                        ldsm4(b, ks0 + chunk_at<kKind, D, true>(r, 2 * ks + c));
                        mma<kB>(ks & 1 ? c1[0] : c0[0], qf[ks], b[0], b[1]);
                        mma<kB>(ks & 1 ? c1[1] : c0[1], qf[ks], b[2], b[3]);
                    }
                } else {
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int seg = 0; seg < D / 64; ++seg) {
                            uint4 x;
                            const uint32_t a = ks0 + chunk_at<kKind, D, true>(nt * 8 + g, 4 * seg + tq);
                            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a) : "memory");
                            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks) {
                                uint32_t b0, b1;
                                widen4<kKind>(xs[ks], b0, b1);
                                mma<false>(ks & 1 ? c1[nt] : c0[nt], qf[4 * seg + ks], b0, b1);
                            }
                        }
                }
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    float f[2] = {1.f, 1.f};
                    if constexpr (kQuantised)
                        asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(f[0]), "=f"(f[1]) : "r"(ks0 + kKeys * S::kRow + 4 * (nt * 8 + 2 * tq)) : "memory");
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = (c0[nt][e] + c1[nt][e]) * qs[e >> 1];
                        s[nt][e] = kQuantised ? x * f[e & 1] : x;
                    }
                }
            }
            const int x0 = key0 + (warp + (i >> 1) * S::kWarps) * kKeys;
            const uint32_t live = live_keys[warp][i % S::kRing];
            const bool partly = x0 < all_lo || x0 + kKeys > all_hi;
            if (partly || live != 0xffffu) {
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int kk = nt * 8 + 2 * tq + (e & 1), x = x0 + kk;
                        if (x < first[e >> 1] || x > last[e >> 1] || !((live >> kk) & 1u)) s[nt][e] = -INFINITY;
                    }
            }
            // ---- the softmax's reference and weights ----
            float mx[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 2));
            }
            copies_wait<S::kRing - 2>();            // (V: its scales are wanted now)
            __syncwarp();
            issue();
            float f[2][2];
            bool grows = mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack;
            int e_max = unit_e;
            if constexpr (kQuantised) {
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(f[nt][0]), "=f"(f[nt][1]) : "r"(vs0 + kKeys * S::kRow + 4 * (nt * 8 + 2 * tq)) : "memory");
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int ex = (__float_as_uint(f[nt][e]) >> 23) & 0xff;
                        if (ex != 255) e_max = max(e_max, min(ex, 253));
                    }
                }
                e_max = max(e_max, __shfl_xor_sync(kFull, e_max, 1));
                e_max = max(e_max, __shfl_xor_sync(kFull, e_max, 2));
                grows = grows || e_max > unit_e;
            }
            if (__any_sync(kFull, grows)) {
                float a[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float now = mx[h] > m[h] + kSlack ? mx[h] - kLift : m[h];
                    a[h] = m[h] == now ? 1.f : ex2(m[h] - now);
                    m[h] = now;
                    l[h] *= a[h];
                }
                float b = 1.f;
                if constexpr (kQuantised) {
                    if (e_max > unit_e) b = e_max - unit_e > 126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - (e_max - unit_e)) << 23);
                    unit_e = e_max;
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][e] *= a[e >> 1] * b;
            }
            float w8[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float ref = m[e >> 1] == -INFINITY ? 0.f : m[e >> 1];
                    const float pe = ex2(s[nt][e] - ref);
                    l[e >> 1] += pe;
                    w8[nt][e] = pe;
                    if constexpr (kQuantised) {
                        const float unit_inv = __uint_as_float(static_cast<uint32_t>(max(254 - unit_e, 1)) << 23);
                        w8[nt][e] = s[nt][e] == -INFINITY ? 0.f : pe * (f[nt][e & 1] * unit_inv);   // (a masked value's scale may be NaN)
                    }
                }
            uint32_t pf[4], pl[4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float a = w8[nt][2 * h], b = w8[nt][2 * h + 1];
                    if constexpr (kB) {
                        pf[2 * nt + h] = pack_b(a, b);
                        pl[2 * nt + h] = pack_b(a - __uint_as_float(pf[2 * nt + h] << 16), b - __uint_as_float(pf[2 * nt + h] & 0xffff0000u));
                    } else {
                        pf[2 * nt + h] = pack_h(a, b);
                    }
                }
            if constexpr (!kQuantised) {
                if (partly) add_unseen<kKind, D>(o, vs0, x0, first, last, live, lane);
            }
            // ---- O += P V ----
            if constexpr (!kQuantised) {
                const int r = lane & 15, c = lane >> 4;
#pragma unroll
                for (int dn = 0; dn < D / 16; ++dn) {
                    uint32_t b[4];
                    ldsm4t(b, vs0 + chunk_at<kKind, D, false>(r, 2 * dn + c));
                    mma<kB>(o[2 * dn], pf, b[0], b[1]);
                    mma<kB>(o[2 * dn + 1], pf, b[2], b[3]);
                    if constexpr (kB) {
                        mma<kB>(o[2 * dn], pl, b[0], b[1]);
                        mma<kB>(o[2 * dn + 1], pl, b[2], b[3]);
                    }
                }
            } else {
                const int r = lane & 15, c = lane >> 4;
#pragma unroll
                for (int dn = 0; dn < D / 32; ++dn) {       // 32 columns: two chunks
                    uint32_t b[4];
                    ldsm4t(b, vs0 + chunk_at<kKind, D, false>(r, 2 * dn + c));
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        // pairs of neighbouring columns of two keys: the even columns are one tile, the odd ones the next
                        uint32_t e0, o0, e1, o1;
                        widen4<kKind>(__byte_perm(b[2 * cc], 0, 0x3120), e0, o0);
                        widen4<kKind>(__byte_perm(b[2 * cc + 1], 0, 0x3120), e1, o1);
                        mma<false>(o[4 * dn + 2 * cc], pf, e0, e1);
                        mma<false>(o[4 * dn + 2 * cc + 1], pf, o0, o1);
                    }
                }
            }
        }
        copies_wait<0>();

        // ---- the warps' parts ----
        // (row sums over the quad; O in the values' unit)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(kFull, l[h], 1);
            l[h] += __shfl_xor_sync(kFull, l[h], 2);
            if (tq == 0) {
                row_m[warp][g + 8 * h] = m[h];
                row_l[warp][g + 8 * h] = l[h];
            }
        }
        __syncthreads();                                    // (every warp has read its ring)
        float* const ow = reinterpret_cast<float*>(ring0);
        {
            float a[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = -INFINITY;
#pragma unroll
                for (int w2 = 0; w2 < S::kWarps; ++w2) top = fmaxf(top, row_m[w2][g + 8 * h]);
                a[h] = m[h] == -INFINITY ? 0.f : ex2(m[h] - top);
                if (warp == 0 && tq == 0) {
                    float sum = 0.f;
#pragma unroll
                    for (int w2 = 0; w2 < S::kWarps; ++w2)
                        // (a row whose scores are all NaN has the reference -inf and the sum NaN, which it keeps)
                        sum += (row_m[w2][g + 8 * h] == -INFINITY ? 0.f : ex2(row_m[w2][g + 8 * h] - top)) * row_l[w2][g + 8 * h];
                    join_m[g + 8 * h] = top;
                    join_l[g + 8 * h] = sum;
                }
                if constexpr (kQuantised) a[h] *= __uint_as_float(static_cast<uint32_t>(unit_e) << 23);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = g + 8 * h;
                float* const to = ow + (warp * kTileRows + r) * D;
                auto part_of = [&](int n, int e) { return a[h] == 0.f ? 0.f : o[n][2 * h + e] * a[h]; };
                if constexpr (!kQuantised) {                // column 8 n + 2 tq + e
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
                        *reinterpret_cast<float2*>(to + join_col<kQuantised>(r, 8 * n + 2 * tq)) = make_float2(part_of(n, 0), part_of(n, 1));
                } else {                                    // tiles of even and of odd columns
#pragma unroll
                    for (int n = 0; n < D / 8; n += 2)
                        *reinterpret_cast<float4*>(to + join_col<kQuantised>(r, 8 * n + 4 * tq)) =
                            make_float4(part_of(n, 0), part_of(n + 1, 0), part_of(n, 1), part_of(n + 1, 1));
                }
            }
        }
        __syncthreads();
        for (int id = tid; id < rows * (D / 4); id += kT) {
            const int r = id / (D / 4), col = 4 * (id - r * (D / 4));
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w2 = 0; w2 < S::kWarps; ++w2) {
                const float4 y = *reinterpret_cast<const float4*>(ow + (w2 * kTileRows + r) * D + join_col<kQuantised>(r, col));
                x[0] += y.x;
                x[1] += y.y;
                x[2] += y.z;
                x[3] += y.w;
            }
            if (part < 0) {
                const float inv = join_l[r] == 0.f ? 0.f : 1.0f / join_l[r];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] *= inv;
                const int rr = tile * kTileRows + r, t = rr / p.ratio;
                put_out(p, token_row(p, row0 + t), head * p.ratio + rr - t * p.ratio, D, col, x);
            } else {
                *reinterpret_cast<float4*>(p.ws + (static_cast<int64_t>(part) * kTileRows + r) * D + col) = make_float4(x[0], x[1], x[2], x[3]);
            }
        }
        if (part >= 0 && tid < kTileRows) {
            float* ml = p.ws + static_cast<int64_t>(2 * gridDim.x) * kTileRows * D + static_cast<int64_t>(part) * 2 * kTileRows;
            ml[tid] = join_m[tid];
            ml[kTileRows + tid] = join_l[tid];
        }
        __syncthreads();
        w += b1 - b0;
    }
}


template <int kKind, int D>
cudaError_t launch(const AttnParams& p, bool joins, int grid, cudaStream_t stream) {
    using S = Shape<kKind, D>;
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 64 || !__atomic_load_n(&ready[dev], __ATOMIC_RELAXED)) {
        err = cudaFuncSetAttribute(gdn_attn_decode_kernel<kKind, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (err != cudaSuccess) return err;
        if (dev < 64) __atomic_store_n(&ready[dev], true, __ATOMIC_RELAXED);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(S::kThreads, 1, 1);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, gdn_attn_decode_kernel<kKind, D>, p);
    if (err != cudaSuccess || !joins) return err;
    cfg.blockDim = dim3(kJThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, gdn_attn_join_kernel<D, kTileRows>, p, grid);
}

template <int kKind>
cudaError_t by_dim(const AttnParams& p, int D, bool joins, int grid, cudaStream_t s) {
    return D == 64    ? launch<kKind, 64>(p, joins, grid, s)
           : D == 128 ? launch<kKind, 128>(p, joins, grid, s)
           : D == 192 ? launch<kKind, 192>(p, joins, grid, s)
                      : launch<kKind, 256>(p, joins, grid, s);
}

template <int kKind>
constexpr int kCtasOf(int D) {
    return D == 64    ? Shape<kKind, 64>::kCtas
           : D == 128 ? Shape<kKind, 128>::kCtas
           : D == 192 ? Shape<kKind, 192>::kCtas
                      : Shape<kKind, 256>::kCtas;
}

// CTAs of the launch: what is resident at once
int grid_of(int D, gdn_dtype type) {
    const int sms = sm_count() ? sm_count() : 148;
    const int ctas = type == GDN_BF16 || type == GDN_F16 ? kCtasOf<kF16>(D) : kCtasOf<kE4m3>(D);
    const int n = sms * ctas;
    return n < kMaxCtas ? n : kMaxCtas;
}

}  // namespace

namespace gdn_kv {

// Which kernel: the tcgen05 one pays from the second tile of 16 query rows on, which this one would read the cache for
// once more (16 sequences of up to 16384 positions, head dim 256, bf16: 32 rows 82 us here and 76 there; 2 of 65535,
// 64 rows: 136 and 66; 32 of 8192, head dim 128, e4m3, 64 rows: 313 and 167); up to 16 rows this one is faster (32 sequences
// of up to 4096 positions, 4 rows: 67 and 85; 256 of up to 500, one row: 71 and 125).  It wants pages of whole groups of 8
// positions, and has no int8 products.
static bool on_tc(const AttnParams& p, gdn_dtype type) {
    return type != GDN_I8 && p.ratio * p.max_T > kTileRows && p.pg.page % 8 == 0 && p.pg.num_pages < (1ll << 31);
}

int64_t attn_workspace(const AttnParams& p, int D, gdn_dtype type) {
    if (on_tc(p, type)) return attn_tc_workspace(D);
    const int64_t grid = grid_of(D, type);
    return grid * kMetaInts * 4 + 2 * grid * kTileRows * (D + 2) * 4;
}

cudaError_t launch_attn(AttnParams p, int D, gdn_dtype type, void* workspace, cudaStream_t stream) {
    if (on_tc(p, type))
        return type == GDN_BF16  ? launch_attn_tc_bf16(p, D, workspace, stream)
               : type == GDN_F16 ? launch_attn_tc_f16(p, D, workspace, stream)
                                 : launch_attn_tc_e4m3(p, D, workspace, stream);
    const int grid = grid_of(D, type);
    p.meta = static_cast<int32_t*>(workspace);
    p.ws = reinterpret_cast<float*>(p.meta + static_cast<int64_t>(grid) * kMetaInts);
    // a unit of one block has nothing to join
    const bool joins = static_cast<int64_t>(p.pg.cols) * p.pg.page + kKeys > kCutKeys;
    return type == GDN_BF16   ? by_dim<kBf16>(p, D, joins, grid, stream)
           : type == GDN_F16  ? by_dim<kF16>(p, D, joins, grid, stream)
           : type == GDN_E4M3 ? by_dim<kE4m3>(p, D, joins, grid, stream)
                              : by_dim<kI8>(p, D, joins, grid, stream);
}

}  // namespace gdn_kv
