// libgdnspec: the paged key-value cache of the attention layers beside the recurrent
// ones: rows into it (gdn_kv_write), quantised where it has 8 bits, and back out of it
// (gdn_kv_read), with the C entry points of the cache and of the attention over it
// (launched in gdnattn.cu).  Declared in include/gdnspec.h.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "gdnkv.h"

using namespace gdn_common;
using namespace gdn_kv;

namespace {

// ---- rows to and from the cache ------------------------------------------------------
//
// Both are copies, one with a maximum over each row's D elements: the bytes bound them for
// many rows, the chain offsets -> page -> row for few (32 rows of 8 heads 2.4 us).  A CTA takes a
// tile of neighbouring rows; first a thread per row finds its sequence, page and place, then
// groups of D / 32 lanes move one head's row of k or v each, kParts pieces of 8 elements a lane,
// all loads of a row on their way at once.  The instructions for an item's place come close to the
// bytes' time, so a lane has four pieces of it: 16211 rows of 8 heads of 128 into an e4m3 cache and back
// 35 us (5.7 TB/s), with two pieces 40, with one 49; 120007 rows read from it 117 us (6.3 TB/s), 118, 142.
// Loads for the next item ahead of the stores of this one gained nothing (35, 116).

constexpr int kRThreads = 256, kRCtas = 4;      // (CTAs of an SM)
constexpr int kParts = 4;
constexpr int kMaxTile = 64;            // rows of a CTA
constexpr int kRounds = 8;              // items of a group, at most
constexpr int kSamples = 256;

struct RowPlace {
    int64_t at;                         // element of head 0 in the caches, -1: none
    int64_t scale;                      // of its scale
    int64_t row;                        // of the dense tensors
};

// The place of the call's row r.  Rows of sequence i are cu[i] .. cu[i+1]-1; `sample` holds every
// `stride`-th of the batch + 1 offsets.
__device__ __forceinline__ RowPlace place_of(const RowsParams& p, const int32_t* sample, int stride, int samples, int r) {
    RowPlace none = {-1, 0, 0};
    int lo = 0, hi = samples - 1;       // the last sample at or before r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sample[mid] <= r) lo = mid; else hi = mid - 1;
    }
    lo *= stride;
    hi = min(lo + stride - 1, p.batch - 1);
    if (lo > hi) return none;           // the last offset itself
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ld(p.cu + mid) <= r) lo = mid; else hi = mid - 1;
    }
    const int s = ld(p.cu + lo), e = ld(p.cu + lo + 1), end = ld(p.cu + p.batch);
    if (r < s || r >= e) return none;
    const int64_t first = p.first ? ld(p.first + lo) : 0;
    // (reported once for a sequence, by its first row)
    const bool tell = r == s || r == 0;
    if (s < 0 || e > end || e > p.num_tokens) {
        if (tell) raise(p.status, GDN_FLAG_TOKEN_ROW);
        return none;
    }
    if (first < 0 || first + (e - s) > static_cast<int64_t>(p.pg.cols) * p.pg.page) {
        if (tell) raise(p.status, GDN_FLAG_SLOT_RANGE);
        return none;
    }
    int row = r;
    if (p.sti) {
        row = ld(p.sti + r);
        if (row < 0 || row >= p.num_tokens) {
            raise(p.status, GDN_FLAG_TOKEN_ROW);
            return none;
        }
    }
    const int32_t x = static_cast<int32_t>(first) + (r - s);
    const int32_t col = p.pg.page_of(x);
    const int64_t page = ld(p.pg.table + static_cast<int64_t>(lo) * p.pg.table_stride + col);
    if (page < 0) return none;
    if (page >= p.pg.num_pages) {
        raise(p.status, GDN_FLAG_SLOT_RANGE);
        return none;
    }
    const int64_t in = x - col * p.pg.page;
    return {page * p.pg.page_stride + in * p.pg.token_stride, page * p.pg.s_page + in * p.pg.s_token, row};
}

__device__ __forceinline__ float bits_f(uint32_t b) { return __uint_as_float(b); }

// An element's type in the cache: how 8 of a row are made from floats, and floats from them.
struct F32 {
    static constexpr int kBytes = 4;
    __device__ static void put(void* dst, const float (&x)[8]) {
        float4* d = static_cast<float4*>(dst);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};
struct Bf16 {
    static constexpr int kBytes = 2;
    using Raw = uint4;
    __device__ static void get(const Raw& raw, float (&x)[8]) {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = bits_f(w[e] << 16);
            x[2 * e + 1] = bits_f(w[e] & 0xffff0000u);
        }
    }
    __device__ static void put(void* dst, const float (&x)[8]) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
        *static_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(h);
    }
};
struct F16 {
    static constexpr int kBytes = 2;
    using Raw = uint4;
    __device__ static void get(const Raw& raw, float (&x)[8]) {
        const __half2* h = reinterpret_cast<const __half2*>(&raw);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(h[e]);
            x[2 * e] = f.x;
            x[2 * e + 1] = f.y;
        }
    }
    __device__ static void put(void* dst, const float (&x)[8]) {
        __half2 h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
        *static_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(h);
    }
};
constexpr float kLeastScale = 0x1p-100f;
struct E4m3 {
    static constexpr int kBytes = 1;
    using Raw = uint2;
    // the least power of two s >= 2^-100 with a <= 448 s, 448 = 1.75 x 2^8
    __device__ static float scale_of(float a) {
        const uint32_t b = __float_as_uint(a);
        int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = max(e, -100);
        return bits_f(static_cast<uint32_t>(e + 127) << 23);
    }
    __device__ static void put(void* dst, const float (&x)[8], float scale) {
        const float inv = bits_f((254u << 23) - __float_as_uint(scale));       // 1 / scale, exact
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h] * inv, x[4 * h + 1] * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h + 2] * inv, x[4 * h + 3] * inv), __NV_SATFINITE, __NV_E4M3);
            w[h] = lo | (hi << 16);
        }
        *static_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    }
    __device__ static void get(const Raw& raw, float (&x)[8]) {
        const uint32_t w[2] = {raw.x, raw.y};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[e / 2] >> (16 * (e & 1))), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            x[2 * e] = f.x;
            x[2 * e + 1] = f.y;
        }
    }
};
struct I8 {
    static constexpr int kBytes = 1;
    using Raw = uint2;
    __device__ static float scale_of(float a) {
        const uint32_t b = __float_as_uint(__fdiv_rn(a, 127.0f));
        return fmaxf(bits_f((b + 0xffffu) & 0xffff0000u), kLeastScale);
    }
    // x / scale through the reciprocal and one correction: scale and x have 8 significant bits, so a
    // quotient that is not halfway between two codes is at least 2^-17 of itself away from there, and one
    // that is comes out exactly
    __device__ static void put(void* dst, const float (&x)[8], float scale) {
        const float inv = __frcp_rn(scale);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float q = x[e] * inv;
            q = fmaf(fmaf(-q, scale, x[e]), inv, q);
            w[e / 4] |= (static_cast<uint32_t>(__float2int_rn(q)) & 0xffu) << (8 * (e & 3));
        }
        *static_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    }
    __device__ static void get(const Raw& raw, float (&x)[8]) {
        const uint32_t w[2] = {raw.x, raw.y};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(static_cast<int8_t>(w[e / 4] >> (8 * (e & 3))));
    }
};

template <typename C>
constexpr bool kQuantised = C::kBytes == 1;

template <int D>
struct Group {                          // of lanes that move a head's row
    static constexpr int kLanes = D == 192 ? 8 : D / 8 / kParts;       // (192: 6 of them work)
    static constexpr int kNum = kRThreads / kLanes;
};

template <typename C, typename Row, int D, bool kWrite>
__global__ void __launch_bounds__(kRThreads, kRCtas) gdn_kv_rows_kernel(const RowsParams p, const int tile) {
    constexpr int kLanes = Group<D>::kLanes, kGroups = Group<D>::kNum;
    constexpr int kApart = D / kParts;                  // a lane's pieces
    __shared__ int32_t sample[kSamples + 1];
    __shared__ RowPlace place[kMaxTile];
    const int tid = threadIdx.x;
    const int r0 = static_cast<int>(blockIdx.x) * tile;
    const int rows = min(tile, p.num_tokens - r0);
    const int lane = tid % kLanes, col = 8 * lane;
    const bool works = col < kApart;
    // The tile's items: head h of k (kv even) or v (odd) of its row kv / 2; a group takes every kGroups-th.
    const int dkv = kGroups / p.heads, dh = kGroups - dkv * p.heads;
    int kv = tid / kLanes / p.heads, h = tid / kLanes - kv * p.heads;
    const int rounds = (2 * rows * p.heads + kGroups - 1) / kGroups;
    dep_wait();

    using Raw = std::conditional_t<kWrite, uint4, typename C::Raw>;
    Raw raw[kParts];
    float scale = 0.f;
    auto load_row = [&](int64_t row) {
        const __nv_bfloat16* src = (kv & 1 ? p.v : p.k) + row * (kv & 1 ? p.v_stride : p.k_stride) + h * D + col;
#pragma unroll
        for (int c = 0; c < kParts; ++c) raw[c] = ld(reinterpret_cast<const Raw*>(src + c * kApart));
    };
    // a written row that is where its number says need not wait for its place
    const bool direct = kWrite && p.sti == nullptr;
    if constexpr (kWrite)
        if (direct && works && kv < 2 * rows) load_row(r0 + (kv >> 1));

    const int stride = (p.batch + 1 + kSamples - 1) / kSamples;
    const int samples = (p.batch + 1 + stride - 1) / stride;
    for (int k = tid; k < samples; k += kRThreads) sample[k] = ld(p.cu + static_cast<int64_t>(k) * stride);
    if (blockIdx.x == 0 && tid == 0 && ld(p.cu + p.batch) > p.num_tokens) raise(p.status, GDN_FLAG_TOKEN_ROW);
    __syncthreads();
    if (tid < rows) place[tid] = place_of(p, sample, stride, samples, r0 + tid);
    __syncthreads();
    dep_launch();

    for (int r = 0; r < rounds; ++r) {                  // (all threads alike: the maximum goes through shuffles)
        const bool is_v = kv & 1;
        RowPlace pl = {-1, 0, 0};
        if (kv < 2 * rows) pl = place[kv >> 1];
        const bool live = pl.at >= 0 && works;
        const int64_t at = (pl.at + h * p.pg.head_stride + col) * C::kBytes, sat = pl.scale + h * p.pg.s_head;
        if constexpr (kWrite) {
            if (live && !(direct && r == 0)) load_row(pl.row);
            char* dst = static_cast<char*>(is_v ? p.v_cache : p.k_cache) + at;
            float x[kParts][8];
#pragma unroll
            for (int c = 0; c < kParts; ++c) Bf16::get(live ? raw[c] : make_uint4(0, 0, 0, 0), x[c]);
            if constexpr (kQuantised<C>) {
                uint32_t big = 0;                       // the largest pattern: infinities and NaN are above the finite ones
#pragma unroll
                for (int c = 0; c < kParts; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e) big = max(big, __float_as_uint(x[c][e]) & 0x7fffffffu);
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(kFull, big, o, kLanes));
                const bool fine = big < 0x7f800000u;
                const float s = fine ? C::scale_of(bits_f(big)) : bits_f(0x7fc00000u);
                if (live) {
#pragma unroll
                    for (int c = 0; c < kParts; ++c) {
                        if (fine) C::put(dst + c * kApart, x[c], s);
                        else *reinterpret_cast<uint2*>(dst + c * kApart) = make_uint2(0, 0);
                    }
                    if (lane == 0) (is_v ? p.v_scale : p.k_scale)[sat] = s;
                }
            } else if (live) {
#pragma unroll
                for (int c = 0; c < kParts; ++c) C::put(dst + c * kApart * C::kBytes, x[c]);
            }
        } else if (live) {
            const char* src = static_cast<const char*>(is_v ? p.v_cache : p.k_cache) + at;
#pragma unroll
            for (int c = 0; c < kParts; ++c) raw[c] = ld(reinterpret_cast<const Raw*>(src + c * kApart * C::kBytes));
            if constexpr (kQuantised<C>) scale = ld((is_v ? p.v_scale : p.k_scale) + sat);
            char* dst = static_cast<char*>(is_v ? p.v_rows : p.k_rows) + (pl.row * (is_v ? p.v_stride : p.k_stride) + h * D + col) * Row::kBytes;
#pragma unroll
            for (int c = 0; c < kParts; ++c) {
                float x[8];
                C::get(raw[c], x);
                if constexpr (kQuantised<C>) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= scale;
                }
                Row::put(dst + c * kApart * Row::kBytes, x);
            }
        }
        kv += dkv;
        h += dh;
        if (h >= p.heads) {
            h -= p.heads;
            ++kv;
        }
    }
}

template <typename C, typename Row, int D, bool kWrite>
cudaError_t launch_rows(const RowsParams& p, cudaStream_t stream) {
    const int sms = sm_count() ? sm_count() : 148;
    // rows a CTA: few rows go to as many CTAs as run at once, more in whole waves of them
    const int64_t most = std::min(kMaxTile, std::max(1, kRounds * Group<D>::kNum / (2 * p.heads)));
    const int64_t wave = static_cast<int64_t>(sms) * kRCtas;
    const int64_t waves = (p.num_tokens + wave * most - 1) / (wave * most);
    const int tile = static_cast<int>((p.num_tokens + wave * waves - 1) / (wave * waves));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.num_tokens + tile - 1) / tile), 1, 1);
    cfg.blockDim = dim3(kRThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gdn_kv_rows_kernel<C, Row, D, kWrite>, p, tile);
}

template <typename C, typename Row, bool kWrite>
cudaError_t rows_by_dim(const RowsParams& p, int D, cudaStream_t s) {
    return D == 64    ? launch_rows<C, Row, 64, kWrite>(p, s)
           : D == 128 ? launch_rows<C, Row, 128, kWrite>(p, s)
           : D == 192 ? launch_rows<C, Row, 192, kWrite>(p, s)
                      : launch_rows<C, Row, 256, kWrite>(p, s);
}

template <typename C>
cudaError_t read_by_row(const RowsParams& p, int D, gdn_dtype row, cudaStream_t s) {
    return row == GDN_F32    ? rows_by_dim<C, F32, false>(p, D, s)
           : row == GDN_BF16 ? rows_by_dim<C, Bf16, false>(p, D, s)
                             : rows_by_dim<C, F16, false>(p, D, s);
}

bool is_cache_type(gdn_dtype t) { return t == GDN_BF16 || t == GDN_F16 || t == GDN_E4M3 || t == GDN_I8; }
bool is_8bit(gdn_dtype t) { return t == GDN_E4M3 || t == GDN_I8; }

// sizes that the three calls share
gdn_status check_dims(const gdn_kv_dims* d, gdn_dtype type) {
    if (d == nullptr) return GDN_ERR_NULL_ARG;
    if (d->batch < 0 || d->num_tokens < 0 || d->batch > kMaxScanned || d->num_tokens > kMaxRows || d->H_kv < 1 ||
        d->H_kv > 4096 || d->D < 1 || d->page_size < 1 || d->page_size > kMaxRows || d->table_cols < 1 || d->num_pages < 1 || d->reserved != 0 ||
        d->page_stride < 0 || d->token_stride < 0 || d->head_stride < 0 || d->scale_page_stride < 0 ||
        d->scale_token_stride < 0 || d->scale_head_stride < 0 || d->table_stride < 0 || d->q_stride < 0 || d->k_stride < 0 ||
        d->v_stride < 0 || d->z_stride < 0 || d->out_stride < 0)
        return GDN_ERR_BAD_SHAPE;
    // (a sequence's positions stay in 31 bits, with a tile to spare)
    if (static_cast<int64_t>(d->table_cols) * d->page_size > 0x7fff0000LL) return GDN_ERR_BAD_SHAPE;
    if ((d->D != 64 && d->D != 128 && d->D != 192 && d->D != 256) || !is_cache_type(type)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// the cache's side of a call; strides come out resolved
gdn_status make_paging(Paging& g, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                       const int32_t* table, const gdn_kv_dims* d, gdn_dtype type) {
    if (!k_cache || !v_cache || !table || (is_8bit(type) && (!k_scale || !v_scale))) return GDN_ERR_NULL_ARG;
    g.table = table;
    g.num_pages = d->num_pages;
    g.head_stride = d->head_stride ? d->head_stride : d->D;
    g.token_stride = d->token_stride ? d->token_stride : static_cast<int64_t>(d->H_kv) * d->D;
    g.page_stride = d->page_stride ? d->page_stride : static_cast<int64_t>(d->page_size) * d->H_kv * d->D;
    g.s_head = d->scale_head_stride ? d->scale_head_stride : 1;
    g.s_token = d->scale_token_stride ? d->scale_token_stride : d->H_kv;
    g.s_page = d->scale_page_stride ? d->scale_page_stride : static_cast<int64_t>(d->page_size) * d->H_kv;
    g.table_stride = d->table_stride ? d->table_stride : d->table_cols;
    g.cols = d->table_cols;
    g.divide_by(d->page_size);
    const int64_t unit = is_8bit(type) ? 16 : 8;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(table, 4) || g.head_stride % unit != 0 ||
        g.token_stride % unit != 0 || g.page_stride % unit != 0 ||
        (is_8bit(type) && (!aligned(k_scale, 4) || !aligned(v_scale, 4))))
        return GDN_ERR_MISALIGNED;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_kv_write(const void* k, const void* v, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                        const int32_t* page_table, const int32_t* kv_lens, const int32_t* cu_seqlens,
                        const int32_t* spec_token_indx, const gdn_kv_dims* dims, gdn_dtype cache_type,
                        int32_t* status_word, gdn_stream_t stream) {
    const gdn_status ds = check_dims(dims, cache_type);
    if (ds != GDN_OK) return ds;
    if (dims->batch == 0 || dims->num_tokens == 0) return GDN_OK;
    if (!k || !v || !kv_lens || !cu_seqlens) return GDN_ERR_NULL_ARG;
    RowsParams p = {};
    const gdn_status ps = make_paging(p.pg, k_cache, v_cache, k_scale, v_scale, page_table, dims, cache_type);
    if (ps != GDN_OK) return ps;
    const int64_t dense = static_cast<int64_t>(dims->H_kv) * dims->D;
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.first = kv_lens;
    p.cu = cu_seqlens;
    p.sti = spec_token_indx;
    p.status = status_word;
    p.k_stride = dims->k_stride ? dims->k_stride : dense;
    p.v_stride = dims->v_stride ? dims->v_stride : dense;
    p.batch = dims->batch;
    p.num_tokens = dims->num_tokens;
    p.heads = dims->H_kv;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kv_lens, 4) || !aligned(cu_seqlens, 4) || !aligned(spec_token_indx, 4) ||
        !aligned(status_word, 4) || p.k_stride % 8 != 0 || p.v_stride % 8 != 0)
        return GDN_ERR_MISALIGNED;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = cache_type == GDN_BF16   ? rows_by_dim<Bf16, Bf16, true>(p, dims->D, s)
                            : cache_type == GDN_F16  ? rows_by_dim<F16, Bf16, true>(p, dims->D, s)
                            : cache_type == GDN_E4M3 ? rows_by_dim<E4m3, Bf16, true>(p, dims->D, s)
                                                     : rows_by_dim<I8, Bf16, true>(p, dims->D, s);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_kv_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                       const int32_t* page_table, const int32_t* kv_begin, const int32_t* cu_seqlens, void* k, void* v,
                       const gdn_kv_dims* dims, gdn_dtype cache_type, gdn_dtype row_type, int32_t* status_word,
                       gdn_stream_t stream) {
    const gdn_status ds = check_dims(dims, cache_type);
    if (ds != GDN_OK) return ds;
    if (!is_dtype(row_type)) return GDN_ERR_UNSUPPORTED;
    if (dims->batch == 0 || dims->num_tokens == 0) return GDN_OK;
    if (!k || !v || !cu_seqlens) return GDN_ERR_NULL_ARG;
    RowsParams p = {};
    const gdn_status ps = make_paging(p.pg, k_cache, v_cache, k_scale, v_scale, page_table, dims, cache_type);
    if (ps != GDN_OK) return ps;
    const int64_t dense = static_cast<int64_t>(dims->H_kv) * dims->D;
    p.k_rows = k;
    p.v_rows = v;
    p.k_cache = const_cast<void*>(k_cache);          // (not written)
    p.v_cache = const_cast<void*>(v_cache);
    p.k_scale = const_cast<float*>(k_scale);
    p.v_scale = const_cast<float*>(v_scale);
    p.first = kv_begin;
    p.cu = cu_seqlens;
    p.status = status_word;
    p.k_stride = dims->k_stride ? dims->k_stride : dense;
    p.v_stride = dims->v_stride ? dims->v_stride : dense;
    p.batch = dims->batch;
    p.num_tokens = dims->num_tokens;
    p.heads = dims->H_kv;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kv_begin, 4) || !aligned(cu_seqlens, 4) || !aligned(status_word, 4) ||
        p.k_stride % 8 != 0 || p.v_stride % 8 != 0)
        return GDN_ERR_MISALIGNED;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = cache_type == GDN_BF16   ? read_by_row<Bf16>(p, dims->D, row_type, s)
                            : cache_type == GDN_F16  ? read_by_row<F16>(p, dims->D, row_type, s)
                            : cache_type == GDN_E4M3 ? read_by_row<E4m3>(p, dims->D, row_type, s)
                                                     : read_by_row<I8>(p, dims->D, row_type, s);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

namespace {

// sizes of the attention
gdn_status check_attn(const gdn_kv_dims* d, gdn_dtype type) {
    const gdn_status ds = check_dims(d, type);
    if (ds != GDN_OK) return ds;
    if (d->H_q < 1 || d->H_q % d->H_kv != 0 || d->H_q > 4096 || d->max_T < 1 || d->max_T > 8 || d->window < 0)
        return GDN_ERR_BAD_SHAPE;
    // (the line of all units' key blocks, times its CTAs, stays in 63 bits)
    const int64_t blocks = (static_cast<int64_t>(d->table_cols) * d->page_size + 127) / 64;
    if (d->batch > 0 && blocks > (1ll << 52) / d->batch / (static_cast<int64_t>(d->H_q) * d->max_T)) return GDN_ERR_BAD_SHAPE;
    return GDN_OK;
}

AttnParams attn_sizes(const gdn_kv_dims* d) {
    AttnParams p = {};
    p.batch = d->batch;
    p.num_tokens = d->num_tokens;
    p.heads = d->H_kv;
    p.ratio = d->H_q / d->H_kv;
    p.max_T = d->max_T;
    p.window = d->window;
    p.pg.page = d->page_size;
    p.pg.num_pages = d->num_pages;
    return p;
}

}  // namespace

extern "C" {

int64_t gdn_attn_decode_workspace(const gdn_kv_dims* dims, gdn_dtype cache_type) {
    if (check_attn(dims, cache_type) != GDN_OK) return -1;
    if (dims->batch == 0 || dims->num_tokens == 0) return 0;
    return attn_workspace(attn_sizes(dims), dims->D, cache_type);
}

gdn_status gdn_attn_decode(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, const int32_t* page_table, const int32_t* kv_lens,
                           const int32_t* cu_seqlens, const int32_t* spec_token_indx, const void* z, void* out,
                           void* workspace, int64_t workspace_bytes, const gdn_kv_dims* dims, float scale,
                           gdn_dtype cache_type, int32_t* status_word, gdn_stream_t stream) {
    const gdn_status ds = check_attn(dims, cache_type);
    if (ds != GDN_OK) return ds;
    if (!std::isfinite(scale)) return GDN_ERR_BAD_SHAPE;
    if (dims->batch == 0 || dims->num_tokens == 0) return GDN_OK;
    if (!q || !kv_lens || !cu_seqlens || !out || !workspace) return GDN_ERR_NULL_ARG;
    AttnParams p = attn_sizes(dims);
    const gdn_status ps = make_paging(p.pg, k_cache, v_cache, k_scale, v_scale, page_table, dims, cache_type);
    if (ps != GDN_OK) return ps;
    if (workspace_bytes < attn_workspace(p, dims->D, cache_type)) return GDN_ERR_BAD_SHAPE;
    const int64_t dense = static_cast<int64_t>(dims->H_q) * dims->D;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.z = static_cast<const __nv_bfloat16*>(z);
    p.k = k_cache;
    p.v = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.kv_lens = kv_lens;
    p.cu = cu_seqlens;
    p.sti = spec_token_indx;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.status = status_word;
    p.q_stride = dims->q_stride ? dims->q_stride : dense;
    p.z_stride = dims->z_stride ? dims->z_stride : dense;
    p.out_stride = dims->out_stride ? dims->out_stride : dense;
    p.scale = scale * 1.4426950408889634f;
    if (!aligned(q, 16) || !aligned(z, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(kv_lens, 4) ||
        !aligned(cu_seqlens, 4) || !aligned(spec_token_indx, 4) || !aligned(status_word, 4) || p.q_stride % 8 != 0 ||
        p.z_stride % 8 != 0 || p.out_stride % 8 != 0)
        return GDN_ERR_MISALIGNED;
    const cudaError_t err = launch_attn(p, dims->D, cache_type, workspace, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
