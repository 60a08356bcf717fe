// Internal to libgdnspec: one token of the state-space recurrence on a
// N x 64 block of the state held in the registers of 128 threads.
//
//     S <- a S + B (d x)^T,   y = S^T C
//
// Thread (row group rg = tid / 8, column group cg = tid % 8) holds rows rg R ..
// rg R + R - 1 (R = N / 16) and 8 columns, as two quads: columns 8 cg .. 8 cg + 7
// of a 16-bit state, 4 cg .. and 32 + 4 cg .. of an FP32 one, so that 8 lanes
// move one whole 128-byte line in either type.  The arithmetic runs on pairs
// of columns (fma.rn.f32x2, each half rounding as fmaf would).
#pragma once

#include "gdn_common.h"
#include "gdn_pairs.h"

namespace gdn_ssm {

using namespace gdn_common;

__device__ __forceinline__ void unpack4(uint2 raw, float (&x)[4]) {
    const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.x));
    const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.y));
    x[0] = lo.x;
    x[1] = lo.y;
    x[2] = hi.x;
    x[3] = hi.y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^x and 1 / x as single instructions (results and inputs below 2^-126 become 0)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;
// silu(z) for a pair: z / (1 + 2^(-z log2 e))
__device__ __forceinline__ u64 silu2(u64 z) {
    const u64 t = fmul2(z, dup2(-kLog2e));
    const u64 den = add2(pk2(ex2(lo2(t)), ex2(hi2(t))), dup2(1.0f));
    return fmul2(z, pk2(rcp(lo2(den)), rcp(hi2(den))));
}

// first column of quad e (0 or 1) of column group cg
template <typename StateT>
__device__ __forceinline__ constexpr int quad_col(int cg, int e) {
    return sizeof(StateT) == 4 ? 32 * e + 4 * cg : 8 * cg + 4 * e;
}

// 8 state elements of one row (streaming: a slot is read once and written once a step)
template <typename StateT>
struct Row8;

template <>
struct Row8<float> {
    static __device__ __forceinline__ void load(const float* row, int cg, u64 (&s)[4]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(row + quad_col<float>(cg, e)));
            s[2 * e] = pk2(v.x, v.y);
            s[2 * e + 1] = pk2(v.z, v.w);
        }
    }
    static __device__ __forceinline__ void store(float* row, int cg, const u64 (&s)[4]) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
            __stcs(reinterpret_cast<float4*>(row + quad_col<float>(cg, e)),
                   make_float4(lo2(s[2 * e]), hi2(s[2 * e]), lo2(s[2 * e + 1]), hi2(s[2 * e + 1])));
    }
};

template <>
struct Row8<__nv_bfloat16> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* row, int cg, u64 (&s)[4]) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(row + 8 * cg));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]));
            s[e] = pk2(f.x, f.y);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* row, int cg, const u64 (&s)[4]) {
        __stcs(reinterpret_cast<uint4*>(row + 8 * cg),
               make_uint4(pack2(lo2(s[0]), hi2(s[0])), pack2(lo2(s[1]), hi2(s[1])), pack2(lo2(s[2]), hi2(s[2])),
                          pack2(lo2(s[3]), hi2(s[3]))));
    }
};

template <>
struct Row8<__half> {
    static __device__ __forceinline__ void load(const __half* row, int cg, u64 (&s)[4]) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(row + 8 * cg));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
            s[e] = pk2(f.x, f.y);
        }
    }
    static __device__ __forceinline__ uint32_t pack(u64 v) {
        const __half2 h = __floats2half2_rn(lo2(v), hi2(v));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ void store(__half* row, int cg, const u64 (&s)[4]) {
        __stcs(reinterpret_cast<uint4*>(row + 8 * cg), make_uint4(pack(s[0]), pack(s[1]), pack(s[2]), pack(s[3])));
    }
};

constexpr int kRThreads = 128;
constexpr int kMaxT = 8;             // tokens of a round

// What the token loop reads and writes in shared memory: the rows of up to 8
// tokens in FP32, their decays and step sizes, and each warp's part of y.
template <int N>
struct alignas(16) Round {
    float x[kMaxT][64];
    float B[kMaxT][N];
    float C[kMaxT][N];
    float y[kMaxT][4][64];
    float decay[kMaxT], step[kMaxT];
    int row[kMaxT];
    int slot[kMaxT];     // the step: slot that takes the state after the token
};

// Token t: the update of this thread's rows, and the warp's part of y.
template <typename StateT, int N>
__device__ __forceinline__ void token(u64 (&S)[N / 16][4], Round<N>& s, int t) {
    constexpr int R = N / 16;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cg = tid & 7, rg = tid >> 3;
    const float a = s.decay[t], d = s.step[t];
    const u64 a2 = pk2(a, a);
    u64 xs[4], y[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float4 v = *reinterpret_cast<const float4*>(&s.x[t][quad_col<StateT>(cg, e)]);
        xs[2 * e] = pk2(d * v.x, d * v.y);
        xs[2 * e + 1] = pk2(d * v.z, d * v.w);
    }
    alignas(16) float b[R], c[R];
#pragma unroll
    for (int j = 0; j < R; j += 4) {
        *reinterpret_cast<float4*>(b + j) = *reinterpret_cast<const float4*>(&s.B[t][rg * R + j]);
        *reinterpret_cast<float4*>(c + j) = *reinterpret_cast<const float4*>(&s.C[t][rg * R + j]);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const u64 b2 = pk2(b[j], b[j]), c2 = pk2(c[j], c[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            S[j][k] = ffma2(b2, xs[k], fmul2(a2, S[j][k]));
            y[k] = ffma2(c2, S[j][k], y[k]);
        }
    }
    // over the warp's four row groups: halve the columns a lane carries at each exchange
    const bool up = (lane & 16) != 0, right = (lane & 8) != 0;
    float v[4], w[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const u64 mine = up ? y[2 + k] : y[k], other = up ? y[k] : y[2 + k];
        v[2 * k] = lo2(mine) + __shfl_xor_sync(kFull, lo2(other), 16);
        v[2 * k + 1] = hi2(mine) + __shfl_xor_sync(kFull, hi2(other), 16);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) w[k] = (right ? v[2 + k] : v[k]) + __shfl_xor_sync(kFull, right ? v[k] : v[2 + k], 8);
    *reinterpret_cast<float2*>(&s.y[t][warp][quad_col<StateT>(cg, up ? 1 : 0) + (right ? 2 : 0)]) =
        make_float2(w[0], w[1]);
}

// out of token t, columns 4 q .. 4 q + 3: (y + D x) silu(z), rounded once
template <int N>
__device__ __forceinline__ void write_out(const Round<N>& s, int t, int q, float D, bool gated, uint2 zraw,
                                          __nv_bfloat16* dst) {
    float4 y = *reinterpret_cast<const float4*>(&s.y[t][0][4 * q]);
#pragma unroll
    for (int w = 1; w < 4; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(&s.y[t][w][4 * q]);
        y.x += v.x;
        y.y += v.y;
        y.z += v.z;
        y.w += v.w;
    }
    const float4 x = *reinterpret_cast<const float4*>(&s.x[t][4 * q]);
    float o[4] = {fmaf(D, x.x, y.x), fmaf(D, x.y, y.y), fmaf(D, x.z, y.z), fmaf(D, x.w, y.w)};
    if (gated) {
        float zz[4];
        unpack4(zraw, zz);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= silu(zz[e]);
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2(o[0], o[1]), pack2(o[2], o[3]));
}

}  // namespace gdn_ssm
