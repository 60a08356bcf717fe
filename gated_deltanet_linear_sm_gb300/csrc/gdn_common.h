// Internal to libgdnspec: host and device helpers that the operators around
// the step share (gdnverify.cu, gdnssm.cu, gdnssm_prefill.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gdnspec.h"

namespace gdn_common {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
constexpr int32_t kMaxRows = 1 << 30;            // of a call: a row number plus a tile's rows stays in 32 bits
// Sequences of a call whose every CTA reads the offsets of those before its own (the tables, the prompt
// convolution): the reads grow with batch times CTAs, to minutes for the offsets that would still fit.
constexpr int32_t kMaxScanned = 1 << 20;
inline bool is_dtype(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16 || t == GDN_F16; }

// SMs of the current device (asked once per device; 0 if that fails)
inline int sm_count() {
    static int sms[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = __atomic_load_n(&sms[dev], __ATOMIC_RELAXED);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        __atomic_store_n(&sms[dev], n, __ATOMIC_RELAXED);
    }
    return n;
}

constexpr unsigned kFull = 0xffffffffu;

// Programmatic dependent launch.  A kernel launched with it may start while its
// predecessor on the stream still runs: it waits (dep_wait) until that has
// completed before it touches memory, and after that wait it may let its own
// successor start (dep_launch).  The kernels here that write what the steps read
// through __ldg (gdn_verify_drafts and gdn_step_tables the tables, gdn_conv_prefill
// conv slots) do not call dep_launch, so their successor starts when they have
// completed: it may then read those before any wait of its own.
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A plain load: unlike __ldg (which promises that nothing writes the memory
// while the kernel runs, early starts included) it stays behind dep_wait.
template <typename T>
__device__ __forceinline__ T ld(const T* p) {
    return *p;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

__device__ __forceinline__ void raise(int32_t* status, int flag) {
    if (status != nullptr) atomicOr(status, flag);
}

// log(1 + e^x) = max(x, 0) + log(1 + u), u = e^-|x| <= 1, and log(1 + u) = 2 atanh(s)
// = 2 s (1 + s^2 / 3 + s^4 / 5 + ...), s = u / (2 + u) <= 1/3: nine terms leave less
// than 2^-30 of the value.
__device__ __forceinline__ float softplus(float x) {
    const float u = expf(-fabsf(x));
    const float s = __fdividef(u, 2.0f + u), q = s * s;
    float p = 1.0f / 17.0f;
    p = fmaf(p, q, 1.0f / 15.0f);
    p = fmaf(p, q, 1.0f / 13.0f);
    p = fmaf(p, q, 1.0f / 11.0f);
    p = fmaf(p, q, 1.0f / 9.0f);
    p = fmaf(p, q, 1.0f / 7.0f);
    p = fmaf(p, q, 1.0f / 5.0f);
    p = fmaf(p, q, 1.0f / 3.0f);
    p = fmaf(p, q, 1.0f);
    return fmaxf(x, 0.0f) + 2.0f * s * p;
}

// silu(z) = z sigmoid(z); for very negative z the denominator overflows and
// the fast division returns zero
__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

}  // namespace gdn_common
