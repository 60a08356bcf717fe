// libgdnspec: the state-space layer over prompts (gdn_ssm_prefill, whose C
// entry point and argument checks are in gdnssm.cu).
#include "gdnssm.h"
#include "gdnssm_recur.cuh"

using namespace gdn_common;
using namespace gdn_ssm;

namespace {

// The token recurrence, 8 tokens a round: one CTA of 128 threads per
// (sequence, head, 64 columns), the state block in FP32 registers.
template <typename StateT, int N>
__global__ void __launch_bounds__(kRThreads, 4) gdn_ssm_prefill_kernel(const Params p) {
    constexpr int R = N / 16;
    __shared__ Round<N> s;
    const int tid = threadIdx.x, cg = tid & 7, rg = tid >> 3;
    const int pb = static_cast<int>(blockIdx.x % p.blocks);
    const int unit = static_cast<int>(blockIdx.x / p.blocks);
    const int i = unit / p.H, h = unit - i * p.H;
    const int g = h / p.group;
    const int bos = __ldg(p.cu + i);
    const int eos = __ldg(p.cu + i + 1);
    const long long rs = __ldg(p.read_slots + i), ws = __ldg(p.write_slots + i);
    if (eos <= bos) return;
    int flag = 0;
    if (bos < 0 || eos > p.num_tokens) flag = GDN_FLAG_TOKEN_ROW;
    else if (rs >= p.num_slots || ws >= p.num_slots) flag = GDN_FLAG_SLOT_RANGE;
    if (flag) {
        if (tid == 0) raise(p.status, flag);
        return;
    }
    const int L = eos - bos;
    const int64_t tile = static_cast<int64_t>(N) * p.P;
    const int64_t at = h * tile + static_cast<int64_t>(rg * R) * p.P + pb * kPB;
    u64 S[R][4] = {};
    if (rs >= 0) {
        const StateT* src = static_cast<const StateT*>(p.pool) + rs * p.H * tile + at;
#pragma unroll
        for (int j = 0; j < R; ++j) Row8<StateT>::load(src + static_cast<int64_t>(j) * p.P, cg, S[j]);
    }
    const int to = tid >> 4, qo = tid & 15;
    const int col = h * p.P + pb * kPB;
    const float rate = -expf(__ldg(p.A_log + h)), bias = __bfloat162float(p.dt_bias[h]);
    const float D = p.D ? __ldg(p.D + h) : 0.f;
    for (int c0 = 0; c0 < L; c0 += kMaxT) {
        const int n = min(kMaxT, L - c0);
        const int64_t r0 = bos + c0;
        if (tid < n) {
            const float d = softplus(__bfloat162float(p.dt[(r0 + tid) * p.dt_stride + h]) + bias);
            s.step[tid] = d;
            s.decay[tid] = expf(rate * d);
        }
        uint2 zraw = make_uint2(0, 0);
        if (to < n) {
            const int64_t r = r0 + to;
            float f[4];
            unpack4(__ldg(reinterpret_cast<const uint2*>(p.x + r * p.x_stride + col + 4 * qo)), f);
            *reinterpret_cast<float4*>(&s.x[to][4 * qo]) = make_float4(f[0], f[1], f[2], f[3]);
            if (p.z) zraw = __ldg(reinterpret_cast<const uint2*>(p.z + r * p.z_stride + col + 4 * qo));
            for (int q = qo; q < N / 4; q += 16) {
                unpack4(__ldg(reinterpret_cast<const uint2*>(p.B + r * p.b_stride + g * N + 4 * q)), f);
                *reinterpret_cast<float4*>(&s.B[to][4 * q]) = make_float4(f[0], f[1], f[2], f[3]);
                unpack4(__ldg(reinterpret_cast<const uint2*>(p.C + r * p.c_stride + g * N + 4 * q)), f);
                *reinterpret_cast<float4*>(&s.C[to][4 * q]) = make_float4(f[0], f[1], f[2], f[3]);
            }
        }
        __syncthreads();
        for (int t = 0; t < n; ++t) token<StateT, N>(S, s, t);
        __syncthreads();
        if (to < n) write_out(s, to, qo, D, p.z != nullptr, zraw, p.out + (r0 + to) * p.out_stride + col + 4 * qo);
        __syncthreads();
    }
    if (ws >= 0) {
        StateT* dst = static_cast<StateT*>(p.pool) + ws * p.H * tile + at;
#pragma unroll
        for (int j = 0; j < R; ++j) Row8<StateT>::store(dst + static_cast<int64_t>(j) * p.P, cg, S[j]);
    }
}

template <typename StateT>
cudaError_t launch(const Params& p, int N, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(p.batch) * p.H * p.blocks), 1, 1);
    cfg.blockDim = dim3(kRThreads, 1, 1);
    cfg.stream = stream;
    return N == 64 ? cudaLaunchKernelEx(&cfg, gdn_ssm_prefill_kernel<StateT, 64>, p)
                   : cudaLaunchKernelEx(&cfg, gdn_ssm_prefill_kernel<StateT, 128>, p);
}

}  // namespace

namespace gdn_ssm {

int64_t prefill_workspace(int, int, int, int) { return 0; }

cudaError_t launch_prefill(const Params& p, int N, gdn_dtype state_dtype, void*, cudaStream_t stream) {
    return state_dtype == GDN_F32    ? launch<float>(p, N, stream)
           : state_dtype == GDN_BF16 ? launch<__nv_bfloat16>(p, N, stream)
                                     : launch<__half>(p, N, stream);
}

}  // namespace gdn_ssm
