// Internal to libgdnspec: the kernel parameters of the state-space layer,
// shared by its step (gdnssm.cu, which also holds the C entry points and their
// checks) and its scan over prompts (gdnssm_prefill.cu).
#pragma once

#include "gdn_common.h"

namespace gdn_ssm {

// Filled on the host from one validated call; passed by value to the kernels.
struct Params {
    const __nv_bfloat16* x;          // prefill: [row][H * P]; step: the projection rows [row][conv_dim]
    const __nv_bfloat16* B;
    const __nv_bfloat16* C;
    const __nv_bfloat16* dt;
    const __nv_bfloat16* z;
    const float* A_log;
    const __nv_bfloat16* dt_bias;
    const float* D;
    void* pool;
    const int32_t* read_slots;
    const int32_t* write_slots;
    const int32_t* cu;
    __nv_bfloat16* out;
    int32_t* status;
    int64_t x_stride, b_stride, c_stride, dt_stride, z_stride, out_stride;
    int64_t num_slots;
    int32_t batch, num_tokens, H, G, P, group, blocks;   // blocks: 64-column blocks of a head, P / 64
    // the step
    const int32_t* idx;
    const int32_t* num_acc;
    const int32_t* sti;
    const __nv_bfloat16* conv_w;     // [conv_dim][width]
    const __nv_bfloat16* conv_b;     // [conv_dim] or null
    __nv_bfloat16* conv_pool;        // [num_conv_slots][state_len][conv_dim]
    const int32_t* conv_in;
    const int32_t* conv_out;
    int64_t num_conv_slots;
    int32_t stride, max_T, conv_dim, conv_width, conv_state_len;
};

constexpr int kPB = 64;              // columns of the head dim that one CTA works on

// Launch the scan over prompts (gdnssm_prefill.cu).
cudaError_t launch_prefill(const Params& p, int N, gdn_dtype state_dtype, void* workspace, cudaStream_t stream);
// Its workspace in bytes on the current device.
int64_t prefill_workspace(int batch, int num_tokens, int units_per_seq, int N);

}  // namespace gdn_ssm
