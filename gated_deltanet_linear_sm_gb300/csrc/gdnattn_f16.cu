// libgdnspec: the attention over a fp16 cache (gdnattn_warp.cuh, gdnattn_tc.cuh).
#include "gdnattn_tc.cuh"
#include "gdnattn_warp.cuh"

namespace gdn_kv {

int64_t attn_workspace_f16(int rows, int D) { return gdn_attn_warp::workspace_kind<gdn_attn_warp::kF16>(rows, D); }

cudaError_t launch_attn_f16(const AttnParams& p, int rows, int D, void* workspace, cudaStream_t stream) {
    return gdn_attn_warp::launch_kind<gdn_attn_warp::kF16>(p, rows, D, workspace, stream);
}

cudaError_t launch_attn_tc_f16(const AttnParams& p, int D, void* workspace, cudaStream_t stream) {
    return gdn_attn_tc::launch_kind<gdn_attn_tc::kF16>(p, D, workspace, stream);
}

}  // namespace gdn_kv
