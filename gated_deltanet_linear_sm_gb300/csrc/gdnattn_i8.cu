// libgdnspec: the attention over an int8 cache (gdnattn_warp.cuh).
#include "gdnattn_warp.cuh"

namespace gdn_kv {

int64_t attn_workspace_i8(int rows, int D) { return gdn_attn_warp::workspace_kind<gdn_attn_warp::kI8>(rows, D); }

cudaError_t launch_attn_i8(const AttnParams& p, int rows, int D, void* workspace, cudaStream_t stream) {
    return gdn_attn_warp::launch_kind<gdn_attn_warp::kI8>(p, rows, D, workspace, stream);
}

}  // namespace gdn_kv
