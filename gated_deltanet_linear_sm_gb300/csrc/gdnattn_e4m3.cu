// libgdnspec: the attention over an e4m3 cache (gdnattn_warp.cuh, gdnattn_tc.cuh).
#include "gdnattn_tc.cuh"
#include "gdnattn_warp.cuh"

namespace gdn_kv {

int64_t attn_workspace_e4m3(int rows, int D) { return gdn_attn_warp::workspace_kind<gdn_attn_warp::kE4m3>(rows, D); }

cudaError_t launch_attn_e4m3(const AttnParams& p, int rows, int D, void* workspace, cudaStream_t stream) {
    return gdn_attn_warp::launch_kind<gdn_attn_warp::kE4m3>(p, rows, D, workspace, stream);
}

cudaError_t launch_attn_tc_e4m3(const AttnParams& p, int D, void* workspace, cudaStream_t stream) {
    return gdn_attn_tc::launch_kind<gdn_attn_tc::kE4m3>(p, D, workspace, stream);
}

}  // namespace gdn_kv
