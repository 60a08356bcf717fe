// libgdnspec: the attention over a bf16 cache (gdnattn_warp.cuh, gdnattn_tc.cuh).
#include "gdnattn_tc.cuh"
#include "gdnattn_warp.cuh"

namespace gdn_kv {

int64_t attn_workspace_bf16(int rows, int D) { return gdn_attn_warp::workspace_kind<gdn_attn_warp::kBf16>(rows, D); }

cudaError_t launch_attn_bf16(const AttnParams& p, int rows, int D, void* workspace, cudaStream_t stream) {
    return gdn_attn_warp::launch_kind<gdn_attn_warp::kBf16>(p, rows, D, workspace, stream);
}

cudaError_t launch_attn_tc_bf16(const AttnParams& p, int D, void* workspace, cudaStream_t stream) {
    return gdn_attn_tc::launch_kind<gdn_attn_tc::kBf16>(p, D, workspace, stream);
}

int64_t attn_tc_workspace(int D) { return gdn_attn_tc::workspace_of(D); }

}  // namespace gdn_kv
