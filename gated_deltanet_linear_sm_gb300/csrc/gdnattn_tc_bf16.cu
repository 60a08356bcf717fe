// libgdnspec: the tcgen05 attention over a bf16 cache (gdnattn_tc.cuh).
#include "gdnattn_tc.cuh"

namespace gdn_kv {

int64_t attn_tc_workspace(int D) {
    const int64_t grid = grid_of();
    return grid * kMetaInts * 4 + 2 * grid * kRowsT * (D + 2) * 4;
}

cudaError_t launch_attn_tc_bf16(const AttnParams& p, int D, void* workspace, cudaStream_t stream) {
    return launch_kind<kBf16>(p, D, workspace, stream);
}

}  // namespace gdn_kv
