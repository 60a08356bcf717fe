// libgdnspec: the tcgen05 attention over a e4m3 cache (gdnattn_tc.cuh).
#include "gdnattn_tc.cuh"

namespace gdn_kv {

cudaError_t launch_attn_tc_e4m3(const AttnParams& p, int D, void* workspace, cudaStream_t stream) {
    return launch_kind<kE4m3>(p, D, workspace, stream);
}

}  // namespace gdn_kv
