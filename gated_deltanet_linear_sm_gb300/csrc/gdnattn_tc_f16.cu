// libgdnspec: the tcgen05 attention over a fp16 cache (gdnattn_tc.cuh).
#include "gdnattn_tc.cuh"

namespace gdn_kv {

cudaError_t launch_attn_tc_f16(const AttnParams& p, int D, void* workspace, cudaStream_t stream) {
    return launch_kind<kF16>(p, D, workspace, stream);
}

}  // namespace gdn_kv
