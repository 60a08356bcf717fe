// libgdnspec: the attention of a step's tokens over the paged key-value cache
// (gdn_attn_decode; its C entry point is in gdnkv.cu).  Declared in include/gdnspec.h.
//
// For a row of scores s_j over keys, with any reference m and weights p_j = 2^(s_j - m)
// (log2 e is in the scale), the output is (sum p_j v_j) / (sum p_j): keys may come in any
// pieces, each with its own m, and (m, sum p, sum p v) of two pieces add up after a factor
// 2^(m - m') on one of them.  So one pass over the cache does, in three levels: a warp over
// its keys, the warps of a CTA, and the CTAs that share a sequence.
//
// A unit is one (sequence, cache head, tile of query rows); its rows are the heads of the
// group times the tokens.  All units' keys, in blocks of 64 or 128, form one line that is cut evenly
// among the CTAs, whatever the lengths; a CTA computes from the lengths alone where its part
// begins.  A part that is a whole unit is finished where it is; the others go to the workspace
// and a second launch joins them in order.
//
// Two kernels run the units: one whose warps have keys of their own (gdnattn_warp.cuh), for few
// query rows, and one on the tcgen05 tensor cores (gdnattn_tc.cuh) for more.
#include "gdnkv.h"

using namespace gdn_common;
using namespace gdn_kv;

namespace {

// Which kernel: the tcgen05 one pays where the other one, whose units have up to 32 rows (16 for a head dim over 128), would read
// the cache a second time; for head dim 64 from the third time on.  32 sequences of up to 4096, 4 heads, tcgen05 and other, in us:
// bf16, head dim 128, 24 rows 54 and 43, 32 rows 54 and 51, 48 rows 58 and 70, 64 rows 62 and 71; e4m3, 24 rows 51 and 40, 32 rows
// 55 and 50, 48 rows 68 and 70; bf16, head dim 256, 16 rows 84 and 65, 24 rows 86 and 87; head dim 64, 48 rows 53 and 45, 64 rows
// 59 and 45.  (It also depends on the lengths, which the host does not know: 128 sequences, 8 heads of 64, 48 rows, bf16, of 64
// positions 68 and 44, of 512 102 and 102, of 2048 224 and 264; head dim 128, of 64 75 and 60, of 128 76 and 82, of 512 108 and 158.)
// It wants pages of whole groups of 8 positions, and has no int8 products.
bool on_tc(const AttnParams& p, int D, gdn_dtype type) {
    const int few = D == 64 ? 64 : D == 128 ? 32 : 16;
    return type != GDN_I8 && p.ratio * p.max_T > few && p.pg.page % 8 == 0 && p.pg.num_pages < (1ll << 31);
}

}  // namespace

namespace gdn_kv {

int64_t attn_workspace(const AttnParams& p, int D, gdn_dtype type) {
    const int rows = p.ratio * p.max_T;
    if (on_tc(p, D, type)) return attn_tc_workspace(D);
    return type == GDN_BF16   ? attn_workspace_bf16(rows, D)
           : type == GDN_F16  ? attn_workspace_f16(rows, D)
           : type == GDN_E4M3 ? attn_workspace_e4m3(rows, D)
                              : attn_workspace_i8(rows, D);
}

cudaError_t launch_attn(const AttnParams& p, int D, gdn_dtype type, void* workspace, cudaStream_t stream) {
    const int rows = p.ratio * p.max_T;
    if (on_tc(p, D, type))
        return type == GDN_BF16  ? launch_attn_tc_bf16(p, D, workspace, stream)
               : type == GDN_F16 ? launch_attn_tc_f16(p, D, workspace, stream)
                                 : launch_attn_tc_e4m3(p, D, workspace, stream);
    return type == GDN_BF16   ? launch_attn_bf16(p, rows, D, workspace, stream)
           : type == GDN_F16  ? launch_attn_f16(p, rows, D, workspace, stream)
           : type == GDN_E4M3 ? launch_attn_e4m3(p, rows, D, workspace, stream)
                              : launch_attn_i8(p, rows, D, workspace, stream);
}

}  // namespace gdn_kv
