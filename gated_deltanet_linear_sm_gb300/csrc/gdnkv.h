// Internal to libgdnspec: the kernel parameters of the paged key-value cache and
// of the attention over it, shared by the cache's kernels with the C entry points
// (gdnkv.cu), the choice of the attention kernel (gdnattn.cu) and the kernels (gdnattn_warp.cuh,
// gdnattn_tc.cuh).
#pragma once

#include "gdn_common.h"

namespace gdn_kv {

// Where the position x of sequence i is: page table[i][x / page], row x % page of it.
// (x / page by a multiplication: with m = ceil(2^(31+s) / page), 2^s >= page, the error
// m page - 2^(31+s) is below 2^s, so the quotient is right for every x < 2^31.)
struct Paging {
    const int32_t* table;
    int64_t num_pages;
    int64_t page_stride, token_stride, head_stride;      // elements, of k_cache and v_cache
    int64_t s_page, s_token, s_head;                     // elements, of their scales
    int64_t table_stride;
    int32_t cols, page;                                  // pages of a sequence, positions of a page
    uint32_t magic, shift;

    void divide_by(int32_t n) {
        page = n;
        uint32_t s = 0;
        while ((1ll << s) < n) ++s;
        magic = static_cast<uint32_t>(((1ull << (31 + s)) + n - 1) / n);
        shift = s;
    }
    __device__ __forceinline__ int32_t page_of(int32_t x) const {
        return static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(x)) * magic) >> (31 + shift));
    }
};

// the rows of gdn_kv_write (new rows to the cache) and gdn_kv_read (the cache to rows)
struct RowsParams {
    Paging pg;
    const __nv_bfloat16* k;         // write: the rows
    const __nv_bfloat16* v;
    void* k_rows;                   // read: the rows
    void* v_rows;
    void* k_cache;
    void* v_cache;
    float* k_scale;
    float* v_scale;
    const int32_t* first;           // the first row's position in each sequence, or null (0)
    const int32_t* cu;
    const int32_t* sti;
    int32_t* status;
    int64_t k_stride, v_stride;     // between rows
    int32_t batch, num_tokens, heads;
};

struct AttnParams {
    Paging pg;
    const __nv_bfloat16* q;
    const __nv_bfloat16* z;
    const void* k;
    const void* v;
    const float* k_scale;
    const float* v_scale;
    const int32_t* kv_lens;
    const int32_t* cu;
    const int32_t* sti;
    __nv_bfloat16* out;
    float* ws;                      // the parts of rows that CTAs share
    int32_t* meta;                  // what each CTA's parts belong to
    int32_t* status;
    int64_t q_stride, z_stride, out_stride;
    float scale;                    // of the scores, times log2(e)
    int32_t batch, num_tokens, heads, ratio, max_T, window;
    // heads whose CTAs stand side by side, on the same keys at the same time (their rows are neighbours in a
    // cache that keeps heads within positions), and groups of so many heads
    int32_t side, groups;

    void stand_side_by_side() {
        side = 1;
        for (int s = 2; s <= 8; ++s)
            if (heads % s == 0) side = s;
        groups = heads / side;
    }
};

constexpr int kMaxCtas = 1024;      // of an attention launch
constexpr int kMetaInts = 16;       // of a CTA: two records of 8

// Workspace in bytes on the current device, and the launch (gdnattn.cu chooses the kernel).
int64_t attn_workspace(const AttnParams& p, int D, gdn_dtype type);
cudaError_t launch_attn(const AttnParams& p, int D, gdn_dtype type, void* workspace, cudaStream_t stream);

// The two kernels, by the cache's type (gdnattn_bf16.cu and its like): for few query rows, and on the
// tcgen05 tensor cores.
int64_t attn_tc_workspace(int D);
int64_t attn_workspace_bf16(int rows, int D);
cudaError_t launch_attn_bf16(const AttnParams& p, int rows, int D, void* workspace, cudaStream_t stream);
cudaError_t launch_attn_tc_bf16(const AttnParams& p, int D, void* workspace, cudaStream_t stream);
int64_t attn_workspace_f16(int rows, int D);
cudaError_t launch_attn_f16(const AttnParams& p, int rows, int D, void* workspace, cudaStream_t stream);
cudaError_t launch_attn_tc_f16(const AttnParams& p, int D, void* workspace, cudaStream_t stream);
int64_t attn_workspace_e4m3(int rows, int D);
cudaError_t launch_attn_e4m3(const AttnParams& p, int rows, int D, void* workspace, cudaStream_t stream);
cudaError_t launch_attn_tc_e4m3(const AttnParams& p, int D, void* workspace, cudaStream_t stream);
int64_t attn_workspace_i8(int rows, int D);
cudaError_t launch_attn_i8(const AttnParams& p, int rows, int D, void* workspace, cudaStream_t stream);

}  // namespace gdn_kv
