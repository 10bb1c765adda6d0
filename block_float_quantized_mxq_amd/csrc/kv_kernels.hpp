// kv_kernels.hpp -- host-side interface between the C entry points of
// include/mxq_kv.h (api_kv.hip) and the kernels of the positions-and-cache
// half of a decode layer.  Arguments arrive here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

// Cache formats; values match mxq_kv_format in include/mxq_kv.h.
enum : int { kKvBf16 = 0, kKvMxfp8 = 2 };

// Rotation of the first rot elements of a head.
struct RopeParams {
    const float* inv_freq;
    int rot;
    int interleaved;
    float mscale;
};

// Paged cache [pages][heads][1 << page_shift][dim]; MXFP8: with scales [...][dim / 32].
struct KvCache {
    int fmt;
    void* k;
    void* v;
    uint8_t* ks;
    uint8_t* vs;
    int64_t pages;
    int page_shift, heads, dim;
};

// The sequences of one step (device arrays; their values are not trusted).
struct KvSeqs {
    const int32_t* table;
    const int32_t* cu_q;
    const int32_t* lens;
    int seqs, max_pages;
    int64_t table_stride;
};

struct RopeArgs {
    const void* x;
    void* y;
    int x_bf16, y_bf16;
    const int32_t* positions;
    RopeParams rope;
    int64_t tokens, heads, dim, x_stride, y_stride;
    int cus;
};

struct AppendArgs {
    const void* q;  // null: keys and values only
    const void* k;
    const void* v;
    int x_bf16;
    uint16_t* q_out;
    const int32_t* positions;  // null: the positions in the cache
    RopeParams rope;
    KvCache cache;
    KvSeqs seqs;
    int64_t tokens, heads, q_stride, k_stride, v_stride;
    int cus;
};

struct AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    float* lse;  // may be null
    KvCache cache;
    KvSeqs seqs;
    int64_t tokens, heads, q_stride;
    float scale;
    int window;  // 0: none
    int64_t max_q;
    void* workspace;
};

bool launch_rope(const RopeArgs& a, hipStream_t st);
bool launch_kv_append(const AppendArgs& a, hipStream_t st);
bool launch_paged_attn(const AttnArgs& a, hipStream_t st);
// Workspace of launch_paged_attn.
int64_t paged_attn_workspace(int64_t heads, int64_t kv_heads, int64_t dim, bool mx, int64_t tokens, int64_t seqs,
                             int64_t max_pages, int64_t page_size, int64_t max_q);

}  // namespace mxq
