// api_kv.hip -- the C entry points declared in include/mxq_kv.h: host-side
// validation in the header's order (format, null pointers, shapes, alignment,
// supported sizes, device), then launch.
#include <cmath>

#include "../../include/mxq_kv.h"
#include "api_util.hpp"
#include "kv_kernels.hpp"

namespace {

using mxq::aligned;

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxTokens = int64_t(1) << 22;      // one workgroup a token: 2^30 work items
constexpr int64_t kMaxRows = int64_t(1) << 25;        // query rows: workgroups of every launch stay below 2^24
constexpr int64_t kMaxPositions = int64_t(1) << 30;   // of a sequence
constexpr float kMaxScale = 0x1p100f;                 // of the scores: scale * log2 e stays finite
constexpr int64_t kMaxStride = int64_t(1) << 36;      // 2^22 tokens of 4 bytes: offsets stay within 64 bits
constexpr int64_t kMaxRopeStride = int64_t(1) << 28;  // 2^31 tokens

int64_t elem_bytes(mxq_out_t t) { return t == MXQ_OUT_BF16 ? 2 : 4; }
bool out_type(mxq_out_t t) { return t == MXQ_OUT_F32 || t == MXQ_OUT_BF16; }

bool rope_format_ok(const mxq_rope_params_t& r) {
    return r.layout == MXQ_ROPE_HALF || r.layout == MXQ_ROPE_INTERLEAVED;
}

bool cache_format_ok(const mxq_kv_cache_t& c) {
    if (c.reserved != 0) return false;
    if (c.format == MXQ_KV_BF16) return !c.k_scales && !c.v_scales;
    return c.format == MXQ_KV_MXFP8;
}

bool cache_null(const mxq_kv_cache_t& c) {
    return !c.k || !c.v || (c.format == MXQ_KV_MXFP8 && (!c.k_scales || !c.v_scales));
}

bool seqs_null(const mxq_kv_seqs_t& s) { return !s.block_table || !s.cu_q || !s.kv_lens; }

// Sizes that are wrong whatever the limits.
bool cache_shape_ok(const mxq_kv_cache_t& c, const mxq_kv_seqs_t& s, int64_t tokens, int64_t heads) {
    return tokens > 0 && heads > 0 && c.num_pages > 0 && c.page_size > 0 && c.kv_heads > 0 && c.head_dim > 0 &&
           heads % c.kv_heads == 0 && s.seqs > 0 && s.max_pages > 0 && s.table_stride >= s.max_pages &&
           (c.page_size & (c.page_size - 1)) == 0;
}

bool cache_align_ok(const mxq_kv_cache_t& c, const mxq_kv_seqs_t& s) {
    return aligned(c.k, 16) && aligned(c.v, 16) && aligned(c.k_scales, 8) && aligned(c.v_scales, 8) &&
           aligned(s.block_table, 4) && aligned(s.cu_q, 4) && aligned(s.kv_lens, 4);
}

bool cache_supported(const mxq_kv_cache_t& c, const mxq_kv_seqs_t& s, int64_t tokens, int64_t heads) {
    return tokens <= kMaxTokens && heads <= 65536 && tokens * heads <= kMaxRows && s.seqs <= MXQ_KV_MAX_SEQS &&
           s.seqs * c.kv_heads <= kMaxRows / 8 && c.num_pages <= kMaxInt && c.page_size >= 16 &&
           c.page_size <= MXQ_KV_MAX_PAGE && (c.head_dim == 64 || c.head_dim == 128 || c.head_dim == 256) &&
           s.max_pages <= kMaxPositions / c.page_size && s.table_stride <= kMaxInt;
}

int log2_of(int64_t v) {
    int n = 0;
    while ((int64_t(1) << n) < v) ++n;
    return n;
}

mxq::KvCache cache_of(const mxq_kv_cache_t& c) {
    return {c.format == MXQ_KV_MXFP8 ? mxq::kKvMxfp8 : mxq::kKvBf16, c.k, c.v, c.k_scales, c.v_scales, c.num_pages,
            log2_of(c.page_size), (int)c.kv_heads, (int)c.head_dim};
}

mxq::KvSeqs seqs_of(const mxq_kv_seqs_t& s) {
    return {s.block_table, s.cu_q, s.kv_lens, (int)s.seqs, (int)s.max_pages, s.table_stride};
}

bool stride_ok(int64_t stride, int64_t heads, int64_t dim) { return stride >= heads * dim; }
bool stride_aligned(int64_t stride, int64_t bytes) { return stride % (16 / bytes) == 0; }

}  // namespace

MXQ_API int mxq_kv_version(void) { return 1; }

MXQ_API mxq_status_t mxq_rope_inv_freq(int scaling, int64_t rot_dim, double theta, double factor, double context,
                                       double low, double high, float* inv_freq, float* mscale) {
    if (scaling < MXQ_ROPE_NONE || scaling > MXQ_ROPE_BANDS) return MXQ_E_FORMAT;
    if (!inv_freq || !mscale) return MXQ_E_NULLPTR;
    if (rot_dim < 2 || rot_dim % 2 != 0 || !(theta > 1.0) || !std::isfinite(theta)) return MXQ_E_SHAPE;
    if (scaling != MXQ_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return MXQ_E_SHAPE;
    const bool ramped = scaling == MXQ_ROPE_YARN || scaling == MXQ_ROPE_BANDS;
    if (ramped && (!(context > 0.0) || !(low > 0.0) || !(high > low) || !std::isfinite(context) || !std::isfinite(high)))
        return MXQ_E_SHAPE;
    if (rot_dim > 1024) return MXQ_E_UNSUPPORTED;
    const double turn = 6.283185307179586476925;
    const int64_t n = rot_dim / 2;
    // theta grows so that the lowest frequency is divided by `factor` (one pair has only the frequency 1)
    const double base = scaling == MXQ_ROPE_NTK && rot_dim > 2
                            ? theta * std::pow(factor, (double)rot_dim / (double)(rot_dim - 2)) : theta;
    // pair index (a real number) whose frequency makes `turns` turns in the trained context
    const auto pair_of = [&](double turns) { return (double)n * std::log(context / (turns * turn)) / std::log(theta); };
    double first = 0.0, last = 1.0;
    if (scaling == MXQ_ROPE_YARN) {
        first = std::fmax(std::floor(pair_of(high)), 0.0);
        last = std::fmin(std::ceil(pair_of(low)), (double)(rot_dim - 1));
        if (!(last > first)) last = first + 0.001;
    }
    for (int64_t i = 0; i < n; ++i) {
        const double f = std::pow(base, -2.0 * (double)i / (double)rot_dim);
        double g = f;
        if (scaling == MXQ_ROPE_LINEAR) g = f / factor;
        if (ramped) {
            const double r = scaling == MXQ_ROPE_YARN ? 1.0 - ((double)i - first) / (last - first)
                                                      : (context * f / turn - low) / (high - low);
            const double keep = std::fmin(std::fmax(r, 0.0), 1.0);
            g = keep * f + (1.0 - keep) * f / factor;
        }
        inv_freq[i] = (float)g;
    }
    *mscale = scaling == MXQ_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return MXQ_OK;
}

MXQ_API mxq_status_t mxq_rope(const void* x, mxq_out_t x_dtype, void* y, mxq_out_t y_dtype, const int32_t* positions,
                              const mxq_rope_params_t* rope, int64_t tokens, int64_t heads, int64_t head_dim,
                              int64_t x_stride, int64_t y_stride, void* stream) {
    if (!out_type(x_dtype) || !out_type(y_dtype) || (rope && !rope_format_ok(*rope))) return MXQ_E_FORMAT;
    if (!x || !y || !positions || !rope || (rope->rot_dim > 0 && !rope->inv_freq)) return MXQ_E_NULLPTR;
    if (tokens <= 0 || heads <= 0 || head_dim <= 0 || head_dim % 16 != 0 || rope->rot_dim < 0 ||
        rope->rot_dim % 16 != 0 || rope->rot_dim > head_dim || heads > kMaxInt || head_dim > kMaxInt ||
        !stride_ok(x_stride, heads, head_dim) || !stride_ok(y_stride, heads, head_dim))
        return MXQ_E_SHAPE;
    // the same memory: only element for element
    if (x == y && (x_dtype != y_dtype || x_stride != y_stride)) return MXQ_E_SHAPE;
    const int64_t xb = elem_bytes(x_dtype), yb = elem_bytes(y_dtype);
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(positions, 4) || !aligned(rope->inv_freq, 4) ||
        !stride_aligned(x_stride, xb) || !stride_aligned(y_stride, yb))
        return MXQ_E_ALIGN;
    if (tokens > kMaxInt || heads * head_dim > kMaxInt || head_dim > 1024 || x_stride > kMaxRopeStride ||
        y_stride > kMaxRopeStride)
        return MXQ_E_UNSUPPORTED;
    int cus = 0;
    mxq_status_t st;
    if ((st = mxq::check_device(&cus)) != MXQ_OK) return st;
    const mxq::RopeArgs a{x, y, xb == 2, yb == 2, positions,
                          {rope->inv_freq, (int)rope->rot_dim, rope->layout == MXQ_ROPE_INTERLEAVED, rope->mscale},
                          tokens, heads, head_dim, x_stride, y_stride, cus};
    return mxq::launched(mxq::launch_rope(a, mxq::as_stream(stream)));
}

MXQ_API mxq_status_t mxq_kv_append(const void* q, const void* k, const void* v, mxq_out_t x_dtype, uint16_t* q_out,
                                   const int32_t* positions, const mxq_rope_params_t* rope,
                                   const mxq_kv_cache_t* cache, const mxq_kv_seqs_t* seqs, int64_t tokens,
                                   int64_t heads, int64_t q_stride, int64_t k_stride, int64_t v_stride, void* stream) {
    if (!out_type(x_dtype) || (rope && !rope_format_ok(*rope)) || (cache && !cache_format_ok(*cache)))
        return MXQ_E_FORMAT;
    if (!k || !v || !rope || !cache || !seqs || !q != !q_out || (rope->rot_dim > 0 && !rope->inv_freq) ||
        cache_null(*cache) || seqs_null(*seqs))
        return MXQ_E_NULLPTR;
    if (!cache_shape_ok(*cache, *seqs, tokens, heads) || rope->rot_dim < 0 || rope->rot_dim % 16 != 0 ||
        rope->rot_dim > cache->head_dim || heads > kMaxInt || cache->head_dim > kMaxInt ||
        (q && !stride_ok(q_stride, heads, cache->head_dim)) || !stride_ok(k_stride, cache->kv_heads, cache->head_dim) ||
        !stride_ok(v_stride, cache->kv_heads, cache->head_dim))
        return MXQ_E_SHAPE;
    const int64_t xb = elem_bytes(x_dtype);
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(positions, 4) ||
        !aligned(rope->inv_freq, 4) || !cache_align_ok(*cache, *seqs) || (q && !stride_aligned(q_stride, xb)) ||
        !stride_aligned(k_stride, xb) || !stride_aligned(v_stride, xb))
        return MXQ_E_ALIGN;
    if (!cache_supported(*cache, *seqs, tokens, heads) || q_stride > kMaxStride || k_stride > kMaxStride ||
        v_stride > kMaxStride)
        return MXQ_E_UNSUPPORTED;
    int cus = 0;
    mxq_status_t st;
    if ((st = mxq::check_device(&cus)) != MXQ_OK) return st;
    const mxq::AppendArgs a{q, k, v, xb == 2, q_out, positions,
                            {rope->inv_freq, (int)rope->rot_dim, rope->layout == MXQ_ROPE_INTERLEAVED, rope->mscale},
                            cache_of(*cache), seqs_of(*seqs), tokens, heads, q_stride, k_stride, v_stride, cus};
    return mxq::launched(mxq::launch_kv_append(a, mxq::as_stream(stream)));
}

MXQ_API int64_t mxq_paged_attn_workspace(const mxq_kv_cache_t* cache, const mxq_kv_seqs_t* seqs, int64_t tokens,
                                         int64_t heads, int64_t max_q) {
    if (!cache || !seqs || !cache_shape_ok(*cache, *seqs, tokens, heads) || max_q <= 0 ||
        !cache_supported(*cache, *seqs, tokens, heads))
        return -1;
    return mxq::paged_attn_workspace(heads, cache->kv_heads, cache->head_dim, cache->format == MXQ_KV_MXFP8, tokens,
                                     seqs->seqs, seqs->max_pages, cache->page_size, max_q);
}

MXQ_API mxq_status_t mxq_paged_attn(const uint16_t* q, uint16_t* out, float* lse, const mxq_kv_cache_t* cache,
                                    const mxq_kv_seqs_t* seqs, int64_t tokens, int64_t heads, int64_t q_stride,
                                    float scale, int64_t window, int64_t max_q, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
    if (cache && !cache_format_ok(*cache)) return MXQ_E_FORMAT;
    if (!q || !out || !cache || !seqs || cache_null(*cache) || seqs_null(*seqs)) return MXQ_E_NULLPTR;
    if (!cache_shape_ok(*cache, *seqs, tokens, heads) || heads > kMaxInt || cache->head_dim > kMaxInt ||
        !stride_ok(q_stride, heads, cache->head_dim) || window < 0 || max_q <= 0 || workspace_bytes < 0 ||
        !(std::fabs(scale) <= kMaxScale))
        return MXQ_E_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16) ||
        !cache_align_ok(*cache, *seqs) || !stride_aligned(q_stride, 2))
        return MXQ_E_ALIGN;
    if (!cache_supported(*cache, *seqs, tokens, heads) || q_stride > kMaxStride || window > kMaxInt)
        return MXQ_E_UNSUPPORTED;
    const int64_t need = mxq_paged_attn_workspace(cache, seqs, tokens, heads, max_q);
    if (need > 0 && !workspace) return MXQ_E_NULLPTR;
    if (workspace_bytes < need) return MXQ_E_SHAPE;
    int cus = 0;  // not used: the split is sized for 256, so that the workspace's size does not depend on the device
    mxq_status_t st;
    if ((st = mxq::check_device(&cus)) != MXQ_OK) return st;
    const mxq::AttnArgs a{q, out, lse, cache_of(*cache), seqs_of(*seqs), tokens, heads, q_stride, scale, (int)window,
                          max_q, workspace};
    return mxq::launched(mxq::launch_paged_attn(a, mxq::as_stream(stream)));
}
