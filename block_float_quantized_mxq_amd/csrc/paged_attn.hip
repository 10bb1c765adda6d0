// paged_attn.hip -- attention of a step's new tokens over a paged cache.
//
// For a query row at position p: o = sum_j softmax_j(scale q.k_j) v_j over the
// cached positions j <= p (and j > p - window).  One pass over the keys with
// the running maximum m and sum l of the softmax: a new score s moves m to
// max(m, s), scales what was summed by exp(m - m'), and adds exp(s - m') v.
#include "kv_device.hpp"

namespace mxq {

// Element e of row `row` of a cache half.
template <int FMT>
__device__ __forceinline__ float cache_value(const void* x, const uint8_t* scales, int64_t row, int dim, int e) {
    if constexpr (FMT == kKvBf16) {
        return __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t*>(x)[row * dim + e] << 16);
    } else {
        const float c = e4m3_to_f32(static_cast<const uint8_t*>(x)[row * dim + e]);
        return c * e8m0_to_f32(scales[row * (dim / 32) + e / 32]);
    }
}

// One wave per (token, query head); lane l holds elements l, l + 64, ...
template <int DIM, int FMT>
__global__ __launch_bounds__(256) void paged_attn_row_kernel(AttnArgs a) {
    constexpr int E = DIM / 64;
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    if (item >= a.tokens * a.heads) return;
    const int64_t t = item / a.heads;
    const int h = (int)(item % a.heads);
    const int s = sequence_of(a.seqs, (int)t);
    if (s >= a.seqs.seqs || t < a.seqs.cu_q[0]) return;
    const int kvh = h / (int)(a.heads / a.cache.heads);
    const int ps = 1 << a.cache.page_shift;
    int64_t len = a.seqs.lens[s];
    const int64_t pos = len - a.seqs.cu_q[s + 1] + t;
    const int64_t cap = (int64_t)a.seqs.max_pages << a.cache.page_shift;
    int64_t hi = pos + 1;
    if (hi > cap) hi = cap;
    int64_t lo = a.window > 0 ? pos - a.window + 1 : 0;
    if (lo < 0) lo = 0;
    float q[E], o[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        q[i] = __builtin_bit_cast(float, (uint32_t)a.q[t * a.q_stride + (int64_t)h * DIM + lane + 64 * i] << 16);
        o[i] = 0.0f;
    }
    float m = -__builtin_inff(), l = 0.0f;
    for (int64_t j = lo; j < hi; ++j) {
        const int64_t page = a.seqs.table[s * a.seqs.table_stride + (j >> a.cache.page_shift)];
        const bool ok = page >= 0 && page < a.cache.pages;
        const int64_t row = (((ok ? page : 0) * a.cache.heads + kvh) << a.cache.page_shift) + (j & (ps - 1));
        float d = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) d += q[i] * cache_value<FMT>(a.cache.k, a.cache.ks, row, DIM, lane + 64 * i);
        d = ok ? group_sum<64>(d) * a.scale : __builtin_nanf("");
        const float n = d > m ? d : m;
        const float keep = n == m ? 1.0f : expf(m - n), w = expf(d - n);
        l = l * keep + w;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = o[i] * keep + w * cache_value<FMT>(a.cache.v, a.cache.vs, row, DIM, lane + 64 * i);
        m = n;
    }
    const bool empty = hi <= lo;
    const float inv = empty ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < E; ++i)
        a.out[(t * a.heads + h) * DIM + lane + 64 * i] = __builtin_bit_cast(uint16_t, (__bf16)(o[i] * inv));
    if (a.lse && lane == 0) a.lse[t * a.heads + h] = empty ? -__builtin_inff() : m + logf(l);
}

template <int DIM>
static void launch_rows(const AttnArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((a.tokens * a.heads + 3) / 4)), block(256);
    if (a.cache.fmt == kKvMxfp8) hipLaunchKernelGGL((paged_attn_row_kernel<DIM, kKvMxfp8>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((paged_attn_row_kernel<DIM, kKvBf16>), grid, block, 0, st, a);
}

bool launch_paged_attn(const AttnArgs& a, hipStream_t st) {
    switch (a.cache.dim) {
        case 64: launch_rows<64>(a, st); return true;
        case 128: launch_rows<128>(a, st); return true;
        case 256: launch_rows<256>(a, st); return true;
    }
    return false;
}

int64_t paged_attn_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

}  // namespace mxq
