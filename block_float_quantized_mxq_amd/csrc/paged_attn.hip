// paged_attn.hip -- attention of a step's new tokens over a paged cache: the
// choice of kernels, the split of the keys, and the join of partial results.
//
// For a query row at position p: o = sum_j softmax_j(scale q.k_j) v_j over the
// cached positions j <= p (and j > p - window), in one pass over the keys with
// the running maximum m and sum l of the softmax.  Where there are too few
// tiles of rows to fill the device, the positions of a sequence are split into
// shares; each leaves (m, l, sum of weights times values) in the workspace,
// and the join weighs them by exp(m_z - max m).
#include "attn_core.hpp"

namespace mxq {

constexpr int kMaxSplits = 256;
constexpr int kDesignCus = 256;  // compute units the split is sized for

// Joins what one of the two kernels left: one wave per row; lane z % 64 holds
// share z's statistics.
template <bool FEW>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, AttnPlan p) {
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    if (row >= a.tokens * a.heads) return;
    const int t = (int)(row / a.heads);
    const int sid = sequence_of(a.seqs, t);
    if (sid >= a.seqs.seqs || t < a.seqs.cu_q[0]) return;
    const Seq seq = sequence(a.seqs, a.tokens, sid);
    if (t < seq.t0 || t - seq.t0 >= seq.n) return;
    if (rows_taken<FEW>(p, seq.n) == 0) return;
    const Span span = span_of(a, p, seq);
    if (span.shares <= 1) return;  // written by the kernel itself
    const int64_t step = a.tokens * a.heads;
    float m[kMaxSplits / 64], l[kMaxSplits / 64], top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kMaxSplits / 64; ++i) {
        const int z = 64 * i + lane;
        m[i] = -__builtin_inff();
        l[i] = 0.0f;
        if (z < span.shares) {
            m[i] = p.part_m[z * step + row];
            l[i] = p.part_l[z * step + row];
        }
        top = __builtin_fmaxf(top, m[i]);
    }
    top = max_halves(max_rows16(top));
    top = __builtin_fmaxf(top, dpp_f32<kDppQuadXor1>(top));
    top = __builtin_fmaxf(top, dpp_f32<kDppQuadXor2>(top));
    top = __builtin_fmaxf(top, dpp_f32<kDppRowHalfMirror>(top));
    top = __builtin_fmaxf(top, dpp_f32<kDppRowMirror>(top));
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxSplits / 64; ++i) {
        m[i] = l[i] == 0.0f ? 0.0f : exp2_hw(m[i] - top);  // the share's weight
        total += l[i] == 0.0f ? 0.0f : m[i] * l[i];
    }
    total = group_sum<64>(total);
    const int dim = a.cache.dim, each = dim / 64;  // adjacent elements per lane: 1, 2 or 4
    float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kMaxSplits / 64; ++i) {
        const int n = span.shares - 64 * i < 64 ? span.shares - 64 * i : 64;
        for (int z = 0; z < n; ++z) {
            const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, m[i]), z));
            if (w == 0.0f) continue;  // nothing was summed there
            const float* src = p.part_o + ((64 * i + z) * step + row) * dim + lane * each;
            if (each == 1) {
                o[0] += w * src[0];
            } else if (each == 2) {
                const f32x2_t x = *reinterpret_cast<const f32x2_t*>(src);
                o[0] += w * x[0];
                o[1] += w * x[1];
            } else {
                const f32x4 x = *reinterpret_cast<const f32x4*>(src);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] += w * x[j];
            }
        }
    }
    const int cap = (int)((int64_t)a.seqs.max_pages << a.cache.page_shift);
    int lo, hi;
    seen_by(a, seq.pos + (t - seq.t0), cap, &lo, &hi);
    const bool empty = hi <= lo;
    const float inv = empty ? 0.0f : 1.0f / total;
    uint16_t* dst = a.out + row * dim + lane * each;
    if (each == 1) {
        dst[0] = (uint16_t)pack_bf16(o[0] * inv, 0.0f);
    } else {
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16(o[0] * inv, o[1] * inv);
        if (each == 4) *reinterpret_cast<uint32_t*>(dst + 2) = pack_bf16(o[2] * inv, o[3] * inv);
    }
    if (a.lse && lane == 0) a.lse[row] = empty ? -__builtin_inff() : (top + __builtin_amdgcn_logf(total)) * 0.69314718055994531f;
}

namespace {

struct Choice {
    bool few, many;
    int few_splits, many_splits;
};

// Which kernels run, and into how many shares the positions are split at most.
// max_q is a hint: with every sequence's rows below kFewRows the decode kernel
// takes all, a single sequence with more goes to the chunk kernel, else both
// run and each takes its side.
Choice choose(int64_t group, int64_t kv_heads, int64_t tokens, int64_t seqs, int64_t positions, int64_t max_q) {
    const int64_t most = (max_q < tokens ? max_q : tokens) * group;
    Choice c{};
    c.few = most <= kFewRows || seqs > 1;
    c.many = most > kFewRows;
    c.few_splits = c.many_splits = 1;
    if (c.few) {
        // about 8 workgroups a compute unit, of at least 128 positions each
        const int64_t tiles = c.many || seqs > tokens * group / kFewRows ? seqs : tokens * group / kFewRows;
        const int64_t units = tiles * kv_heads;
        int64_t s = (8 * kDesignCus + units - 1) / units;
        const int64_t top = (positions + 127) / 128;
        s = s < top ? s : top;
        c.few_splits = (int)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
    }
    if (c.many) {
        // two workgroups are resident on a compute unit: the number of shares
        // that fills the last round best, with a price for each share's join
        const int64_t units = ((tokens * group + kChunkRows - 1) / kChunkRows) * kv_heads;
        const int64_t top = (positions + 255) / 256;
        double best = 1e30;
        for (int64_t s = 1; s <= 32 && s <= top; ++s) {
            const double rounds = (double)((units * s + 2 * kDesignCus - 1) / (2 * kDesignCus));
            const double cost = rounds / (double)s * (1.0 + 0.03 * (double)(s - 1));
            if (cost < best) {
                best = cost;
                c.many_splits = (int)s;
            }
        }
    }
    return c;
}

int64_t partial_floats(int64_t splits, int64_t rows, int64_t dim) { return splits > 1 ? splits * rows * (dim + 2) : 0; }

AttnPlan plan_of(const AttnArgs& a, int splits, int least, bool filter, float* ws) {
    AttnPlan p{};
    p.group = (int)(a.heads / a.cache.heads);
    const float mag = a.scale < 0.0f ? -a.scale : a.scale;
    p.c = mag == 0.0f ? 1.0f : mag * 1.44269504088896341f;
    p.q_sign = a.scale > 0.0f ? 1 : a.scale < 0.0f ? -1 : 0;
    p.splits = splits;
    p.least = least;
    p.filter = filter ? 1 : 0;
    const int64_t rows = (int64_t)splits * a.tokens * a.heads;
    p.part_o = ws;
    p.part_m = ws + rows * a.cache.dim;
    p.part_l = p.part_m + rows;
    return p;
}

}  // namespace

int64_t paged_attn_workspace(int64_t heads, int64_t kv_heads, int64_t dim, int64_t tokens, int64_t seqs,
                             int64_t max_pages, int64_t page_size, int64_t max_q) {
    const Choice c = choose(heads / kv_heads, kv_heads, tokens, seqs, max_pages * page_size, max_q);
    const int64_t rows = tokens * heads;
    return 4 * ((c.few ? partial_floats(c.few_splits, rows, dim) : 0) + (c.many ? partial_floats(c.many_splits, rows, dim) : 0));
}

bool launch_paged_attn(const AttnArgs& a, hipStream_t st) {
    const int64_t group = a.heads / a.cache.heads;
    const Choice c = choose(group, a.cache.heads, a.tokens, a.seqs.seqs, (int64_t)a.seqs.max_pages << a.cache.page_shift, a.max_q);
    float* ws = static_cast<float*>(a.workspace);
    const AttnPlan few = plan_of(a, c.few_splits, 128, c.many, ws);
    if (c.few) ws += partial_floats(c.few_splits, a.tokens * a.heads, a.cache.dim);
    const AttnPlan many = plan_of(a, c.many_splits, 256, c.few, ws);
    if (c.many && !launch_attn_chunk(a, many, st)) return false;
    if (c.few && !launch_attn_decode(a, few, st)) return false;
    const dim3 grid((unsigned)((a.tokens * a.heads + 3) / 4)), block(256);
    if (c.many && c.many_splits > 1) hipLaunchKernelGGL(attn_join_kernel<false>, grid, block, 0, st, a, many);
    if (c.few && c.few_splits > 1) hipLaunchKernelGGL(attn_join_kernel<true>, grid, block, 0, st, a, few);
    return true;
}

}  // namespace mxq
