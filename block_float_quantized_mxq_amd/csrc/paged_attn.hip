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

constexpr int kMaxSplits = 32;   // of the chunk kernel
constexpr int kDesignCus = 256;  // compute units the split is sized for

__device__ __forceinline__ void write_row(const AttnArgs& a, int64_t at, int dim, int e, const f32x4& sum, float top,
                                          float total, bool empty) {
    const float inv = empty ? 0.0f : 1.0f / total;
    *reinterpret_cast<u32x2_t*>(a.out + at * dim + e) =
        u32x2_t{pack_bf16(sum[0] * inv, sum[1] * inv), pack_bf16(sum[2] * inv, sum[3] * inv)};
    if (a.lse && e == 0) a.lse[at] = empty ? -__builtin_inff() : (top + __builtin_amdgcn_logf(total)) * 0.69314718055994531f;
}

// A share's weight in the join; a share that summed nothing has none, and its
// sums were not written.
__device__ __forceinline__ float share_weight(float m, float l, float top) { return l == 0.0f ? 0.0f : exp2_hw(m - top); }

__device__ __forceinline__ bool sees_nothing(const AttnArgs& a, const Seq& seq, int tok) {
    int lo, hi;
    seen_by(a, seq.pos + tok, (int)((int64_t)a.seqs.max_pages << a.cache.page_shift), &lo, &hi);
    return hi <= lo;
}

// Join of the chunk kernel's shares: a thread takes 4 elements of a row and
// adds its few shares up in order.  Bound by reading them: 512 tokens of 40
// heads of 128 in 3 shares, 31 MB, 12.8 us.
template <int D>
__global__ __launch_bounds__(256) void attn_join_chunk_kernel(AttnArgs a, AttnPlan p) {
    constexpr int LANES = D / 4, R = 256 / LANES;
    const int64_t at = (int64_t)blockIdx.x * R + threadIdx.x / LANES;
    const int64_t step = a.tokens * a.heads;
    // the rows of a wave may lie in different sequences: one after the other
    const int64_t last = (int64_t)blockIdx.x * R + (threadIdx.x | 63) / LANES;
    int sid = -1;
    for (int64_t row = (int64_t)blockIdx.x * R + (threadIdx.x & ~63) / LANES; row <= last; ++row) {
        const int s = row < step ? sequence_of(a.seqs, (int)(row / a.heads)) : a.seqs.seqs;
        if (row == at) sid = s;
    }
    const int t = (int)(at / a.heads);
    if (at >= step || sid >= a.seqs.seqs) return;
    const Seq seq = sequence(a.seqs, a.tokens, sid);
    if (t < seq.t0 || t - seq.t0 >= seq.n || rows_taken<false>(p, seq.n) == 0) return;
    int shares;
    share_of(p, span_of(a, p, seq), &shares);
    if (shares <= 1) return;  // written by the kernel itself
    const int e = 4 * (threadIdx.x % LANES);
    float m[kMaxSplits], top = -__builtin_inff();
#pragma unroll
    for (int z = 0; z < kMaxSplits; ++z) {
        m[z] = z < shares ? p.part_m[z * step + at] : -__builtin_inff();
        top = __builtin_fmaxf(top, m[z]);
    }
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    float total = 0.0f;
#pragma unroll
    for (int z = 0; z < kMaxSplits; ++z) {
        if (z < shares) {
            const float l = p.part_l[z * step + at], w = share_weight(m[z], l, top);
            const f32x4 x = *reinterpret_cast<const f32x4*>(p.part_o + (z * step + at) * D + e);
            if (l != 0.0f) {
                sum += w * x;
                total += w * l;
            }
        }
    }
    write_row(a, at, D, e, sum, top, total, sees_nothing(a, seq, t - seq.t0));
}

// Join of the decode kernel's shares: a workgroup takes a row, D / 4 threads
// its elements and 256 / (D / 4) groups of them every so many shares.  Bound by
// the launch and one round of loads: 8 rows of 128 shares each 6.3 us, 3360
// rows of 4 shares 9.0.
template <int D>
__global__ __launch_bounds__(256) void attn_join_decode_kernel(AttnArgs a, AttnPlan p) {
    constexpr int LANES = D / 4, G = 256 / LANES, U = 4;
    __shared__ f32x4 sums[G][LANES];
    __shared__ float stat[2][G];
    const int heads = a.cache.heads, kvh = (int)(blockIdx.x % (unsigned)heads);
    Work w;
    if (!find_work<true>(a, p, (int)(blockIdx.x / (unsigned)heads), &w) || w.slot < 0) return;
    const Seq seq = sequence(a.seqs, a.tokens, w.sid);
    const int first = w.tile * kFewRows, rows = seq.n * p.group - first;
    const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int64_t step = (int64_t)heads * kFewRows;
    for (int r = blockIdx.y; r < rows && r < kFewRows; r += gridDim.y) {
        const int64_t base = ((int64_t)w.slot * heads + kvh) * kFewRows + r;
        f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
        float top = -__builtin_inff(), total = 0.0f;
        for (int z0 = group; z0 < w.shares; z0 += G * U) {
            f32x4 x[U];
            float m[U], l[U], next = top;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = z0 + u * G < w.shares;
                const int64_t at = base + (in ? z0 + u * G : z0) * step;
                x[u] = *reinterpret_cast<const f32x4*>(p.part_o + at * D + 4 * lane);
                m[u] = p.part_m[at];
                l[u] = in ? p.part_l[at] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) next = l[u] == 0.0f ? next : __builtin_fmaxf(next, m[u]);
            const float keep = next == top ? 1.0f : exp2_hw(top - next);
            sum *= keep;
            total *= keep;
            top = next;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (l[u] != 0.0f) {
                    const float v = exp2_hw(m[u] - top);
                    sum += v * x[u];
                    total += v * l[u];
                }
            }
        }
        sums[group][lane] = sum;
        if (lane == 0) {
            stat[0][group] = top;
            stat[1][group] = total;
        }
        __syncthreads();
        if (group == 0) {
            top = stat[0][0];
#pragma unroll
            for (int i = 1; i < G; ++i) top = __builtin_fmaxf(top, stat[0][i]);
            sum = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const float l = stat[1][i];
                if (l != 0.0f) {
                    const float v = exp2_hw(stat[0][i] - top);
                    sum += v * sums[i][lane];
                    total += v * l;
                }
            }
            const int tok = (first + r) / p.group;
            const int64_t at = (int64_t)(seq.t0 + tok) * a.heads + kvh * p.group + (first + r - tok * p.group);
            write_row(a, at, D, 4 * lane, sum, top, total, sees_nothing(a, seq, tok));
        }
        __syncthreads();
    }
}

template <int D>
static void launch_join_chunk(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
    const int64_t rows = 1024 / D;
    const dim3 grid((unsigned)((a.tokens * a.heads + rows - 1) / rows)), block(256);
    hipLaunchKernelGGL(attn_join_chunk_kernel<D>, grid, block, 0, st, a, p);
}
template <int D>
static void launch_join_decode(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
    const int64_t most = (a.max_q < a.tokens ? a.max_q : a.tokens) * p.group;
    const dim3 grid((unsigned)(decode_tiles(a, p) * a.cache.heads), (unsigned)(most < kFewRows ? most : kFewRows)), block(256);
    hipLaunchKernelGGL(attn_join_decode_kernel<D>, grid, block, 0, st, a, p);
}

namespace {

struct Choice {
    bool few, many;
    int target;  // decode kernel: shares of the call
    int waves;   // chunk kernel: waves of a workgroup
    int splits;  // chunk kernel: shares of a sequence
};

// The chunk kernel's workgroups and shares, from a model of what they take (in
// microseconds, fitted to MI355X measurements).  One 64-key tile, heads of 128
// in bf16: two workgroups of 4 waves on a compute unit 2.3 together, one alone
// 1.63; one of 8 waves 2.15 for its 256 rows, and longer to start.  (512 tokens
// over 16k, 40/8 heads: 4 waves x 3 shares 220 us, 8 waves x 3 shares 195,
// unsplit 420; a 1000-token prompt: 4 waves unsplit 37 us, 8 waves 41, 2 shares
// 50.)  MXFP8 tiles take a sixth more.  Heads of 256 run one workgroup on a
// compute unit, of 8 waves and 128 rows (4.0 a tile) or, where those are few,
// of 4 waves and 64 (3.4; a prompt of 545 tokens, 16/2 heads, 34 us against
// 41), heads of 64 three.  Shares cost a launch and their partial sums
// (a 4096-token prompt with 16/2 heads of 256: whole 229 us, 3 shares 326).
//
// most and mean: the tiles that the last row sees, and a row on average; rows
// between see evenly fewer, so that some rows have nothing in the last shares.
void choose_chunk(Choice* c, int64_t rows_head, int64_t kv_heads, int64_t dim, bool mx, double most, double mean) {
    const double more = mx ? 1.16 : 1.0;
    const double full = (dim == 256 ? 3.4 : dim == 64 ? 1.9 : 2.3) * more;  // of all that are resident together
    const double two = (dim == 256 ? 3.4 : dim == 64 ? 1.25 : 2.3) * more, alone = (dim == 256 ? 3.4 : dim == 64 ? 0.85 : 1.63) * more;
    const double eight = (dim == 256 ? 4.0 : 2.15) * more;
    const int64_t resident = (dim == 256 ? 1 : dim == 64 ? 3 : 2) * kDesignCus;
    double best = 1e30;
    for (int waves = 4; waves <= (dim == 64 ? 4 : 8); waves += 4) {
        const int64_t rows = (dim == 256 ? 16 : 32) * waves;
        const double units = (double)(((rows_head + rows - 1) / rows) * kv_heads);
        const double slots = (double)(waves == 8 ? kDesignCus : resident), each = waves == 8 ? eight : full;
        for (int64_t s = 1; s <= kMaxSplits && (s == 1 || 64.0 * most >= 256.0 * (double)s); ++s) {
            // workgroups with something to do; their longest, mean and least work
            const double n = s == 1 ? units : units * ((double)s * mean / most + (most - mean) / most);
            const double long_s = most / (double)s, mean_s = units * mean / n, least_s = __builtin_fmax(2.0 * mean_s - long_s, 0.0);
            const double whole = __builtin_floor(n / slots), rest = n - whole * slots;
            // the longest start first, and the shortest even out the end
            const double last = waves == 8 ? eight : rest > kDesignCus ? two : alone;
            double t = last * long_s;
            if (whole > 0.0) {
                t = each * mean_s * whole;
                if (rest > 0.0) t += last * (rest * mean_s + (slots - rest) * least_s) / slots;
                t = __builtin_fmax(t, each * long_s);
            }
            t += (waves == 8 ? 6.0 : 3.0) * __builtin_ceil(n / slots);
            if (s > 1) t += 12.0 + (double)(rows_head * kv_heads * dim * 4 * s) / 2.5e6;
            if (t < best) {
                best = t;
                c->waves = waves;
                c->splits = (int)s;
            }
        }
    }
}

// Which kernels run, and into how many shares the positions are split.  max_q
// is a hint: if it puts every sequence's rows below kFewRows the decode kernel
// takes all; else the chunk kernel runs, and beside it the decode kernel if the
// number of tokens leaves room for sequences with few.
//
// The decode kernel also takes a call with more rows that has few tiles of 16
// of them: it reads the keys once a tile, but from the caches, and spreads over
// the device where the chunk kernel's tiles of 128 rows would be mostly empty
// (one sequence, 32/4 heads of 128: 64 rows over 3000 positions 14 us against
// 22, over 30000 40 and 51; 96 rows, 24 tiles, over 30000 68 and 52; 8/1 heads
// of 256, 512 rows, 32 tiles, over 8000 35 and 47, over 30000 91 and 81; 8
// sequences of 2000, 32/4 heads: 48 rows, 96 tiles, 31 and 26).
Choice choose(int64_t group, int64_t kv_heads, int64_t dim, bool mx, int64_t tokens, int64_t seqs, int64_t positions,
              int64_t max_q) {
    const int64_t most_q = max_q < tokens ? max_q : tokens;
    Choice c{};
    const int64_t by_hint = (most_q * group + kFewRows - 1) / kFewRows * seqs, by_rows = tokens * group / kFewRows + seqs;
    const int64_t tiles = (by_hint < by_rows ? by_hint : by_rows) * kv_heads;
    c.many = most_q * group > kFewRows && tiles > (positions <= 8192 ? 32 : 16);
    c.few = !c.many || (seqs > 1 && 4 * tokens < 3 * seqs * most_q);
    if (c.few) {
        // Few tiles: about as many shares as workgroups are resident less one
        // a compute unit; more tiles have other lengths each, and more and
        // shorter shares even out the last round.  (Heads of 128: one token
        // over 131071 51 us in 512 shares, 64 in 2304.)
        const int64_t units = c.many ? seqs * kv_heads : tiles;
        c.target = units > 64 ? 9 * kDesignCus : (dim == 64 ? 3 : dim == 128 ? 2 : 1) * kDesignCus;
        // Short tables: the join's launch costs more than the split saves, in a
        // captured graph below 500 positions of heads of 128, called one by one
        // below 900 (one token over 1000: whole 15.7 us captured and 17.2
        // called, split 11.0 and 18.2; 8 sequences of 600 called: 14.4 and
        // 18.6; heads of 256, 2 of 600: 23.1 and 17.6).
        if (positions * (dim == 64 ? 96 : dim) <= 768 * 128) c.target = 0;
    }
    c.waves = 4;
    c.splits = 1;
    if (c.many) {
        // tiles of the last row, and of a row on average
        const double most = (double)(positions + 63) / 64.0;
        choose_chunk(&c, tokens * group, kv_heads, dim, mx, most, most - (double)(most_q < positions ? most_q : positions) / 128.0);
    }
    return c;
}

// Rows of the partial results.  Decode: a split tile has less than twice its
// part of the target in shares, and a slot each.
int64_t chunk_rows(const Choice& c, int64_t rows) { return c.many && c.splits > 1 ? c.splits * rows : 0; }
int64_t decode_rows(const Choice& c, int64_t kv_heads) {
    return c.few && c.target > 0 ? (2 * (c.target / kv_heads) + 2) * kv_heads * kFewRows : 0;
}

AttnPlan plan_of(const AttnArgs& a, bool filter, int64_t rows, float* ws) {
    AttnPlan p{};
    p.group = (int)(a.heads / a.cache.heads);
    const float mag = a.scale < 0.0f ? -a.scale : a.scale;
    p.c = mag == 0.0f ? 1.0f : mag * 1.44269504088896341f;
    p.q_sign = a.scale > 0.0f ? 1 : a.scale < 0.0f ? -1 : 0;
    p.splits = 1;
    p.waves = 4;
    p.filter = filter ? 1 : 0;
    p.part_o = ws;
    p.part_m = ws + rows * a.cache.dim;
    p.part_l = p.part_m + rows;
    return p;
}

}  // namespace

int64_t paged_attn_workspace(int64_t heads, int64_t kv_heads, int64_t dim, bool mx, int64_t tokens, int64_t seqs,
                             int64_t max_pages, int64_t page_size, int64_t max_q) {
    const Choice c = choose(heads / kv_heads, kv_heads, dim, mx, tokens, seqs, max_pages * page_size, max_q);
    return 4 * (dim + 2) * (chunk_rows(c, tokens * heads) + decode_rows(c, kv_heads));
}

bool launch_paged_attn(const AttnArgs& a, hipStream_t st) {
    const Choice c = choose(a.heads / a.cache.heads, a.cache.heads, a.cache.dim, a.cache.fmt == kKvMxfp8, a.tokens, a.seqs.seqs,
                            (int64_t)a.seqs.max_pages << a.cache.page_shift, a.max_q);
    float* ws = static_cast<float*>(a.workspace);
    if (c.few) {
        AttnPlan p = plan_of(a, c.many, decode_rows(c, a.cache.heads), ws);
        p.target = c.target;
        p.enough = (a.cache.dim == 64 || a.cache.fmt == kKvMxfp8 ? 2 : 1) * kDesignCus;
        p.least = decode_tiles(a, p) * a.cache.heads < kDesignCus ? 128 : 512;
        if (!launch_attn_decode(a, p, st)) return false;
        if (c.target > 0) switch (a.cache.dim) {
            case 64: launch_join_decode<64>(a, p, st); break;
            case 128: launch_join_decode<128>(a, p, st); break;
            case 256: launch_join_decode<256>(a, p, st); break;
        }
        ws += decode_rows(c, a.cache.heads) * (a.cache.dim + 2);
    }
    if (c.many) {
        AttnPlan p = plan_of(a, c.few, chunk_rows(c, a.tokens * a.heads), ws);
        p.splits = c.splits;
        p.waves = c.waves;
        p.least = 256;
        if (!launch_attn_chunk(a, p, st)) return false;
        if (c.splits > 1) {
            switch (a.cache.dim) {
                case 64: launch_join_chunk<64>(a, p, st); break;
                case 128: launch_join_chunk<128>(a, p, st); break;
                case 256: launch_join_chunk<256>(a, p, st); break;
            }
        }
    }
    return true;
}

}  // namespace mxq
