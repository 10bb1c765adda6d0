// rope_append.hip -- rotary positions, and appending a step's keys and values
// to a paged cache with the rotation applied on the way.
//
// A pair (a, b) of a head's elements turns by the angle w = position *
// inv_freq: (a cos w - b sin w, b cos w + a sin w), times mscale.  The angle is
// formed in double (a 32-bit position times an fp32 frequency is exact up to
// 2^-53), reduced there to an eighth of a turn, and only then rounded to fp32,
// so that a position of 10^6 turns as exactly as position 1.
//
// One workgroup takes one token (or a share of its heads): a few lanes
// compute the token's rot / 2 sines and cosines once into LDS, then every lane
// turns 8 pairs of one head, reading 2 x 8 consecutive elements and writing
// the same.  HBM bound: each element is read once and written once.  Measured
// (MI355X): 8191 tokens of 32 bf16 heads of 128 in 23.5 us, 5.7 TB/s where a
// large copy takes 4.95; appending 5260 tokens, 32/4 bf16 heads of 128, in 20.1
// us, 5.4 TB/s; a decode step of 8 tokens in 3.0 us, of 64 into MXFP8 in 4.2,
// which is a launch with its chain of three loads (sequence, page, row).
#include "kv_device.hpp"

namespace mxq {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 512;  // rot <= 1024

// (cos, sin) of pos * inv_freq, times mscale.
__device__ __forceinline__ f32x2_t turn(int pos, float inv_freq, float mscale) {
    double r = (double)pos * (double)inv_freq * 0.15915494309189533577;  // in turns
    r -= __builtin_rint(r);
    const double q = __builtin_rint(4.0 * r);  // nearest quarter turn, -2 .. 2
    float s, c;
    sincospif(2.0f * (float)(r - 0.25 * q), &s, &c);
    const int k = (int)q & 3;
    const float cc = (k & 1) ? s : c, ss = (k & 1) ? c : s;
    return f32x2_t{((k == 1 || k == 2) ? -cc : cc) * mscale, ((k >= 2) ? -ss : ss) * mscale};
}

// The token's table of (cos, sin) pairs; ends with a barrier.
__device__ __forceinline__ void fill_turns(f32x2_t* cs, const RopeParams& r, int pos) {
    for (int i = threadIdx.x; i < r.rot / 2; i += kRopeThreads) cs[i] = turn(pos, r.inv_freq[i], r.mscale);
    __syncthreads();
}

// Where unit u (16 elements, two runs of 8) of a head lies.  Units below
// rot / 16 hold 8 pairs: two runs of rot / 2 apart, or one run of 16
// interleaved elements; the others are 16 elements that do not turn.
__device__ __forceinline__ int unit_first(const RopeParams& r, int u) {
    return (!r.interleaved && u < r.rot / 16) ? 8 * u : 16 * u;
}
__device__ __forceinline__ int unit_second(const RopeParams& r, int u) {
    return (!r.interleaved && u < r.rot / 16) ? 8 * u + r.rot / 2 : 16 * u + 8;
}

__device__ __forceinline__ void turn_unit(const RopeParams& r, const f32x2_t* cs, int u, float (&a)[8], float (&b)[8]) {
    if (u >= r.rot / 16) return;
    if (r.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2_t t0 = cs[8 * u + j], t1 = cs[8 * u + 4 + j];
            const float x0 = a[2 * j], y0 = a[2 * j + 1], x1 = b[2 * j], y1 = b[2 * j + 1];
            a[2 * j] = x0 * t0[0] - y0 * t0[1];
            a[2 * j + 1] = y0 * t0[0] + x0 * t0[1];
            b[2 * j] = x1 * t1[0] - y1 * t1[1];
            b[2 * j + 1] = y1 * t1[0] + x1 * t1[1];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const f32x2_t t = cs[8 * u + j];
            const float x = a[j], y = b[j];
            a[j] = x * t[0] - y * t[1];
            b[j] = y * t[0] + x * t[1];
        }
    }
}

// 8 consecutive elements from element e of a head at `off`, turned; the
// partners of a half-split pair are read a second time (from the caches).
template <bool BF16>
__device__ __forceinline__ void load8_turned(const RopeParams& r, const f32x2_t* cs, const void* x, int64_t off, int e,
                                             float (&v)[8]) {
    load8<BF16>(x, off + e, v);
    if (e >= r.rot) return;
    if (r.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2_t t = cs[e / 2 + j];
            const float a = v[2 * j], b = v[2 * j + 1];
            v[2 * j] = a * t[0] - b * t[1];
            v[2 * j + 1] = b * t[0] + a * t[1];
        }
    } else {
        const int half = r.rot / 2;
        const bool first = e < half;
        float p[8];
        load8<BF16>(x, off + (first ? e + half : e - half), p);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const f32x2_t t = cs[(first ? e : e - half) + j];
            v[j] = first ? v[j] * t[0] - p[j] * t[1] : v[j] * t[0] + p[j] * t[1];
        }
    }
}

template <bool XB, bool YB>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
    __shared__ f32x2_t cs[kMaxPairs];
    const int units = (int)a.dim / 16;
    const int64_t all = a.heads * units;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        __syncthreads();  // the last token's table is no longer read
        fill_turns(cs, a.rope, a.positions[t]);
        for (int64_t i = (int64_t)blockIdx.y * kRopeThreads + threadIdx.x; i < all; i += (int64_t)gridDim.y * kRopeThreads) {
            const int64_t h = i / units;
            const int u = (int)(i % units);
            const int e0 = unit_first(a.rope, u), e1 = unit_second(a.rope, u);
            const int64_t src = t * a.x_stride + h * a.dim, dst = t * a.y_stride + h * a.dim;
            float p[8], q[8];
            load8<XB>(a.x, src + e0, p);
            load8<XB>(a.x, src + e1, q);
            turn_unit(a.rope, cs, u, p, q);
            store8<YB>(a.y, dst + e0, p);
            store8<YB>(a.y, dst + e1, q);
        }
    }
}

// 8 fp32 values of a 32-element block that 4 adjacent lanes share -> E4M3
// codes (the MX conversion: shared exponent floor(log2 amax) - 8, nearest
// value with ties to even, saturating at 448).  Straight from the fp32 value,
// one rounding; *scale is the block's E8M0 byte.  Magnitudes are compared as
// integers, where infinities and NaN come out on top: such a block gets the
// NaN scale 255, so the value shows up when the cache is read.
__device__ __forceinline__ u32x2_t mx8_codes(const float (&v)[8], uint32_t* scale) {
    uint32_t top = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t m = __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu;
        top = m > top ? m : top;
    }
    const uint32_t x1 = __builtin_bit_cast(uint32_t, dpp_f32<kDppQuadXor1>(__builtin_bit_cast(float, top)));
    top = x1 > top ? x1 : top;
    const uint32_t x2 = __builtin_bit_cast(uint32_t, dpp_f32<kDppQuadXor2>(__builtin_bit_cast(float, top)));
    top = x2 > top ? x2 : top;
    int se = -127;
    if (top != 0u) {
        se = __builtin_amdgcn_frexp_expf(__builtin_bit_cast(float, top)) - 9;
        se = se < -127 ? -127 : (se > 127 ? 127 : se);
    }
    *scale = top >= 0x7F800000u ? 255u : (uint32_t)(se + 127);
    const float mul = __builtin_amdgcn_ldexpf(1.0f, -se);
    typedef short s16x2_t __attribute__((ext_vector_type(2)));
    u32x2_t out = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float p0 = __builtin_fminf(__builtin_fmaxf(v[j] * mul, -448.0f), 448.0f);
        const float p1 = __builtin_fminf(__builtin_fmaxf(v[j + 1] * mul, -448.0f), 448.0f);
        const s16x2_t hw = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(s16x2_t{0, 0}, p0, p1, 1.0f, false);
        out[j / 4] |= ((uint32_t)(uint16_t)hw[0]) << (8 * (j % 4));
    }
    return out;
}

// Work items of a token: per query head dim / 16 units of 16 elements, then
// per key and per value head the same (bf16 cache) or dim / 8 runs of 8
// (MXFP8: four adjacent lanes share a block).
template <bool XB, int FMT>
__global__ __launch_bounds__(kRopeThreads) void kv_append_kernel(AppendArgs a) {
    __shared__ f32x2_t cs[kMaxPairs];
    const int t = (int)blockIdx.x;
    const int s = sequence_of(a.seqs, t);
    if (s >= a.seqs.seqs || t < a.seqs.cu_q[0]) return;  // the whole workgroup alike
    const int dim = a.cache.dim, hk = a.cache.heads;
    const int64_t p = (int64_t)a.seqs.lens[s] - a.seqs.cu_q[s + 1] + t;
    fill_turns(cs, a.rope, a.positions ? a.positions[t] : (int)p);
    int64_t page = -1;
    if (p >= 0 && (p >> a.cache.page_shift) < a.seqs.max_pages)
        page = a.seqs.table[s * a.seqs.table_stride + (p >> a.cache.page_shift)];
    const bool stored = page >= 0 && page < a.cache.pages;
    // row of head 0 in the cache, in rows of dim elements; head h lies h pages' rows further
    const int64_t row0 = ((page * hk) << a.cache.page_shift) + (p & ((1 << a.cache.page_shift) - 1));
    const int units = dim / 16, runs = dim / (FMT == kKvMxfp8 ? 8 : 16);
    const int nq = a.q ? (int)a.heads * units : 0, nk = hk * runs;
    for (int i = blockIdx.y * kRopeThreads + threadIdx.x; i < nq + 2 * nk; i += gridDim.y * kRopeThreads) {
        if (i < nq) {
            const int h = i / units, u = i % units;
            const int e0 = unit_first(a.rope, u), e1 = unit_second(a.rope, u);
            const int64_t src = t * a.q_stride + (int64_t)h * dim, dst = (t * a.heads + h) * dim;
            float x[8], y[8];
            load8<XB>(a.q, src + e0, x);
            load8<XB>(a.q, src + e1, y);
            turn_unit(a.rope, cs, u, x, y);
            store8<true>(a.q_out, dst + e0, x);
            store8<true>(a.q_out, dst + e1, y);
        } else if (stored) {
            const bool is_v = i >= nq + nk;
            const int w = i - nq - (is_v ? nk : 0);
            const int h = w / runs, u = w % runs;
            const void* x = is_v ? a.v : a.k;
            const int64_t src = t * (is_v ? a.v_stride : a.k_stride) + (int64_t)h * dim;
            const int64_t row = row0 + ((int64_t)h << a.cache.page_shift);
            void* dst = is_v ? a.cache.v : a.cache.k;
            RopeParams r = a.rope;
            if (is_v) r.rot = 0;
            if constexpr (FMT == kKvBf16) {
                const int e0 = unit_first(r, u), e1 = unit_second(r, u);
                float x0[8], x1[8];
                load8<XB>(x, src + e0, x0);
                load8<XB>(x, src + e1, x1);
                turn_unit(r, cs, u, x0, x1);
                store8<true>(dst, row * dim + e0, x0);
                store8<true>(dst, row * dim + e1, x1);
            } else {
                float x0[8];
                load8_turned<XB>(r, cs, x, src, 8 * u, x0);
                uint32_t scale;
                const u32x2_t c = mx8_codes(x0, &scale);
                *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(dst) + row * dim + 8 * u) = c;
                if ((u & 3) == 0) (is_v ? a.cache.vs : a.cache.ks)[row * (dim / 32) + u / 4] = (uint8_t)scale;
            }
        }
    }
}

// Workgroups along y: enough that few tokens still spread over the device.
static unsigned shares(int64_t items, int64_t tokens, int cus) {
    const int64_t most = (items + kRopeThreads - 1) / kRopeThreads;
    const int64_t want = (4 * (int64_t)cus + tokens - 1) / tokens;
    const int64_t n = want < most ? want : most;
    return (unsigned)(n < 1 ? 1 : n > 65535 ? 65535 : n);
}

bool launch_rope(const RopeArgs& a, hipStream_t st) {
    const int64_t rows = a.tokens < (int64_t(1) << 22) ? a.tokens : (int64_t(1) << 22);
    const dim3 grid((unsigned)rows, shares(a.heads * (a.dim / 16), rows, a.cus)), block(kRopeThreads);
    if (a.x_bf16 && a.y_bf16) hipLaunchKernelGGL((rope_kernel<true, true>), grid, block, 0, st, a);
    else if (a.x_bf16) hipLaunchKernelGGL((rope_kernel<true, false>), grid, block, 0, st, a);
    else if (a.y_bf16) hipLaunchKernelGGL((rope_kernel<false, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((rope_kernel<false, false>), grid, block, 0, st, a);
    return true;
}

bool launch_kv_append(const AppendArgs& a, hipStream_t st) {
    const int64_t runs = a.cache.dim / (a.cache.fmt == kKvMxfp8 ? 8 : 16);
    const int64_t items = (a.q ? a.heads * (a.cache.dim / 16) : 0) + 2 * a.cache.heads * runs;
    const dim3 grid((unsigned)a.tokens, shares(items, a.tokens, a.cus)), block(kRopeThreads);
    const bool mx = a.cache.fmt == kKvMxfp8;
    if (a.x_bf16 && mx) hipLaunchKernelGGL((kv_append_kernel<true, kKvMxfp8>), grid, block, 0, st, a);
    else if (a.x_bf16) hipLaunchKernelGGL((kv_append_kernel<true, kKvBf16>), grid, block, 0, st, a);
    else if (mx) hipLaunchKernelGGL((kv_append_kernel<false, kKvMxfp8>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((kv_append_kernel<false, kKvBf16>), grid, block, 0, st, a);
    return true;
}

}  // namespace mxq
