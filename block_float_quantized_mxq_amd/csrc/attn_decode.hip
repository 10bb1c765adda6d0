// attn_decode.hip -- paged attention for few query rows per key/value head
// (decode: one new token of a sequence, or a few): bound by the stream of the
// cache from HBM.
//
// A workgroup owns up to 16 rows of one sequence and key/value head and a
// share of its positions; its 4 waves walk blocks of 32 positions on their own
// (no barrier until they join), each with the next block's rows in flight:
// 16 KB a wave for heads of 128 in bf16.  More waves a workgroup do not help
// where a call has few: one token over 1000 positions, unsplit, took 15.7 us
// with 4 and 16.8 with 12; a compute unit's own stream is the limit, so few
// tiles are split over more workgroups instead.
//
// Measured (MI355X): one token over 131071 positions, 32/4 heads of 128 in
// bf16, 44.4 us, 6.0 TB/s, and its join 6.3; 64 sequences of up to 16000
// positions, 40/8 heads in MXFP8, 197 us, 5.7 TB/s, and the join 9.0.  A plain
// stream of loads reads 5.6 to 5.8 TB/s there.
//
// Products are transposed as in the chunk kernel, on the 16x16x32 bf16 MFMA:
// S^T = K Q^T takes K rows from HBM straight into the A operand's lanes (lane
// l: key l % 16, elements by l / 16), so only V passes through LDS, to be read
// by columns.  A lane's scores belong to one row (l % 16); two score blocks of
// 16 keys make the second product's 32 keys, in the order 4 (l / 16) .. + 3 of
// the one and of the other.  The matrix unit has time to spare here, so the
// softmax weights enter as two bf16 (value and remainder): 2^-16 relative.
#include "attn_core.hpp"

namespace mxq {

constexpr int kBlock = 32;  // positions per wave and step
constexpr float kDecodeSlack = 8.0f;

template <int D, int FMT>
__global__ __launch_bounds__(256, D == 256 ? 1 : D == 128 ? 3 : 4) void attn_decode_kernel(AttnArgs a, AttnPlan plan) {
    constexpr int KSTEPS = D / 32;                       // MFMA steps of the first product
    constexpr int DB = D / 16;                           // 16-row blocks of O^T
    constexpr bool MX = FMT == kKvMxfp8;
    constexpr int EB = MX ? 1 : 2;
    constexpr int KL = MX ? D / 64 : D / 32;             // 16-byte loads of a key's row per lane
    constexpr int TPR = D * EB / 16, RPP = 64 / TPR, PASSES = kBlock / RPP;  // loads of value rows
    constexpr int W = MX ? 2 : 1;                        // 16-byte chunks of bf16 per load
    constexpr int kRow = D + 4;                          // fp32 per row of the joined sums
    constexpr int kValueBytes = kBlock * D * 2;
    constexpr int kShared = 4 * kValueBytes > 4 * kFewRows * kRow * 4 ? 4 * kValueBytes : 4 * kFewRows * kRow * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kShared];
    __shared__ float ml[2][4][kFewRows];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int col = lane & 15, quad = lane >> 4;
    const int kvh = (int)(blockIdx.x % (unsigned)a.cache.heads);
    Work work;
    if (!find_work<false>(a, plan, (int)(blockIdx.x / (unsigned)a.cache.heads), &work)) return;
    const int sid = work.sid, tile = work.tile;
    const Seq seq = sequence(a.seqs, a.tokens, sid);
    const Span span = span_of(a, plan, seq);

    const int g = plan.group, rows = seq.n * g;
    const int first = tile * kFewRows, last = (first + kFewRows < rows ? first + kFewRows : rows) - 1;
    const int cap = (int)((int64_t)a.seqs.max_pages << a.cache.page_shift);
    int lo_out, hi_in, lo_in, hi_out;
    seen_by(a, seq.pos + first / g, cap, &lo_out, &hi_in);
    seen_by(a, seq.pos + last / g, cap, &lo_in, &hi_out);
    const int begin = span.lo + work.z * work.share;
    int end = begin + work.share < span.hi ? begin + work.share : span.hi;
    if (end > hi_out) end = hi_out;
    const bool mixed = hi_in != hi_out || lo_in != lo_out;  // rows that see different positions

    const int r = first + col;
    const bool live = r < rows;
    const int tok = live ? r / g : 0, hg = live ? r - tok * g : 0;
    int lo = 0, hi = 0;
    if (live) seen_by(a, seq.pos + tok, cap, &lo, &hi);

    bf16x8 q[KSTEPS];
    {
        const uint32_t flip = plan.q_sign < 0 ? 0x80008000u : 0u, keep = (live && plan.q_sign != 0) ? 0xFFFFFFFFu : 0u;
        const uint16_t* src = a.q + (seq.t0 + tok) * a.q_stride + (int64_t)(kvh * g + hg) * D;
#pragma unroll
        for (int s = 0; s < KSTEPS; ++s) {
            // MXFP8 keys come 16 codes a lane: steps 2n and 2n + 1 take their halves
            const int e = MX ? 64 * (s / 2) + 16 * quad + 8 * (s % 2) : 32 * s + 8 * quad;
            u32x4_t w = *reinterpret_cast<const u32x4_t*>(src + e);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (w[i] ^ flip) & keep;
            q[s] = __builtin_bit_cast(bf16x8, w);
        }
    }

    f32x4 o[DB];
    float m, l;

    const int ps = a.cache.page_shift, pmask = (1 << ps) - 1;
    const int32_t* table = a.seqs.table + sid * a.seqs.table_stride;
    auto page_of = [&](int k) __attribute__((always_inline)) {
        const int p = k >> ps;
        return table[p < a.seqs.max_pages ? p : a.seqs.max_pages - 1];
    };
    auto in_range = [&](int page) __attribute__((always_inline)) { return page >= 0 && page < a.cache.pages; };
    // row of the cache where the 16 positions from k0 (in one page) start
    auto row_of = [&](int page, int k0) __attribute__((always_inline)) {
        return (((int64_t)(in_range(page) ? page : 0) * a.cache.heads + kvh) << ps) + (k0 & pmask);
    };
    u32x4_t kx[2][KL], vx[PASSES];
    uint32_t ksc[2][KL], vsc[PASSES];
    const int vrow = lane / TPR, vchunk = lane % TPR;
    auto load_k = [&](int k0, int p0, int p1) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int64_t base = row_of(b ? p1 : p0, k0 + 16 * b);
            const uint8_t* x = static_cast<const uint8_t*>(a.cache.k) + base * (D * EB);
#pragma unroll
            for (int n = 0; n < KL; ++n) {
                kx[b][n] = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4_t*>(x + (uint32_t)(col * (D * EB) + 64 * n + 16 * quad)));
                if constexpr (MX) ksc[b][n] = (a.cache.ks + base * (D / 32))[(uint32_t)(col * (D / 32) + 2 * n + quad / 2)];
            }
        }
    };
    auto load_v = [&](int k0, int p0, int p1) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < PASSES; ++n) {
            const int row0 = n * RPP;
            const int64_t base = row_of(row0 >= 16 ? p1 : p0, k0 + row0);
            const uint8_t* x = static_cast<const uint8_t*>(a.cache.v) + base * (D * EB);
            vx[n] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(x + (uint32_t)(vrow * (D * EB) + vchunk * 16)));
            if constexpr (MX) vsc[n] = (a.cache.vs + base * (D / 32))[(uint32_t)(vrow * (D / 32) + vchunk / 2)];
        }
    };
    // Rows of 2 D bytes; the 16-byte chunk index is XORed so that the 8 rows x
    // 32 bytes that 32 lanes read by columns hit distinct banks.
    uint8_t* vt = lds + wave * kValueBytes;
    auto swizzle = [&](int row) __attribute__((always_inline)) { return D == 64 ? ((row >> 1) & 3) << 1 : (row & 7) << 1; };
    const int step = 4 * kBlock;
    // Both parts of a weight times an infinite value may make NaN of it.  If a
    // sum comes out as NaN, the wave takes its blocks once more with all values
    // that are not finite out of the products, as those always are that only
    // some rows see.
    bool taken_out = false, all_out = false;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        m = -__builtin_inff();
        l = 0.0f;
        int k0 = begin + wave * kBlock;
        if (k0 >= end) break;
        int p0 = page_of(k0), p1 = page_of(k0 + 16);
        load_k(k0, p0, p1);
        load_v(k0, p0, p1);
        int n0 = page_of(k0 + step), n1 = page_of(k0 + step + 16);
        for (; k0 < end; k0 += step) {
            const bool more = k0 + step < end;
            const bool bad0 = !in_range(p0), bad1 = k0 + 16 < end && !in_range(p1);
            const bool edge = k0 + kBlock > hi_in || k0 < lo_in || k0 + kBlock > end || bad0 || bad1;
            const bool out = all_out || (edge && mixed);  // values that are not finite
            // ---- scores ----
            f32x4 s[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                s[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int n = 0; n < KL; ++n) {
                    if constexpr (MX) {
                        const float e = e8m0_exponent(ksc[b][n]);
                        const u32x4_t x0 = mx8_to_bf16(kx[b][n][0], kx[b][n][1], e);
                        const u32x4_t x1 = mx8_to_bf16(kx[b][n][2], kx[b][n][3], e);
                        s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x0), q[2 * n], s[b], 0, 0, 0);
                        s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x1), q[2 * n + 1], s[b], 0, 0, 0);
                    } else {
                        s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kx[b][n]), q[n], s[b], 0, 0, 0);
                    }
                }
            }
            if (more) load_k(k0 + step, n0, n1);
            // ---- values into LDS ----
#pragma unroll
            for (int n = 0; n < PASSES; ++n) {
                const int row = n * RPP + vrow;
                u32x4_t w[W];
                if constexpr (MX) {
                    const float e = e8m0_exponent(vsc[n]);
                    w[0] = mx8_to_bf16(vx[n][0], vx[n][1], e);
                    w[1] = mx8_to_bf16(vx[n][2], vx[n][3], e);
                } else {
                    w[0] = vx[n];
                }
                if (edge || all_out) {
                    const bool keep = (k0 + row < end) & (k0 + row >= lo_out) & !(row < 16 ? bad0 : bad1);
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        if (!keep) w[i] = u32x4_t{0, 0, 0, 0};
                        if (out) taken_out |= take_out_not_finite(w[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < W; ++i)
                    *reinterpret_cast<u32x4_t*>(vt + row * (D * 2) + 16 * ((vchunk * W + i) ^ swizzle(row))) = w[i];
            }
            if (more) {
                load_v(k0 + step, n0, n1);
                p0 = n0;
                p1 = n1;
                n0 = page_of(k0 + 2 * step);
                n1 = page_of(k0 + 2 * step + 16);
            }
            // ---- softmax ----
            if (edge) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = k0 + 16 * b + 4 * quad + i;
                        if (b ? bad1 : bad0) s[b][i] = __builtin_nanf("");
                        s[b][i] = ((key >= lo) & (key < hi) & (key < end)) ? s[b][i] : -__builtin_inff();
                    }
            }
            float top = s[0][0];
#pragma unroll
            for (int i = 0; i < 4; ++i) top = __builtin_fmaxf(top, __builtin_fmaxf(s[0][i], s[1][i]));
            top *= plan.c;
            if (__any(top > m + kDecodeSlack)) {
                const float n = __builtin_fmaxf(m, max_halves(max_rows16(top)));
                const float keep = n == m ? 1.0f : exp2_hw(m - n);
                l *= keep;
#pragma unroll
                for (int d = 0; d < DB; ++d) o[d] *= keep;
                m = n;
            }
            const float shift = m == -__builtin_inff() ? 0.0f : m;
            u32x4_t ph, pl;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float x0 = exp2_hw(__builtin_fmaf(s[i / 4][i % 4], plan.c, -shift));
                const float x1 = exp2_hw(__builtin_fmaf(s[i / 4][i % 4 + 1], plan.c, -shift));
                l += x0 + x1;
                ph[i / 2] = pack_bf16(x0, x1);
                pl[i / 2] = pack_bf16(x0 - bf16_lo_to_f32(ph[i / 2]), x1 - bf16_hi_to_f32(ph[i / 2]));
            }
            // ---- values ----
            const int kq = 4 * quad + col / 4;  // row of this lane in a transpose read, and + 16
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                const int off = 16 * ((2 * d + ((lane & 3) >> 1)) ^ swizzle(kq)) + 8 * (lane & 1);
                const u32x2_t v0 = read_column4(vt + kq * (D * 2) + off);
                const u32x2_t v1 = read_column4(vt + (kq + 16) * (D * 2) + off);
                const bf16x8 v = __builtin_bit_cast(bf16x8, u32x4_t{v0[0], v0[1], v1[0], v1[1]});
                o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8, ph), o[d], 0, 0, 0);
                o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8, pl), o[d], 0, 0, 0);
            }
        }
        bool none = true;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) none &= o[d][i] == o[d][i];
        if (all_out || __all(none)) break;
        all_out = true;
    }
    if (__any(taken_out)) {
        // values that are not finite, staged as zeros: added where a row sees them
#pragma unroll 1
        for (int b = begin + wave * kBlock; b < end; b += step) {
#pragma unroll 1
            for (int key = b; key < b + kBlock && key < end; ++key) {
                const int page = page_of(key);
                if (!in_range(page) || !(all_out || b + kBlock > hi_in || b < lo_in)) continue;
                const int64_t row = (((int64_t)page * a.cache.heads + kvh) << ps) + (key & pmask);
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    o[d] += not_finite_part<FMT>(a.cache.v, a.cache.vs, row, D, 16 * d + 4 * quad, (key >= lo) & (key < hi));
            }
        }
    }

    // ---- join the four waves ----
    l = sum_halves(sum_rows16(l));
    float* sums = reinterpret_cast<float*>(lds);
    __syncthreads();  // every wave is done with its values
#pragma unroll
    for (int d = 0; d < DB; ++d)
        *reinterpret_cast<f32x4*>(sums + (wave * kFewRows + col) * kRow + 16 * d + 4 * quad) = o[d];
    if (quad == 0) {
        ml[0][wave][col] = m;
        ml[1][wave][col] = l;
    }
    __syncthreads();
    const int row = tid / 16, part = tid % 16;  // 16 threads a row
    if (first + row >= rows) return;
    float top = ml[0][0][row];
#pragma unroll
    for (int w = 1; w < 4; ++w) top = __builtin_fmaxf(top, ml[0][w][row]);
    float weight[4], total = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float lw = ml[1][w][row];
        weight[w] = lw == 0.0f ? 0.0f : exp2_hw(ml[0][w][row] - top);
        total += lw == 0.0f ? 0.0f : weight[w] * lw;
    }
    const int t = (first + row) / g;
    const int64_t at = (int64_t)(seq.t0 + t) * a.heads + kvh * g + (first + row - t * g);
    int rlo, rhi;
    seen_by(a, seq.pos + t, cap, &rlo, &rhi);
    const bool empty = rhi <= rlo;
    const float inv = empty ? 0.0f : 1.0f / total;
    // row of the partial results
    const int64_t slot = ((int64_t)(work.slot + work.z) * a.cache.heads + kvh) * kFewRows + row;
#pragma unroll
    for (int e = 4 * part; e < D; e += 64) {
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < 4; ++w)
            if (weight[w] != 0.0f) x += weight[w] * *reinterpret_cast<const f32x4*>(sums + (w * kFewRows + row) * kRow + e);
        if (work.slot < 0)
            *reinterpret_cast<u32x2_t*>(a.out + at * D + e) = u32x2_t{pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv)};
        else
            *reinterpret_cast<f32x4*>(plan.part_o + slot * D + e) = x;
    }
    if (part == 0) {
        if (work.slot < 0) {
            if (a.lse) a.lse[at] = empty ? -__builtin_inff() : (top + __builtin_amdgcn_logf(total)) * 0.69314718055994531f;
        } else {
            plan.part_m[slot] = top;
            plan.part_l[slot] = total;
        }
    }
}

template <int D>
static void launch_dim(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
    const dim3 grid((unsigned)(decode_shares(a, p) * a.cache.heads)), block(256);
    if (a.cache.fmt == kKvMxfp8) hipLaunchKernelGGL((attn_decode_kernel<D, kKvMxfp8>), grid, block, 0, st, a, p);
    else hipLaunchKernelGGL((attn_decode_kernel<D, kKvBf16>), grid, block, 0, st, a, p);
}

bool launch_attn_decode(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
    switch (a.cache.dim) {
        case 64: launch_dim<64>(a, p, st); return true;
        case 128: launch_dim<128>(a, p, st); return true;
        case 256: launch_dim<256>(a, p, st); return true;
    }
    return false;
}

}  // namespace mxq
