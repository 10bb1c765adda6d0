// attn_chunk.hip -- paged attention for tiles of many query rows (a chunk of a
// prompt, a whole prompt): matrix-core bound.
//
// A workgroup of 4 or 8 waves owns 128 or 256 rows (32 a wave) of one sequence
// and key/value head and walks the keys they see in tiles of 64, staged in LDS
// as bf16 and double buffered; the next tile's rows travel from HBM to registers
// while the current one is multiplied.
//
// Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T, on the
// 32x32x16 bf16 MFMA.  Then a lane's accumulators all belong to one query row
// (column lane % 32): the softmax maximum and sum are per-lane values, the
// rescaling is a per-lane product, and the weights P^T come out of the first
// product in the lanes that need them as the second one's B operand -- the key
// order inside an MFMA step is free, so V^T is read in the order P^T has (16
// keys: 4h .. 4h+3 and 8+4h .. 8+4h+3 for wave half h).  V^T's A operand is a
// column read of the row-major tile (the LDS transpose read).
//
// The running maximum only moves when a score exceeds it by 2^8 (one vote of
// the wave): until then weights up to 2^8 are summed, which costs nothing in
// fp32 or in bf16's relative precision, and saves the rescaling of the sums.
//
// The weights are rounded to bf16 for the second product: relative 2^-8 each,
// of the same size as the rounding of the output, and averaged over the keys.
// The softmax's sum takes the unrounded weights.
//
// Heads of 256 do not leave room for a row's queries and sums in the registers
// of a wave that shares its SIMD: two waves share 32 rows, both take the whole
// first product and each half of the output's elements.  That is half as much
// matrix work again, and still faster than one wave a SIMD (a prompt of 4096
// tokens, 16/2 heads, in 3 shares: 331 us against 400; in one 229).  A
// workgroup there has 64 or 128 rows.
//
// Measured (MI355X; bf16, 40/8 heads of 128): a prompt of 8192 tokens 710 us,
// 970 TFLOP/s; 512 tokens over 16000 191 us with the join, 890 TFLOP/s; 2
// prompts of 4000, window 1024, 32/8 heads of 64, 107 us, 610 TFLOP/s, where a
// score has half the matrix work and the same vector work.  A
// library matrix product of 8192 x 8192 x 8192 takes 1390-1480 TFLOP/s, and a
// loop of nothing but these MFMAs on such data 1756: the power limit, not the
// issue rate, ends both.  Here the softmax's vector work and the staging share
// the issue slots with the MFMAs: without any staging the same kernel took 26%
// less, without the maximum 6%, without the page lookups 7%.
#include "attn_core.hpp"

namespace mxq {

constexpr float kSlack = 8.0f;

// Keys per tile, in blocks of the 32 of an MFMA: heads of 256 take half the keys (64 spill: 335 us against 331 for a
// prompt of 4096 tokens split alike).
template <int D>
constexpr int kKeyBlocks = D == 256 ? 1 : 2;

// Waves that share 32 rows, each with its part of the output's elements.
template <int D>
constexpr int kParts = D == 256 ? 2 : 1;

// LDS tile of rows of D bf16, in 16-byte chunks; the chunk index is XORed
// with bits of the row so that a column of rows (K: 16-byte reads of 32 rows)
// or 4 rows x 64 bytes (V: transpose reads) hit distinct banks.
template <int D>
struct Tile {
    static constexpr int kKeys = 32 * kKeyBlocks<D>;
    static constexpr int CH = D / 8;
    static constexpr int kBytes = kKeys * D * 2;
    static constexpr int kMask = CH < 16 ? CH - 1 : 15;
    static __device__ __forceinline__ int k_chunk(int row, int chunk) { return chunk ^ (row & kMask); }
    static __device__ __forceinline__ int v_swizzle(int row) {
        return D == 64 ? ((row >> 1) & 1) << 2 : (row & 3) << 2;
    }
};

// How the threads share the loads of a tile's rows (one half, k or v).
template <int D, int FMT, int NW>
struct Stage {
    static constexpr int NT = 64 * NW;
    static constexpr int VEC = FMT == kKvBf16 ? 8 : 16;       // elements per 16-byte load
    static constexpr int TPR = D / VEC;                       // threads per row
    static constexpr int RPP = NT / TPR;                      // rows per pass
    static constexpr int PASSES = Tile<D>::kKeys / RPP;
    static constexpr int RPW = 64 / TPR;                      // rows per wave and pass
};

template <int D, int FMT, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 && NW == 4 ? 1 : 2) void attn_chunk_kernel(AttnArgs a, AttnPlan plan) {
    using T = Tile<D>;
    using St = Stage<D, FMT, NW>;
    constexpr int PARTS = kParts<D>, ROWS = 32 * NW / PARTS;
    constexpr int NB = kKeyBlocks<D>, kKeys = T::kKeys;
    constexpr int KSTEPS = D / 16;  // MFMA steps of the first product
    constexpr int DB = D / 32 / PARTS;  // 32-row blocks of a wave's O^T
    __shared__ __attribute__((aligned(16))) uint8_t k_lds[2][T::kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t v_lds[2][T::kBytes];
    __shared__ int taken_out, bad_pages;  // whether a value that is not finite was staged as zero

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int half = lane >> 5, col = lane & 31;
    const int kvh = (int)(blockIdx.x % (unsigned)a.cache.heads);
    // the last tiles of a sequence see the most keys: they start first
    const int index = (int)(gridDim.x / (unsigned)a.cache.heads) - 1 - (int)(blockIdx.x / (unsigned)a.cache.heads);
    int sid, tile;
    if (!find_tile<ROWS, false>(a, plan, index, &sid, &tile)) return;
    const Seq seq = sequence(a.seqs, a.tokens, sid);
    const Span span = span_of(a, plan, seq);
    int shares;
    const int share = share_of(plan, span, &shares);
    const int z = blockIdx.y;
    if (z > 0 && z >= shares) return;

    const int g = plan.group, rows = seq.n * g;
    const int first = tile * ROWS, last = (first + ROWS < rows ? first + ROWS : rows) - 1;
    const int cap = (int)((int64_t)a.seqs.max_pages << a.cache.page_shift);
    // positions that all rows of the tile see: [lo_in, hi_in); that some see: [lo_out, hi_out)
    int lo_out, hi_in, lo_in, hi_out;
    seen_by(a, seq.pos + first / g, cap, &lo_out, &hi_in);
    seen_by(a, seq.pos + last / g, cap, &lo_in, &hi_out);
    const int begin = span.lo + z * share;
    int end = begin + share < span.hi ? begin + share : span.hi;
    if (end > hi_out) end = hi_out;
    int t0 = begin;  // first tile of this workgroup
    if (lo_out > t0) t0 = lo_out & ~(kKeys - 1);

    // this lane's row
    const int part = wave / (NW / PARTS);  // of the elements
    const int r = first + (wave - part * (NW / PARTS)) * 32 + col;
    const bool live = r < rows;
    const int tok = live ? r / g : 0, hg = live ? r - tok * g : 0;
    const int64_t token = seq.t0 + tok;
    const int head = kvh * g + hg;
    int lo = 0, hi = 0;
    if (live) seen_by(a, seq.pos + tok, cap, &lo, &hi);

    bf16x8 q[KSTEPS];
    {
        const uint32_t flip = plan.q_sign < 0 ? 0x80008000u : 0u, keep = (live && plan.q_sign != 0) ? 0xFFFFFFFFu : 0u;
        const uint16_t* src = a.q + token * a.q_stride + (int64_t)head * D + 8 * half;
#pragma unroll
        for (int s = 0; s < KSTEPS; ++s) {
            u32x4_t w = *reinterpret_cast<const u32x4_t*>(src + 16 * s);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (w[i] ^ flip) & keep;
            q[s] = __builtin_bit_cast(bf16x8, w);
        }
    }

    f32x16 o[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;

    const int ps = a.cache.page_shift, pmask = (1 << ps) - 1;
    const int32_t* table = a.seqs.table + sid * a.seqs.table_stride;
    // A wave's rows of a pass lie in one group of 16 positions, and so in one
    // page: its id, and the first row's address in units of rows.
    typedef int Ids __attribute__((ext_vector_type(8)));
    auto page_at = [&](int k) __attribute__((always_inline)) {
        const int p = k >> ps;
        return table[p < a.seqs.max_pages ? p : a.seqs.max_pages - 1];
    };
    auto pages_of = [&](int k0) __attribute__((always_inline)) {
        Ids id = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int n = 0; n < St::PASSES; ++n) id[n] = page_at(k0 + n * St::RPP + wave * St::RPW);
        return id;
    };
    bool some_bad = false;
    const int srow = lane / St::TPR, schunk = lane % St::TPR;
    // what this thread carries of the next tile
    u32x4_t kst[St::PASSES], vst[St::PASSES];
    uint32_t ksc[St::PASSES], vsc[St::PASSES];
    // Loads one half of a tile (k or v); each wave's rows of a pass start at a
    // uniform address, a lane adds a 32-bit offset.
    auto load = [&](const void* half_base, const uint8_t* scales, int k0, const Ids id, u32x4_t (&x)[St::PASSES],
                    uint32_t (&sc)[St::PASSES]) __attribute__((always_inline)) {
        constexpr int64_t EB = FMT == kKvBf16 ? 2 : 1;
#pragma unroll
        for (int n = 0; n < St::PASSES; ++n) {
            const int row0 = n * St::RPP + wave * St::RPW;  // of this wave and pass; one 16-key group
            const int page = ((id[n] < 0) | (id[n] >= a.cache.pages)) ? 0 : id[n];
            const int64_t base = (((int64_t)page * a.cache.heads + kvh) << ps) + ((k0 + row0) & pmask);
            const uint32_t off = (uint32_t)(srow * D * (int)EB + schunk * 16);
            x[n] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(half_base) + base * D * EB + off);
            if constexpr (FMT == kKvMxfp8) sc[n] = (scales + base * (D / 32))[(uint32_t)(srow * (D / 32) + schunk / 2)];
        }
    };
    auto load_tile = [&](int k0, const Ids id) __attribute__((always_inline)) {
        load(a.cache.k, a.cache.ks, k0, id, kst, ksc);
        load(a.cache.v, a.cache.vs, k0, id, vst, vsc);
    };
    // The 16-position groups of a tile whose page is out of range, as bits;
    // bad_pages says whether there are any at all.
    auto bad_groups = [&](int k0) __attribute__((always_inline)) {
        int bad = 0;
        if (some_bad) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int page = page_at(k0 + 16 * i);
                if (k0 + 16 * i < end && (page < 0 || page >= a.cache.pages)) bad |= 1 << i;
            }
        }
        return bad;
    };
    auto masked_tile = [&](int k0, int bad) __attribute__((always_inline)) { return k0 + kKeys > hi_in || k0 < lo_in || k0 + kKeys > end || bad != 0; };
    // A lane's 16 loaded bytes as bf16: one 16-byte chunk, or two decoded ones.
    constexpr int W = FMT == kKvBf16 ? 1 : 2;
    auto decoded = [&](const u32x4_t x, uint32_t scale, u32x4_t (&w)[W]) __attribute__((always_inline)) {
        if constexpr (FMT == kKvBf16) {
            w[0] = x;
        } else {
            w[0] = mx8_to_bf16(x[0], x[1], e8m0_exponent(scale));
            w[1] = mx8_to_bf16(x[2], x[3], e8m0_exponent(scale));
        }
    };
    auto store_k = [&](int number) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < St::PASSES; ++n) {
            const int row = n * St::RPP + wave * St::RPW + srow;
            u32x4_t w[W];
            decoded(kst[n], ksc[n], w);
#pragma unroll
            for (int i = 0; i < W; ++i)
                *reinterpret_cast<u32x4_t*>(k_lds[number & 1] + row * (D * 2) + 16 * T::k_chunk(row, schunk * W + i)) = w[i];
        }
    };
    // In a tile that some row does not see whole, values of positions outside
    // [lo_out, end) and values that are not finite become zeros (a row's zero
    // weight times NaN would be NaN); the latter raise the tile's flag.
    auto store_v = [&](int k0, int number, int bad) __attribute__((always_inline)) {
        const bool edge = masked_tile(k0, bad);
        bool odd = false;
#pragma unroll
        for (int n = 0; n < St::PASSES; ++n) {
            const int row = n * St::RPP + wave * St::RPW + srow;
            u32x4_t w[W];
            decoded(vst[n], vsc[n], w);
            if (edge) {
                const bool keep = (k0 + row < end) & (k0 + row >= lo_out) & !((bad >> (row / 16)) & 1);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if (!keep) w[i] = u32x4_t{0, 0, 0, 0};
                    odd |= take_out_not_finite(w[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < W; ++i)
                *reinterpret_cast<u32x4_t*>(v_lds[number & 1] + row * (D * 2) +
                                            16 * ((schunk * W + i) ^ T::v_swizzle(row))) = w[i];
        }
        if (edge && odd) taken_out = 1;
    };

    if (t0 < end) {
        if (tid == 0) taken_out = bad_pages = 0;
        __syncthreads();
        for (int p = (t0 >> ps) + tid; p <= (end - 1) >> ps; p += 64 * NW) {
            const int page = table[p];
            if (page < 0 || page >= a.cache.pages) bad_pages = 1;
        }
        const Ids id = pages_of(t0);
        load_tile(t0, id);
        Ids id_next = pages_of(t0 + kKeys);
        __syncthreads();
        some_bad = __builtin_amdgcn_readfirstlane(bad_pages) != 0;
        int bad = bad_groups(t0);
        store_k(0);
        store_v(t0, 0, bad);
        __syncthreads();
        int number = 0;
        for (int k0 = t0; k0 < end; k0 += kKeys, ++number) {
            const bool more = k0 + kKeys < end;
            int bad_next = 0;
            if (more) {
                load_tile(k0 + kKeys, id_next);
                bad_next = bad_groups(k0 + kKeys);
                id_next = pages_of(k0 + 2 * kKeys);
            }
            // ---- scores ----
            const uint8_t* kt = k_lds[number & 1];
            f32x16 s[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[b][i] = 0.0f;
#pragma unroll
            for (int t = 0; t < KSTEPS; ++t) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(
                        kt + (b * 32 + col) * (D * 2) + 16 * T::k_chunk(col, 2 * t + half));
                    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), q[t], s[b], 0, 0, 0);
                }
            }
            const bool edge = masked_tile(k0, bad);
            if (edge) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int key = k0 + 32 * b + 8 * (i / 4) + 4 * half + i % 4;
                        if ((bad >> (2 * b + i / 8)) & 1) s[b][i] = __builtin_nanf("");
                        s[b][i] = ((key >= lo) & (key < hi) & (key < end)) ? s[b][i] : -__builtin_inff();
                    }
            }
            // ---- softmax ----
            float top = s[0][0];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[b][i]);
            top *= plan.c;
            if (__any(top > m + kSlack)) {
                const float n = __builtin_fmaxf(m, max_halves(top));
                const float keep = n == m ? 1.0f : exp2_hw(m - n);
                l *= keep;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[d][i] *= keep;
                m = n;
            }
            const float shift = m == -__builtin_inff() ? 0.0f : m;
            u32x4_t p[2 * NB];  // weights of the 16-key steps, as bf16 pairs
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float p0 = exp2_hw(__builtin_fmaf(s[b][i], plan.c, -shift));
                    const float p1 = exp2_hw(__builtin_fmaf(s[b][i + 1], plan.c, -shift));
                    l += p0 + p1;
                    p[2 * b + i / 8][(i / 2) % 4] = pack_bf16(p0, p1);
                }
            // ---- values ----
            const uint8_t* vt = v_lds[number & 1];
            const int kq = (lane & 15) / 4;  // row of this lane in a transpose read
            const uint8_t* vrow = vt + (4 * half + kq) * (D * 2) + 8 * (lane & 1);
            const int vchunk = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
            const int vx = T::v_swizzle(kq);
#pragma unroll
            for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    const int off = 16 * ((4 * (DB * part + d) + vchunk) ^ vx);
                    const u32x2_t v0 = read_column4(vrow + (16 * t) * (D * 2) + off);
                    const u32x2_t v1 = read_column4(vrow + (16 * t + 8) * (D * 2) + off);
                    const u32x4_t v = {v0[0], v0[1], v1[0], v1[1]};
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v),
                                                                   __builtin_bit_cast(bf16x8, p[t]), o[d], 0, 0, 0);
                }
            if (more) {
                store_k(number + 1);
                store_v(k0 + kKeys, number + 1, bad_next);
            }
            bad = bad_next;
            __syncthreads();
        }
        if (taken_out) {
#pragma unroll 1
            for (int k0 = t0; k0 < end; k0 += kKeys) {
                if (!masked_tile(k0, bad_groups(k0))) continue;
#pragma unroll 1
                for (int key = k0; key < k0 + kKeys && key < end; ++key) {
                    const int64_t page = table[key >> ps];
                    if (page < 0 || page >= a.cache.pages) continue;
                    const int64_t row = ((page * a.cache.heads + kvh) << ps) + (key & pmask);
                    const bool sees = (key >= lo) & (key < hi);
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const f32x4 x = not_finite_part<FMT>(a.cache.v, a.cache.vs, row, D, 32 * (DB * part + d) + 2 * i + 4 * half, sees);
#pragma unroll
                            for (int j = 0; j < 4; ++j) o[d][i + j] += x[j];
                        }
                }
            }
        }
    }

    // ---- out ----
    l = sum_halves(l);
    if (!live) return;
    const int64_t at = token * a.heads + head;
    if (shares <= 1) {
        const bool empty = hi <= lo;
        const float inv = empty ? 0.0f : 1.0f / l;
        uint16_t* dst = a.out + at * D + 32 * DB * part + 4 * half;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<u32x2_t*>(dst + 32 * d + 2 * i) =
                    u32x2_t{pack_bf16(o[d][i] * inv, o[d][i + 1] * inv), pack_bf16(o[d][i + 2] * inv, o[d][i + 3] * inv)};
        if (a.lse && half == 0 && part == 0)
            a.lse[at] = empty ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
    } else {
        const int64_t slot = (int64_t)z * a.tokens * a.heads + at;
        float* dst = plan.part_o + slot * D + 32 * DB * part + 4 * half;
        if (t0 < end) {
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<f32x4*>(dst + 32 * d + 2 * i) = f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
        }
        if (half == 0 && part == 0) {
            plan.part_m[slot] = m;
            plan.part_l[slot] = l;
        }
    }
}

template <int D, int NW>
static void launch_dim(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
    const int64_t tiles = a.tokens * p.group / (32 * NW / kParts<D>) + a.seqs.seqs;
    const dim3 grid((unsigned)(tiles * a.cache.heads), (unsigned)p.splits), block(64 * NW);
    if (a.cache.fmt == kKvMxfp8) hipLaunchKernelGGL((attn_chunk_kernel<D, kKvMxfp8, NW>), grid, block, 0, st, a, p);
    else hipLaunchKernelGGL((attn_chunk_kernel<D, kKvBf16, NW>), grid, block, 0, st, a, p);
}

bool launch_attn_chunk(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
    switch (a.cache.dim) {
        case 64: launch_dim<64, 4>(a, p, st); return true;
        case 128:
            if (p.waves == 8) launch_dim<128, 8>(a, p, st);
            else launch_dim<128, 4>(a, p, st);
            return true;
        case 256:
            if (p.waves == 8) launch_dim<256, 8>(a, p, st);
            else launch_dim<256, 4>(a, p, st);
            return true;
    }
    return false;
}

}  // namespace mxq
