// attn_core.hpp -- what the two attention kernels (attn_chunk.hip for tiles of
// many query rows, attn_decode.hip for few) share: which rows and keys a
// workgroup owns, the split of the keys, and the partial results.
//
// A row is one query head of one new token; the rows of a sequence that share
// a key/value head are numbered r = token * group + head in group, so that all
// of them read a key once.
#pragma once

#include "kv_device.hpp"

namespace mxq {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Rows of a tile of the decode kernel.  Where both kernels run, it takes the
// sequences of one such tile per key/value head, and the chunk kernel the others.
constexpr int kFewRows = 16;
// Key tiles are split in multiples of this many positions.
constexpr int kSplitUnit = 64;

struct AttnPlan {
    int group;      // query heads per key/value head
    float c;        // |scale| * log2 e: scores are kept in powers of two
    int q_sign;     // -1, 0, 1: the sign of scale, applied to the queries
    int splits;     // chunk kernel: shares of the keys of a sequence, at most
    int waves;      // chunk kernel: waves of a workgroup, 32 rows each
    int target;     // decode kernel: workgroups to split the work of a call into, about; 0: no split
    int enough;     // decode kernel: tiles that fill the device unsplit
    int least;      // positions of a share, at least; a multiple of kSplitUnit
    int filter;     // 1: this kernel takes only the sequences on its side of kFewRows
    float* part_o;  // unnormalised sums of the shares: chunk [splits][tokens * heads][dim], decode [slot][16][dim]
    float* part_m;  // their running maxima (powers of two)
    float* part_l;  // their sums of weights
};

// A sequence's new tokens as the kernels use them: rows t0 .. t0 + n - 1 of
// the token-major tensors, the first at position pos.  Whatever the metadata
// holds, the rows lie inside the tensors.
struct Seq {
    int t0, n;
    int64_t pos;
};
__device__ __forceinline__ Seq sequence(const KvSeqs& q, int64_t tokens, int s) {
    const int t0 = q.cu_q[s], t1 = q.cu_q[s + 1];
    Seq r;
    r.t0 = t0;
    const int64_t n = t0 < 0 ? 0 : (int64_t)(t1 < tokens ? t1 : tokens) - t0;
    r.n = n > 0 ? (int)n : 0;
    r.pos = (int64_t)q.lens[s] - ((int64_t)t1 - t0);
    return r;
}

// The rows that a kernel takes of a sequence of n new tokens.
template <bool FEW>
__device__ __forceinline__ int rows_taken(const AttnPlan& p, int n) {
    const int rows = n * p.group;
    return (p.filter && (rows <= kFewRows) != FEW) ? 0 : rows;
}

// Maximum and sum over the two halves of a wave (lane l and l + 32), and over
// pairs of 16-lane rows (l and l ^ 16); every lane ends with the result, in a
// fixed order of operands.  (A vector's element goes through a variable before
// it is bit-cast: the compiler takes element 0 otherwise.)
__device__ __forceinline__ float max_halves(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t x = r[0], y = r[1];
    return __builtin_fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
__device__ __forceinline__ float sum_halves(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t x = r[0], y = r[1];
    return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}
__device__ __forceinline__ float max_rows16(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t x = r[0], y = r[1];
    return __builtin_fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
__device__ __forceinline__ float sum_rows16(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t x = r[0], y = r[1];
    return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}

// Maximum over the lanes of a wave.
__device__ __forceinline__ float wave_max(float v) {
    v = __builtin_fmaxf(v, dpp_f32<kDppQuadXor1>(v));
    v = __builtin_fmaxf(v, dpp_f32<kDppQuadXor2>(v));
    v = __builtin_fmaxf(v, dpp_f32<kDppRowHalfMirror>(v));
    v = __builtin_fmaxf(v, dpp_f32<kDppRowMirror>(v));
    return max_halves(max_rows16(v));
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // last lane of rows 0, 2 into rows 1, 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 into the upper half
    return v;
}
__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Tile `index` of the tiles of BM rows of all sequences: its sequence, and its
// number there.  One sequence per lane, 64 at a time.
template <int BM, bool FEW>
__device__ __forceinline__ bool find_tile(const AttnArgs& a, const AttnPlan& p, int index, int* seq, int* tile) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int base = 0; base < a.seqs.seqs; base += 64) {
        int n = 0;
        if (base + lane < a.seqs.seqs) {
            const int t0 = a.seqs.cu_q[base + lane], t1 = a.seqs.cu_q[base + lane + 1];
            const int64_t m = t0 < 0 ? 0 : (int64_t)(t1 < a.tokens ? t1 : a.tokens) - t0;
            n = (rows_taken<FEW>(p, m > 0 ? (int)m : 0) + BM - 1) / BM;
        }
        const int sum = wave_scan(n);
        const uint64_t past = __ballot(before + sum > index);
        if (past) {
            const int l = __builtin_ctzll(past);
            *seq = base + l;
            *tile = index - before - (lane_value(sum, l) - lane_value(n, l));
            return true;
        }
        before += lane_value(sum, 63);
    }
    return false;
}

// Positions of a sequence that its new tokens see, [lo, hi), with lo on a
// kSplitUnit boundary.
struct Span {
    int lo, hi;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, const AttnPlan& p, const Seq& s) {
    const int64_t cap = (int64_t)a.seqs.max_pages << a.cache.page_shift;
    int64_t hi = s.pos + s.n;
    hi = hi < 0 ? 0 : hi > cap ? cap : hi;
    int64_t lo = a.window > 0 ? s.pos - a.window + 1 : 0;
    lo = lo < 0 ? 0 : lo > hi ? hi : lo;
    return {(int)lo & ~(kSplitUnit - 1), (int)hi};
}

// The chunk kernel's split of a sequence's positions: shares of one length, a
// multiple of kSplitUnit, at most plan.splits of them.
__device__ __forceinline__ int share_of(const AttnPlan& p, const Span& s, int* shares) {
    const int units = (s.hi - s.lo + kSplitUnit - 1) / kSplitUnit;
    int per = (units + p.splits - 1) / p.splits;
    if (per < p.least / kSplitUnit) per = p.least / kSplitUnit;
    *shares = (units + per - 1) / per;
    return per * kSplitUnit;
}

// The decode kernel's split: every share of every sequence has the same length,
// that of the call's tiles of 16 rows times their positions divided by
// plan.target (but plan.least at least), so that workgroups carry equal work
// whatever the lengths are.  A call has at most plan.target / kv_heads + tiles
// shares; those of tiles that are split (at most 2 plan.target / kv_heads) have
// a slot each for their partial result.  Where the tiles alone fill the device
// and no length is far above the mean, nothing is split: 32 sequences of 8000
// positions, 40/8 heads of 128 in bf16, take 157 us whole and 171 us in 2304
// shares; 64 sequences of 165 to 16000 positions (MXFP8) 258 us whole and 207.
// A tile a compute unit fills it with heads of 128 in bf16; rows of fewer bytes
// need two (the same 32 sequences in MXFP8: 124 us whole, 109 in shares; heads
// of 64 in MXFP8: 88 and 61; 64 of those: 108 whole, 109 in shares).
struct Work {
    int sid, tile, z;     // sequence, tile of it, share of the tile
    int shares, share;    // of the tile; their length
    int slot;             // first share's slot of the tile; -1: not split
};
// Share `index` of the call's shares (BY_TILE: the tile `index` of its tiles).
template <bool BY_TILE>
__device__ __forceinline__ bool find_work(const AttnArgs& a, const AttnPlan& p, int index, Work* w) {
    const int lane = threadIdx.x & 63;
    // (tiles, units of the positions) of this lane's sequence
    auto load = [&](int base, int* tiles, int* units) __attribute__((always_inline)) {
        *tiles = *units = 0;
        if (base + lane < a.seqs.seqs) {
            const Seq s = sequence(a.seqs, a.tokens, base + lane);
            const Span span = span_of(a, p, s);
            *tiles = (rows_taken<true>(p, s.n) + kFewRows - 1) / kFewRows;
            *units = (span.hi - span.lo + kSplitUnit - 1) / kSplitUnit;
        }
    };
    int tiles0, units0;  // the first 64 sequences' stay in registers
    load(0, &tiles0, &units0);
    float total = 0.0f, count = 0.0f, longest = 0.0f;
    for (int base = 0; base < a.seqs.seqs; base += 64) {
        int tiles = tiles0, units = units0;
        if (base) load(base, &tiles, &units);
        total += group_sum<64>((float)tiles * (float)units);
        count += group_sum<64>((float)tiles);
        longest = __builtin_fmaxf(longest, wave_max(tiles ? (float)units : 0.0f));
    }
    const float heads = (float)a.cache.heads;
    float want = longest;
    if (p.target > 0 && (count * heads < (float)p.enough || longest * count > 1.25f * total))
        want = __builtin_fmaxf(__builtin_ceilf(total * heads / (float)p.target), (float)(p.least / kSplitUnit));
    const int per = __builtin_amdgcn_readfirstlane((int)__builtin_fminf(__builtin_fmaxf(want, 1.0f), 16777216.0f));
    int before = 0, slots = 0;
    for (int base = 0; base < a.seqs.seqs; base += 64) {
        int tiles = tiles0, units = units0;
        if (base) load(base, &tiles, &units);
        const int shares = units > per ? (units + per - 1) / per : 1;
        const int n = BY_TILE ? tiles : tiles * shares, used = shares > 1 ? tiles * shares : 0;
        const int sum = wave_scan(n), sum_used = wave_scan(used);
        const uint64_t past = __ballot(before + sum > index);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int at = index - before - (lane_value(sum, l) - lane_value(n, l));
            w->sid = base + l;
            w->shares = lane_value(shares, l);
            w->share = per * kSplitUnit;
            w->tile = BY_TILE ? at : at / w->shares;
            w->z = BY_TILE ? 0 : at - w->tile * w->shares;
            w->slot = w->shares > 1 ? slots + lane_value(sum_used, l) - lane_value(used, l) + w->tile * w->shares : -1;
            return true;
        }
        before += lane_value(sum, 63);
        slots += lane_value(sum_used, 63);
    }
    return false;
}

// Positions [lo, hi) that the token at position p sees.
__device__ __forceinline__ void seen_by(const AttnArgs& a, int64_t p, int cap, int* lo, int* hi) {
    const int64_t h = p + 1 < 0 ? 0 : p + 1 > cap ? cap : p + 1;
    int64_t l = a.window > 0 ? p - a.window + 1 : 0;
    l = l < 0 ? 0 : l > h ? h : l;
    *lo = (int)l;
    *hi = (int)h;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// 4 bf16 of a column of a row-major LDS tile: each 16-lane group reads a
// 4 x 16 block (lane l its elements 4 (l % 4) .. of row l / 4) and lane l gets
// column l of the 4 rows.
__device__ __forceinline__ u32x2_t read_column4(const void* lds) {
    typedef __attribute__((address_space(3))) s16x4* p3;
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((p3)(lds)));
}

// Zeroes the bf16 in v that are infinite or NaN; whether there were any.
__device__ __forceinline__ bool take_out_not_finite(u32x4_t& v) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool lo = (v[i] & 0x7F80u) == 0x7F80u, hi = (v[i] & 0x7F800000u) == 0x7F800000u;
        v[i] &= (lo ? 0u : 0x0000FFFFu) | (hi ? 0u : 0xFFFF0000u);
        any |= lo | hi;
    }
    return any;
}

// 8 E4M3 codes (two dwords) with their block's E8M0 byte -> 8 bf16.
__device__ __forceinline__ u32x4_t mx8_to_bf16(uint32_t c0, uint32_t c1, float sexp) {
    const uint32_t c[2] = {c0, c1};
    uint32_t p[4];
    decode_dwords_scaled<kMXFP8, 2>(c, sexp, p);
    return u32x4_t{p[0], p[1], p[2], p[3]};
}

// Elements e .. e + 3 (e a multiple of 4) of a row of the cache's values where
// they are infinite or NaN and the caller's row sees them, else 0.
template <int FMT>
__device__ __forceinline__ f32x4 not_finite_part(const void* v, const uint8_t* scales, int64_t row, int dim, int e,
                                                 bool sees) {
    u32x2_t w;
    if constexpr (FMT == kKvBf16) {
        w = *reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(v) + row * dim + e);
    } else {
        const uint32_t c = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(v) + row * dim + e);
        const u32x4_t d = mx8_to_bf16(c, 0u, e8m0_exponent(scales[row * (dim / 32) + e / 32]));
        w = u32x2_t{d[0], d[1]};
    }
    f32x4 x = {bf16_lo_to_f32(w[0]), bf16_hi_to_f32(w[0]), bf16_lo_to_f32(w[1]), bf16_hi_to_f32(w[1])};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float e = x[i];
        const uint32_t b = __builtin_bit_cast(uint32_t, e);
        x[i] = __builtin_bit_cast(float, (sees & ((b & 0x7F800000u) == 0x7F800000u)) ? b : 0u);
    }
    return x;
}

// Tiles of the decode kernel, at most (a sequence that passes the filter is
// one tile), and their shares.
inline int64_t decode_tiles(const AttnArgs& a, const AttnPlan& p) {
    return p.filter ? a.seqs.seqs : a.tokens * p.group / kFewRows + a.seqs.seqs;
}
inline int64_t decode_shares(const AttnArgs& a, const AttnPlan& p) {
    return decode_tiles(a, p) + p.target / a.cache.heads + 1;
}

bool launch_attn_chunk(const AttnArgs& a, const AttnPlan& p, hipStream_t st);
bool launch_attn_decode(const AttnArgs& a, const AttnPlan& p, hipStream_t st);

}  // namespace mxq
