// kv_device.hpp -- device-side building blocks of the kernels that work on a
// paged cache: finding a token's sequence, and reading bf16 or fp32 rows.
#pragma once

#include "kv_kernels.hpp"
#include "mxq_device.hpp"
#include "rows_core.hpp"

namespace mxq {

// Number of sequences whose end cu_q[s + 1] lies at or before row t: the index
// of the sequence that holds row t, or seqs if t lies behind the last one.
// Called by whole waves (each of the 64 lanes takes every 64th sequence).
__device__ __forceinline__ int sequence_of(const KvSeqs& q, int t) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int i = 0; i < q.seqs; i += 64) {
        const bool before = i + lane < q.seqs && q.cu_q[i + lane + 1] <= t;
        n += __builtin_popcountll(__ballot(before));
    }
    return n;
}

// 8 consecutive elements at p (16-byte aligned) as fp32.
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t off, float (&v)[8]) {
    if constexpr (BF16) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(base) + off);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo_to_f32(w[i]);
            v[2 * i + 1] = bf16_hi_to_f32(w[i]);
        }
    } else {
        typedef float f32x4_t __attribute__((ext_vector_type(4)));
        const f32x4_t* p = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(base) + off);
        const f32x4_t a = p[0], b = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const bf16x2_t b = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, b);
}

// 8 fp32 values rounded to bf16 (nearest, ties to even), or as they are.
template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t off, const float (&v)[8]) {
    if constexpr (BF16) {
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(base) + off) =
            u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    } else {
        typedef float f32x4_t __attribute__((ext_vector_type(4)));
        f32x4_t* p = reinterpret_cast<f32x4_t*>(static_cast<float*>(base) + off);
        p[0] = f32x4_t{v[0], v[1], v[2], v[3]};
        p[1] = f32x4_t{v[4], v[5], v[6], v[7]};
    }
}

}  // namespace mxq
