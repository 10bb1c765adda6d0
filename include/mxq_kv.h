/*
 * mxq_kv.h -- C ABI of libmxq, second part: what a decode layer runs between
 * its QKV projection and its output projection on AMD Instinct MI355X
 * (gfx950).  Rotary positions, appending a step's keys and values to a paged
 * cache, and attention of the new tokens over that cache.  The cache is the
 * other stream that decode reads at every token ("The memory wall" section of
 * the "MLxcel 0.8 release" post, slide 15 of the Strix Halo talk), and it is
 * kept in bf16 or in the MXFP8 blocks of mxq.h, decoded exactly inside the
 * kernel.
 *
 * Inputs are what mxq_gemv and mxq_gemm write (fp32 or bf16 rows, strided, so
 * that q, k and v may be slices of one fused QKV row); the attention output is
 * what they read (bf16 rows).
 *
 * Conventions are those of mxq.h: device pointers owned by the caller, work
 * enqueued on `stream`, validation on the host first (FORMAT, NULLPTR, SHAPE,
 * ALIGN, UNSUPPORTED, DEVICE, in this order) with nothing launched by a
 * rejected call, 64-bit offsets, no allocation, no atomics, deterministic
 * results.  The parameter structures are read during the call only.
 *
 * Paged cache: k and v hold rows of head_dim elements, laid out as
 *   [num_pages][kv_heads][page_size][head_dim]
 * in bf16 (MXQ_KV_BF16, 2 bytes an element), or as E4M3 codes of that shape
 * with E8M0 scales [num_pages][kv_heads][page_size][head_dim / 32]
 * (MXQ_KV_MXFP8): the weight layout of mxq.h with num_pages * kv_heads *
 * page_size rows, so mxq_dequant reads a cache too.
 *
 * Sequences: sequence s has its new tokens in rows cu_q[s] .. cu_q[s+1] - 1 of
 * the token-major tensors, and kv_lens[s] positions in the cache, the new ones
 * included; its i-th new token is at position
 *   p = kv_lens[s] - (cu_q[s+1] - cu_q[s]) + i
 * and position p is row p % page_size of page block_table[s][p / page_size].
 * cu_q does not decrease.  Rows before cu_q[0] or from cu_q[seqs] on belong to
 * no sequence: their outputs are left as they were.
 */
#ifndef MXQ_KV_H
#define MXQ_KV_H

#include "mxq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Cache formats (an int, as mxq_format_t): bf16, or MXFP8 blocks. */
enum mxq_kv_format { MXQ_KV_BF16 = 0, MXQ_KV_MXFP8 = MXQ_FMT_MXFP8 };

/* Pairs of rotary elements: (i, i + rot_dim/2) or (2i, 2i + 1). */
enum mxq_rope_layout { MXQ_ROPE_HALF = 0, MXQ_ROPE_INTERLEAVED = 1 };

/* How inverse frequencies are stretched for contexts longer than the trained one. */
enum mxq_rope_scaling {
    MXQ_ROPE_NONE = 0,   /* f_i = theta^(-2i / rot_dim) */
    MXQ_ROPE_LINEAR = 1, /* f_i / factor */
    MXQ_ROPE_NTK = 2,    /* theta * factor^(rot_dim / (rot_dim - 2)) in place of theta */
    MXQ_ROPE_YARN = 3,   /* f_i / factor where a full turn is longer than the trained context / low, f_i where it is
                            shorter than context / high, a linear ramp over i between; mscale = 0.1 ln(factor) + 1 */
    MXQ_ROPE_BANDS = 4   /* as YARN with a ramp linear in context / wavelength, and mscale 1 */
};

/* Rotation: mscale multiplies the rotated elements (1 if there is no long-context scaling). */
typedef struct {
    const float *inv_freq; /* fp32 [rot_dim / 2] on the device; may be NULL if rot_dim is 0 */
    int64_t rot_dim;       /* 0 .. head_dim, a multiple of 16: the first rot_dim elements of a head turn */
    int32_t layout;        /* enum mxq_rope_layout */
    float mscale;
} mxq_rope_params_t;

/* A paged cache. */
typedef struct {
    int32_t format;     /* enum mxq_kv_format */
    int32_t reserved;   /* 0 */
    void *k, *v;        /* 16-byte aligned */
    uint8_t *k_scales, *v_scales; /* MXFP8: E8M0 scales, 8-byte aligned; bf16: NULL */
    int64_t num_pages, page_size, kv_heads, head_dim;
} mxq_kv_cache_t;

/* The sequences of one step.  Values are read on the device and not trusted: see each entry point. */
typedef struct {
    const int32_t *block_table; /* [seqs][max_pages], rows table_stride int32 apart */
    const int32_t *cu_q;        /* [seqs + 1] */
    const int32_t *kv_lens;     /* [seqs] */
    int64_t seqs, max_pages, table_stride;
} mxq_kv_seqs_t;

#define MXQ_KV_MAX_SEQS 4096
#define MXQ_KV_MAX_PAGE 1024

/*
 * Inverse frequencies of a rotation, computed on the HOST in double and
 * rounded once: the table a program makes when a model loads.  inv_freq and
 * mscale are HOST pointers.
 *   scaling  enum mxq_rope_scaling (else MXQ_E_FORMAT)
 *   rot_dim  even, 2 .. 1024;  theta > 1;  factor >= 1
 *   context  the trained context length, > 0, and low < high (both > 0): YARN
 *            and BANDS only (turns per trained context below which a
 *            frequency is divided by factor, above which it is kept)
 */
mxq_status_t mxq_rope_inv_freq(int scaling, int64_t rot_dim, double theta, double factor, double context, double low,
                               double high, float *inv_freq, float *mscale);

/*
 * Rotary positions.  For token t, head h and pair i < rot_dim / 2 with
 * elements (a, b) = (x[i], x[i + rot_dim/2]) or (x[2i], x[2i + 1]) and the
 * angle w = positions[t] * inv_freq[i],
 *   y_a = mscale * (a cos w - b sin w)      y_b = mscale * (b cos w + a sin w)
 * and y = x in the elements from rot_dim on.  The angle is reduced in double
 * (exact product of a 32-bit position and an fp32 frequency up to 2^-53), so
 * positions far out lose nothing; the rotation is fp32, rounded once.
 *   x          fp32 or bf16 (x_dtype, enum mxq_out) [tokens][heads][head_dim],
 *              tokens x_stride elements apart
 *   y          fp32 or bf16 (y_dtype), tokens y_stride elements apart; y may
 *              be x with the same type and stride (in place), otherwise the
 *              two must not overlap
 *   positions  int32 [tokens]
 *   head_dim   a multiple of 16, up to 1024;  strides at least heads *
 *              head_dim and multiples of 16 bytes;  x, y 16-byte aligned
 *   tokens, heads * head_dim < 2^31;  strides up to 2^28
 */
mxq_status_t mxq_rope(const void *x, mxq_out_t x_dtype, void *y, mxq_out_t y_dtype, const int32_t *positions,
                      const mxq_rope_params_t *rope, int64_t tokens, int64_t heads, int64_t head_dim,
                      int64_t x_stride, int64_t y_stride, void *stream);

/*
 * Appends the new tokens' keys and values to the cache, rotating the keys on
 * the way, and rotates the queries: one launch between the QKV projection and
 * the attention.  A rotated key (and a value as it is) goes from fp32 to the
 * cache's format in one rounding: to bf16, or per 32 elements by the MX
 * conversion of mxq_quantize; 32 elements with an infinity or a NaN among them
 * get the scale byte 255, which reads as NaN.
 *   k, v       fp32 or bf16 (x_dtype) [tokens][kv_heads][head_dim], k_stride
 *              and v_stride elements apart
 *   q, q_out   both or neither: queries [tokens][heads][head_dim] (q_stride)
 *              in x_dtype, and the rotated queries, bf16 [tokens][heads]
 *              [head_dim], contiguous.  q_out may not overlap the inputs.
 *   positions  int32 [tokens]: the positions to rotate by; NULL: the tokens'
 *              positions p in the cache
 *   head_dim   64, 128 or 256;  page_size a power of two, 16 ..
 *              MXQ_KV_MAX_PAGE;  seqs up to MXQ_KV_MAX_SEQS;  tokens up to
 *              2^22;  heads up to 65536;  tokens * heads up to 2^25, seqs *
 *              kv_heads up to 2^22;  max_pages * page_size up to 2^30;
 *              strides up to 2^36, otherwise as in mxq_rope, as the pointers
 * A token whose p is negative or beyond the table, or whose page is outside
 * [0, num_pages), stores nothing in the cache (its query is still rotated).
 * Two sequences that append to one page must not do so at the same row.
 */
mxq_status_t mxq_kv_append(const void *q, const void *k, const void *v, mxq_out_t x_dtype, uint16_t *q_out,
                           const int32_t *positions, const mxq_rope_params_t *rope, const mxq_kv_cache_t *cache,
                           const mxq_kv_seqs_t *seqs, int64_t tokens, int64_t heads, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, void *stream);

/*
 * Attention of the new tokens over the paged cache, which already holds their
 * own keys and values: decode (one new token a sequence), a chunk of a prompt
 * over what is cached, a whole prompt, or a mix.  Query head h reads key/value
 * head h / (heads / kv_heads).  The token at position p sees the positions
 *   j <= p,  and j > p - window if window > 0:
 *   out = sum_j softmax_j(scale * q . k_j) v_j
 *   lse = log sum_j exp(scale * q . k_j)
 * with fp32 scores, statistics and sums, one pass over the keys.  MXFP8 rows
 * are decoded to bf16: exact from scale byte 3 on, and below that rounded to
 * bf16's smallest subnormal steps; scale byte 255 is NaN.  The softmax
 * weights enter the value product as bf16 (long chunks) or as a pair of bf16
 * (few rows); both accumulate in fp32.
 *   q      bf16 [tokens][heads][head_dim], tokens q_stride elements apart
 *   out    bf16 [tokens][heads][head_dim], contiguous
 *   lse    fp32 [tokens][heads], or NULL
 *   max_q  the largest number of new tokens of a sequence, as a hint for the
 *          choice of kernel: any value >= 1 is correct
 *   window 0: no window
 *   workspace  mxq_paged_attn_workspace(...) bytes for the same sizes, 16-byte
 *          aligned; NULL is allowed if that is 0.  Each call writes what it
 *          reads there: no clearing, and calls on one stream may share it;
 *          calls that overlap in time may not.
 *   limits on heads (a multiple of kv_heads), pages, sequences and strides as
 *   in mxq_kv_append; |scale| up to 2^100;  out must not overlap q
 * A row that sees no position (kv_lens[s] smaller than its new tokens) gets
 * zeros and lse -inf.  kv_lens is taken as at most max_pages * page_size.  A
 * row that sees a position whose page is outside [0, num_pages) gets NaN.
 * What lies in cache rows that a token does not see, NaN and infinities
 * included, does not reach its output.  An infinite value that it sees makes
 * that element infinite (NaN where the other sign's meets it, or where its
 * weight is below 2^-126).
 */
mxq_status_t mxq_paged_attn(const uint16_t *q, uint16_t *out, float *lse, const mxq_kv_cache_t *cache,
                            const mxq_kv_seqs_t *seqs, int64_t tokens, int64_t heads, int64_t q_stride, float scale,
                            int64_t window, int64_t max_q, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace of mxq_paged_attn for these sizes (pointers are not read), or -1 if the sizes are invalid. */
int64_t mxq_paged_attn_workspace(const mxq_kv_cache_t *cache, const mxq_kv_seqs_t *seqs, int64_t tokens,
                                 int64_t heads, int64_t max_q);

/* Version of this header: 1. */
int mxq_kv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_KV_H */
