/*
 * nvfp4_attention.h -- C ABI of the attention operators of libnvfp4_amd.so: rotary
 * positions with several axes, a paged cache of keys and values in NVFP4, attention of
 * single tokens over that cache, and attention of whole prompts.
 *
 * Status codes and conventions (device pointers, 16-byte alignment of tensors, caller-
 * allocated outputs, argument checks before anything is enqueued, no host
 * synchronisation, no allocation, no state between calls) are those of nvfp4.h.  No call
 * records a memset, so all of them can be captured into a HIP graph.
 *
 * Rows: a tensor [t, heads, d] has its heads one after the other and `stride` elements
 * from token to token (heads * d where it is contiguous; more where it is a part of a
 * wider one, such as the q, k or v of a fused projection): a multiple of 8, at most
 * NVFP4_ATTENTION_MAX_STRIDE.
 *
 * The cache:
 *   kv:    [pages, 2, heads, page, d/2] bytes, packed e2m1, the keys' rows and then the
 *          values'; element 2i of a row in the low nibble of its byte i.
 *   kv_sf: [pages, 2, heads, d/16, page] bytes, one ue4m3 scale per 16 elements of a row.
 *   kv_gs: [2] fp32, the global scales of keys and values (448 * 6 / amax of what the cache
 *          is to hold, as nvfp4_quantize's in STATIC mode).  An element is
 *          e2m1 * ue4m3 / kv_gs.
 * A slot is (page index) * page + (position within the page).  A sequence's position i
 * lies on page block_table[i / page].  page is a power of two from 16 to
 * NVFP4_KV_MAX_PAGE, d a multiple of 16 up to NVFP4_KV_MAX_DIM.  Bytes no call has
 * written are never used: a cache need not be cleared.
 */
#ifndef NVFP4_ATTENTION_H
#define NVFP4_ATTENTION_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits (NVFP4_UNSUPPORTED beyond them, NVFP4_BAD_SHAPE for strides).  Every workgroup finds its
 * sequence by going over all lengths or offsets, 64 at a time, so a call's time has a part that grows with the
 * square of the batch: 1024 sequences of up to 100 tokens, 8 heads, decode in 111 us, 4096 in 928, 8192
 * in 3180; 1024 prompts of 60, 8 heads, in 185 us, 4096 in 1480.  Batches of several thousand are faster in
 * calls of about a thousand. */
#define NVFP4_ROPE_MAX_AXES 4
#define NVFP4_ROPE_MAX_DIM 1024
#define NVFP4_KV_MAX_DIM 256
#define NVFP4_KV_MAX_PAGE 4096
#define NVFP4_ATTENTION_MAX_STRIDE (1 << 22)
#define NVFP4_ATTENTION_MAX_BATCH 65536
#define NVFP4_ATTENTION_MAX_TOKENS 64

/*
 * Rotary positions with several axes (text: one; an image or a video: height and width,
 * or time, height and width), in one launch for all heads of a row.  Pair i of the
 * sum(sections) pairs belongs to the axis whose section it falls into; with
 *   angle = positions[axis, token] * inv_freq[i]
 * formed in 64 bits, the pair (x1, x2) becomes
 *   (x1 cos - x2 sin, x2 cos + x1 sin),
 * computed in fp32 and rounded once to bf16.  The pair is (x[i], x[i + pairs]) of a head, or
 * (x[2i], x[2i + 1]) with interleaved != 0.  Elements from 2 * pairs on are copied.
 *   x: [t, heads, d] bf16, x_stride; out: the same shape, out_stride; out may be x (with
 *   the same stride), but may not overlap it otherwise.
 *   positions: [axes, t] int32; inv_freq: [pairs] fp32 (radians a position).
 *   sections: `axes` numbers of pairs, in HOST memory, read before the call returns.
 * Requires 1 <= axes <= 4, sections >= 0, their sum positive, even and at most
 * d / 2, d a multiple of 16, t * heads * d at most 2^36.
 */
int rope_axes(const void* x, int64_t x_stride, void* out, int64_t out_stride, int64_t t, int64_t heads, int64_t d,
              const int32_t* positions, const float* inv_freq, const int32_t* sections, int axes, int interleaved,
              void* stream);

/*
 * Quantizes rows of keys and values into the cache: row i of k and v, bit for bit as
 * nvfp4_quantize in STATIC mode with kv_gs, goes to slots[i].  A slot outside
 * [0, pages * page) (-1 by custom: a row of padding) is passed over.  Slots of one call
 * are distinct; other bytes of the cache keep their values.
 *   k, v: [t, heads, d] bf16 with k_stride, v_stride, at most 2^35 elements each;
 *   slots: [t] int32.
 */
int nvfp4_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t t, int64_t heads,
                    int64_t d, const int32_t* slots, const float* kv_gs, uint8_t* kv, uint8_t* kv_sf, int64_t pages,
                    int64_t page, void* stream);

/*
 * The rows of slots[i] as bf16: bf16((e2m1 * ue4m3) / kv_gs), the quotient rounded to fp32
 * first.  For a cached prefix that a prompt's attention reads.  Rows of slots outside
 * [0, pages * page) are left as they were.
 *   k, v: [t, heads, d] bf16 with k_stride, v_stride, at most 2^35 elements each, written.
 */
int nvfp4_kv_read(const uint8_t* kv, const uint8_t* kv_sf, const float* kv_gs, int64_t pages, int64_t page,
                  const int32_t* slots, int64_t t, int64_t heads, int64_t d, void* k, int64_t k_stride, void* v,
                  int64_t v_stride, void* stream);

/* Parts of split sequences that the workspace holds: 16 rows of d (rounded up to 64, 128 or
 * 256) fp32 sums, their maximum and sum each. */
#define NVFP4_ATTENTION_MAX_SLOTS 2048
#define NVFP4_ATTENTION_WS_BYTES(b, d)                 \
    ((8 * (int64_t)(b) + 255) / 256 * 256 +            \
     (int64_t)NVFP4_ATTENTION_MAX_SLOTS * 64 * (((d) <= 64 ? 64 : (d) <= 128 ? 128 : 256) + 2))

/*
 * Attention of t new tokens a sequence (1, or a few drafted ones) over the cache, which
 * holds them already: with L = lengths[i] (clamped to [0, table_pages * page]), token j of
 * sequence i sees the positions below L - (t - 1 - j), and for each of its heads h
 *   out = sum_p softmax_p(scale * q . K_p) V_p,   KV head h / (q_heads / heads).
 * A token that sees nothing gets zeros (and lse = -inf).  Scores times log2(e) have to lie within
 * fp32's range (this holds for attention_prefill too).  Pages outside [0, pages) are
 * passed over as if their positions were not seen.  The keys and values are
 * exact; q enters the products as fp16 scaled by a power of two per head (exact, but off by up to
 * 2^-39 of the head's largest where it is below 2^-28 of it), the probabilities as fp16 (off by
 * 2^-11 of themselves, or, below 2^-26 of the largest, by 2^-37 of it); sums are fp32.  The tokens
 * of long sequences are split over workgroups, whose parts a second launch joins; how, depends on
 * the lengths, which are read on the device (a captured graph follows them), and on the width of
 * the table: one far wider than the longest sequence costs up to a quarter (16 of 500 tokens: 9.2
 * us, with a table for 65536 11.7).  Results are the same on every call.
 *   q: [b, t, q_heads, d] bf16 with q_stride from token to token; block_table:
 *   [b, table_pages] int32 (entries past a sequence's last page are not read); lengths: [b]
 *   int32; out: [b, t, q_heads, d] bf16; lse: NULL or [b, t, q_heads] fp32,
 *   log(sum exp(scale * q . K_p)).
 *   workspace: workspace_bytes >= NVFP4_ATTENTION_WS_BYTES(b, d), 16-byte aligned; contents
 *   ignored on entry, undefined on exit; calls that share one must not overlap.
 * Requires q_heads a multiple of heads, 0 < scale <= 2e38, t at most
 * NVFP4_ATTENTION_MAX_TOKENS, b at most NVFP4_ATTENTION_MAX_BATCH, b * t * q_heads at most
 * 2^23, table_pages * page at most 2^30.
 */
int nvfp4_attention_decode(const void* q, int64_t q_stride, int64_t b, int64_t t, int64_t q_heads, const uint8_t* kv,
                           const uint8_t* kv_sf, const float* kv_gs, int64_t heads, int64_t d, int64_t pages,
                           int64_t page, const int32_t* block_table, int64_t table_pages, const int32_t* lengths,
                           float scale, void* out, float* lse, void* workspace, int64_t workspace_bytes,
                           void* stream);

/* A workspace of attention_prefill that suffices for all sizes. */
#define NVFP4_ATTENTION_PREFILL_WS_BYTES(d) \
    ((int64_t)512 * 129 * 4 * (((d) <= 64 ? 64 : (d) <= 128 ? 128 : 256) + 4))

/*
 * Attention of whole prompts, packed one after the other: sequence i has the rows
 * cu_q[i] .. cu_q[i + 1] - 1 of q and the keys cu_k[i] .. cu_k[i + 1] - 1, which may reach
 * further back (a cached prefix).  With n rows and m keys, row r sees all keys, or with
 * causal != 0 the keys up to r + m - n; head h of q uses KV head h / (q_heads / heads).
 *   out = sum_p softmax_p(scale * q . k_p) v_p,
 * zeros (and lse = -inf) for a row that sees nothing.  What a row does not see has no
 * effect on it, whatever its values.  Rows of q outside all sequences are left as they were.
 * Probabilities, one at most, are rounded to bf16 for their product with v; sums are fp32 (and
 * divided by the probabilities' sum, that of the unrounded ones, at the end).
 *   q: [tq, q_heads, d], k, v: [tk, heads, d], out: [tq, q_heads, d], bf16, each with its
 *   stride; cu_q, cu_k: [b + 1] int32 on the device, ascending (values outside the tensors
 *   are clamped); lse: NULL or [tq, q_heads] fp32.
 * Requires q_heads a multiple of heads, d a multiple of 16 up to NVFP4_KV_MAX_DIM, 0 < scale
 * <= 2e38, b at most NVFP4_ATTENTION_MAX_BATCH, (tq / 128 + b) * q_heads below 2^23.  Results
 * are the same on every call.
 *   workspace: NULL, or workspace_bytes >= NVFP4_ATTENTION_PREFILL_WS_BYTES(d) (16-byte
 *   aligned, contents ignored on entry, undefined on exit, not shared by calls that overlap).
 *   With one, few rows behind many keys have the keys split over workgroups, whose sums, fp32,
 *   a second launch joins.  Less than that is taken where it suffices for the sizes at hand.
 * The kernel is chosen by the average sequence: a long prompt and many single rows are faster in
 * two calls (32 / 8 heads of 128: 4096 rows beside 15 of one row behind 2000 keys 194 us, apart 128 + 28).
 */
int attention_prefill(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, int64_t tq, int64_t tk, int64_t q_heads, int64_t heads, int64_t d,
                      const int32_t* cu_q, const int32_t* cu_k, int64_t b, float scale, int causal, void* out,
                      int64_t out_stride, float* lse, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_ATTENTION_H */
