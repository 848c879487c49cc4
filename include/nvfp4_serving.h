/*
 * nvfp4_serving.h -- C ABI of the serving operators of libnvfp4_amd.so: a whole
 * mixture-of-experts layer for a few tokens, and low-rank adapters of many
 * requests beside a shared NVFP4 projection.
 *
 * Formats, status codes and conventions (device pointers, 16-byte alignment,
 * caller-allocated outputs, argument checks before anything is enqueued, no
 * host synchronisation, no allocation, no state between calls) are those of
 * nvfp4.h.
 */
#ifndef NVFP4_SERVING_H
#define NVFP4_SERVING_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a router's logit becomes a routing weight. */
enum nvfp4_route_score {
    NVFP4_ROUTE_SOFTMAX = 0,  /* exp(l_e) / sum of exp over all experts */
    NVFP4_ROUTE_SIGMOID = 1   /* 1 / (1 + exp(-l_e)), each expert by itself */
};

/* Limits of nvfp4_moe_small (NVFP4_UNSUPPORTED beyond them). */
#define NVFP4_MOE_SMALL_MAX_TOKENS 64
#define NVFP4_MOE_SMALL_MAX_EXPERTS 256
#define NVFP4_MOE_SMALL_MAX_TOP_K 16

/*
 * Bytes of workspace of nvfp4_moe_small: the activations of the t * top_k
 * (token, expert) pairs, `inter` fp32 columns each; 1024 rows of partial fp32
 * outputs; the routing tables; a counter per 16 output columns (h rounded up to
 * 128).
 */
#define NVFP4_MOE_SMALL_WS_BYTES(t, top_k, h, inter) \
    (4 * (int64_t)(t) * (int64_t)(top_k) * (int64_t)(inter) + 4096 + (4096 * 4 + 1) * (((int64_t)(h) + 127) / 128 * 32))

/*
 * A whole mixture-of-experts layer for a few tokens, in two or three launches.
 * Routing, for each token i: the experts are ordered by logit, largest first,
 * equal logits by the lower index first; the first top_k of them whose logit is
 * neither NaN nor -inf are chosen.  Slot j of the token holds the j-th of them,
 *   topk_ids[i, j]     its index (-1 in slots left over),
 *   topk_weights[i, j] its weight: `score` of its logit, divided by the sum of
 *                      the chosen ones' when renormalize != 0 (0 in slots left
 *                      over).  A logit of +inf makes a softmax weight NaN.
 * Then, with W13[e] = [gate; up] and W2[e] dequantized,
 *   [g, u]    = alpha13[e] * x[i] @ W13[e]^T
 *   a         = g / (1 + exp(-g)) * u
 *   out[i, :] = bf16(sum over the chosen e of topk_weights * alpha2[e] * a @ W2[e]^T).
 * A token that chose no expert gets zeros.  Sums and a are formed in fp32, the
 * dequantized weights are exact.  x and a enter the products as fp16 values scaled by
 * 128 columns, x as one (exact, but off by up to 2^-38 of the largest of those columns
 * where it is below 2^-29 of it), a as two (off by 2^-20 of itself, or by 2^-38 of the
 * largest).  Results are the same on every call (no atomic sums).
 *   x: [t, h] bf16; logits: [t, E], bf16 (logits_dtype 0) or fp32 (1).
 *   w13: [E, 2*inter, h/2] packed e2m1, gate rows [0, inter) then up rows;
 *   w13_sf: [E, pad_up(2*inter,128)*pad_up(h/16,4)] ue4m3, swizzled;
 *   w2: [E, h, inter/2]; w2_sf: [E, pad_up(h,128)*pad_up(inter/16,4)];
 *   alpha13, alpha2: [E] fp32 (1 / the weights' global scales).
 *   out: [t, h] bf16; topk_ids: [t, top_k] int32; topk_weights: [t, top_k] fp32.
 *   workspace: workspace_bytes >= NVFP4_MOE_SMALL_WS_BYTES(t, top_k, h, inter),
 *   16-byte aligned; contents ignored on entry, undefined on exit; calls that
 *   share one must not overlap.
 * Requires 1 <= t <= 64, 1 <= E <= 256, 1 <= top_k <= min(E, 16), h and inter
 * >= 16 and multiples of 16.  Returns NVFP4_NULL_POINTER, NVFP4_BAD_SHAPE (also
 * for a workspace that is too small), NVFP4_BAD_DTYPE, NVFP4_UNSUPPORTED (the
 * limits above; an unknown score; one expert's w13 of 2^31 bytes or more)
 * or NVFP4_MISALIGNED before launching anything.
 */
int nvfp4_moe_small(const void *x, int64_t t, int64_t h, const void *logits, int logits_dtype, int64_t E,
                    int64_t top_k, int score, int renormalize, const uint8_t *w13, const uint8_t *w13_sf,
                    const float *alpha13, const uint8_t *w2, const uint8_t *w2_sf, const float *alpha2,
                    int64_t inter, void *out, int32_t *topk_ids, float *topk_weights, void *workspace,
                    int64_t workspace_bytes, void *stream);

/* Bytes of workspace the adapter calls need: the rows' projections onto their
 * adapters' r ranks, fp32.  With NVFP4_GEMM_WS_BYTES (nvfp4.h) more they spread a
 * product over more workgroups, whose partial sums go there. */
#define NVFP4_ADAPTERS_WS_BYTES(m, r) (((int64_t)(m) * (int64_t)(r) * 4 + 255) / 256 * 256)

/* Largest adapter rank (NVFP4_BAD_RANK beyond it). */
#define NVFP4_ADAPTERS_MAX_RANK 256

/*
 * A shared NVFP4 projection with a low-rank adapter per row, for decode: the
 * weight-only product of nvfp4_gemm_w4a16 plus, for row i with a = adapter[i],
 *   out[i, :] = bf16(alpha * x[i] @ dequant(b)^T
 *                    + scaling[a] * (x[i] @ lora_a[a]^T) @ lora_b[a]^T (+ bias)),
 * the adapter's term left out where adapter[i] is outside [0, n_adapters) (-1
 * by custom).  Rows may use any adapters in any order; each distinct adapter of
 * 16 consecutive rows is read once for them (lora_b of up to 64 rows where the weight is
 * large, lora_a of up to 32 where there are many rows).  The projection
 * onto the ranks is summed and held in fp32 and enters the second product whole, as
 * three bf16 parts.  Results are the same on every call (no atomic sums); the order of
 * the fp32 sums depends on m and on the list of adapters.
 * Non-finite values of a row or an adapter reach the rows that hold or use them (an
 * infinity in lora_b as NaN: it meets parts that are 0).
 *   x: [m, k] bf16; b: [n, k/2]; b_sf: swizzled scales; alpha: [1] fp32.
 *   lora_a: [n_adapters, r, k] bf16; lora_b: [n_adapters, n, r] bf16 (adapters of
 *   lower rank padded with zeros); adapter: [m] int32; scaling: NULL (1.0) or
 *   [n_adapters] fp32; bias: NULL or [n] bf16; out: [m, n] bf16.
 *   workspace: workspace_bytes >= NVFP4_ADAPTERS_WS_BYTES(m, r), 16-byte aligned,
 *   contents ignored on entry; calls that share one must not overlap.  With
 *   NVFP4_GEMM_WS_BYTES more the K axis may be split over workgroups (the same
 *   results but for the order of the fp32 sums).
 * Requires m, n >= 1, n_adapters >= 1, k >= 16, k % 16 == 0, r in 8 .. 256 and a
 * multiple of 8 (NVFP4_BAD_RANK), n * r below 2^32 and k at most 2^23
 * (NVFP4_UNSUPPORTED).  Any m up to 2^20 works; for many rows quantize the
 * activation and use nvfp4_gemm_adapters.
 */
int nvfp4_linear_adapters(const void *x, const uint8_t *b, const uint8_t *b_sf, const float *alpha,
                          const void *lora_a, const void *lora_b, const int32_t *adapter, const float *scaling,
                          const void *bias, void *out, int64_t m, int64_t n, int64_t k, int64_t r,
                          int64_t n_adapters, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The same beside the block-scaled product of nvfp4_gemm, for prefill: x comes
 * quantized (a, a_sf, any nvfp4_quantize call) and as it was, for the adapters:
 *   out[i, :] = bf16(alpha * (A @ B^T)[i, :]
 *                    + scaling[t] * (x[i] @ lora_a[t]^T) @ lora_b[t]^T (+ bias)),
 * t = adapter[i].  The adapters' term is added to the GEMM's fp32 accumulators
 * before the output is written; a row without an adapter comes out as
 * nvfp4_gemm's (nvfp4_gemm_ws's), bit for bit, and a row's bits do not depend on the
 * adapters of the rows beside it.
 *   a: [m, k/2], a_sf: its scales; alpha: [1] fp32 = 1 / (gs_a * gs_b); the rest,
 *   and the limits, as nvfp4_linear_adapters.
 *   workspace: as there; with NVFP4_ADAPTERS_WS_BYTES(m, r) + NVFP4_GEMM_WS_BYTES
 *   bytes or more the GEMM takes the split-tail schedule of nvfp4_gemm_ws.
 */
int nvfp4_gemm_adapters(const uint8_t *a, const uint8_t *b, const uint8_t *a_sf, const uint8_t *b_sf,
                        const float *alpha, const void *x, const void *lora_a, const void *lora_b,
                        const int32_t *adapter, const float *scaling, const void *bias, void *out, int64_t m,
                        int64_t n, int64_t k, int64_t r, int64_t n_adapters, void *workspace,
                        int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_SERVING_H */
