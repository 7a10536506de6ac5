/*
 * libnvfp4moe -- latent attention: the operators that a block with latent
 * attention runs before its expert layer (include/nvfp4moe.h).
 *
 * A token is cached as one row of 576 values that every head reads: 512
 * latent values (normalised) and 64 rotary ones (rotated by the token's
 * position).  The cache is paged: [num_pages, page_size, 576], row-major;
 * slot s is row s % page_size of page s / page_size.
 *
 *   mla_append   writes new tokens into the cache and rotates their queries
 *   mla_decode   absorbed form: queries of 576 values against the cached rows,
 *                whose first 512 values are also the values
 *   mla_prefill  expanded form: per-head keys of 128 + 64 values (the 64 are
 *                shared by the heads) and values of 128
 *
 * The sizes are fixed.  A layer that caches 512 + 64 values a token but expands
 * them to other keys or values (192 + 64 and 256, say) is served by mla_append
 * and mla_decode and not by mla_prefill.
 *
 * Conventions are those of nvfp4moe.h: C ABI, status codes and messages,
 * caller-owned 16-byte aligned device buffers, work enqueued on `stream`
 * without synchronising, programmatic dependent launch, compute capability
 * 10.3.  Device data out of range (a slot, a page, a position, a length) is
 * never followed: the work is skipped or clamped as stated at each call and
 * nvfp4moe_sync_status() reports NVFP4MOE_ERR_DEVICE_DATA.  Strides count
 * elements.  All tensors of one call have the same 16-bit type (dtype);
 * sums, softmax statistics and norms are float32.
 */
#ifndef NVFP4MLA_H
#define NVFP4MLA_H

#include "nvfp4moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NVFP4MLA_BF16 0
#define NVFP4MLA_FP16 1

#define NVFP4MLA_LATENT 512 /* latent values of a cached row */
#define NVFP4MLA_ROPE    64 /* rotary values of a cached row, a query or an expanded key */
#define NVFP4MLA_ROW    576
#define NVFP4MLA_NOPE   128 /* expanded form: unrotated values of a key or query */
#define NVFP4MLA_VALUE  128 /* expanded form: values of a head */

/* Appends T tokens to the cache.  For token t with position p = positions[t]:
 *   n      = latent[t] / sqrt(mean(latent[t]^2) + eps) * norm_weight  (norm_weight NULL: n = latent[t])
 *   row[t] = [n, R_p k_rope[t]], rounded once to dtype
 *   cache slot slots[t] = row[t] (slots[t] < 0: no slot, nothing written)
 *   rows_out[t] = row[t]                                         (unless NULL)
 *   q_out[t, h] = R_p q_rope[t, h] for h < H                     (H = 0: no queries)
 * R_p rotates 32 pairs (a_i, b_i) -> (a c_i - b s_i, b c_i + a s_i) with c_i =
 * rope_table[p, i], s_i = rope_table[p, 32 + i]; the pairs are (2i, 2i + 1)
 * with interleaved = 1 and (i, i + 32) with 0.  The caller makes the table
 * (any base or scaling of the angles).
 * latent [T, 512], k_rope [T, 64], q_rope and q_out [T, H, 64]: innermost
 * dimension contiguous, the given strides multiples of 8 (0 in an input: the
 * same row again).  q_out's rows must not overlap; it may be q_rope itself (same
 * strides) and must not overlap it otherwise.
 * norm_weight [512]; positions device int32 [T]; slots device int64 [T];
 * rope_table device float32 [max_positions, 64]; cache [num_slots, 576];
 * rows_out [T, 576].
 * Two tokens of a call must not share a slot.  A position outside [0,
 * max_positions) leaves the token's outputs untouched; a slot >= num_slots
 * leaves the cache untouched; both raise NVFP4MOE_ERR_DEVICE_DATA.
 * Limits: 0 <= T <= 2^30, 0 <= H <= 1024, T * (1 + ceil(H / 16)) <= 8 * (2^31 - 1). */
int mla_append(const void* latent, int64_t latent_stride, const void* k_rope, int64_t k_rope_stride,
               const void* norm_weight, float eps, const int32_t* positions, const int64_t* slots, int T,
               const float* rope_table, int64_t max_positions, int interleaved, int dtype,
               void* cache, int64_t num_slots, void* rows_out,
               const void* q_rope, int64_t q_token_stride, int64_t q_head_stride, int H,
               void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, cudaStream_t stream);

/* Absorbed attention of Sq new tokens a sequence over the paged cache.  Row
 * (s, h) of sequence b, n = seq_lens[b] (which counts the Sq new tokens, whose
 * rows are in the cache already), sees keys 0 .. n - Sq + s:
 *   S_j = scale * q[b, s, h] . row_j,  out[b, s, h] = sum_j softmax(S)_j row_j[:512]
 *   lse[b, s, h] = ln sum_j exp(S_j)
 * A row that sees no key gets zeros and -inf.  Key j of sequence b is row j %
 * page_size of page block_tables[b * table_stride + j / page_size]; entries
 * past a sequence's last page and cache rows past its last key are never used,
 * whatever they hold; with Sq > 1 the rows of all Sq new tokens must be finite
 * (a weight of zero is multiplied with those that a row does not see).  A page
 * id outside [0, num_pages) reads as zero rows, a length is clamped to [0,
 * max_pages * page_size]; both raise NVFP4MOE_ERR_DEVICE_DATA.
 * q [B, Sq, H, 576], out [B, Sq, H, 512], lse float32 [B, Sq, H], cache
 * [num_pages, page_size, 576], all contiguous; block_tables device int32;
 * seq_lens device int32 [B].  The softmax's weights are rounded to dtype for
 * the product with the values (fp16: to half a step, or 2^-32 of the row's
 * largest weight if that is more); their sum is not.
 * ws: device scratch of mla_decode_workspace_size() bytes, 256-byte aligned,
 * not initialised; calls that share it must not overlap on the GPU.
 * Limits: page_size a power of two >= 16; num_pages * page_size < 2^31; B, Sq,
 * H >= 1 with B * Sq * H < 2^31 (B = 0 is a no-op) and B * ceil(Sq * H / 64)
 * * ceil(max_pages * page_size / 64) < 2^31; scale > 0 and finite. */
size_t mla_decode_workspace_size(void);
int mla_decode(const void* q, const void* cache, int num_pages, int page_size,
               const int32_t* block_tables, int64_t table_stride, int max_pages, const int32_t* seq_lens,
               int B, int Sq, int H, float scale, int dtype, void* out, float* lse,
               void* ws, size_t ws_bytes, cudaStream_t stream);

/* Expanded attention over a ragged batch.  Sequence b has queries cu_q[b] ..
 * cu_q[b+1] - 1 and keys cu_k[b] .. cu_k[b+1] - 1 (nq and nk of them); its
 * query i sees keys 0 .. nk - nq + i with causal = 1 (the queries are the
 * last of the keys) and all nk with 0.  For head h, query t and key j:
 *   S_j = scale * (q[t, h, :128] . k_nope[j, h] + q[t, h, 128:] . k_rope[j])
 *   out[t, h] = sum_j softmax(S)_j v[j, h],  lse[t, h] = ln sum_j exp(S_j)
 * A query that sees no key gets zeros and -inf.  Values of v that a query does
 * not see must be finite where they are of its own sequence (a weight of zero
 * is multiplied with them); those of other sequences may be anything.
 * q [Tq, H, 192], k_nope [Tk, H, 128], k_rope [Tk, 64], v [Tk, H, 128]:
 * innermost dimension contiguous, strides multiples of 8 and below 2^38; they may be
 * slices of larger tensors.  out [Tq, H, 128] and lse float32 [Tq, H]
 * contiguous.  cu_q, cu_k device int32 [B + 1], ascending, within [0, Tq] and
 * [0, Tk]: offsets outside are clamped and raise NVFP4MOE_ERR_DEVICE_DATA.
 * Outputs of tokens in no sequence are left untouched.  The softmax's weights
 * are rounded as in mla_decode.
 * Limits: B, H >= 1, Tq, Tk >= 0, Tq * H and Tk * H < 2^31, (Tq / 256 + B) * H < 2^31
 * (B = 0, Tq = 0 or H = 0 is a no-op); scale > 0 and finite. */
int mla_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                const void* k_nope, int64_t k_nope_token_stride, int64_t k_nope_head_stride,
                const void* k_rope, int64_t k_rope_token_stride,
                const void* v, int64_t v_token_stride, int64_t v_head_stride,
                const int32_t* cu_q, const int32_t* cu_k, int B, int Tq, int Tk, int H,
                float scale, int causal, int dtype, void* out, float* lse, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4MLA_H */
