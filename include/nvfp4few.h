/*
 * libnvfp4moe -- the expert layer at few tokens: a router with groups and the
 * products of at most 32 tokens with the weights of include/nvfp4moe.h, whose
 * activations stay 16-bit.
 *
 *   moe_route_grouped   the router: groups, a bias that selects, a factor
 *   moe_matvec_*        one 4-bit matrix
 *   moe_experts_*       the chosen experts' gated products and their sum
 *
 * Conventions are those of nvfp4moe.h: C ABI, status codes and messages,
 * caller-owned device buffers, work enqueued on `stream` without
 * synchronising, programmatic dependent launch, compute capability 10.3.
 * Strides count elements.  Outputs and workspaces overlap nothing else.
 */
#ifndef NVFP4FEW_H
#define NVFP4FEW_H

#include "nvfp4moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Routing with groups of experts, a bias that only selects and a factor on
 * the weights.  With v = logits[t], s_e = sigma(v_e) or softmax(v)_e over all
 * E experts, and c_e = s_e + select_bias[e] (NULL: c = s):
 *   1. group g holds experts g * E / n_group .. ; its value is its largest c
 *      (group_best = 1) or the sum of its two largest (2); the topk_group best
 *      groups are kept, the lower index on ties (n_group = 1: all);
 *   2. the k best c in kept groups, descending, the lower index on ties;
 *   3. topk_w[t, j] = scale * s_j, with renormalize = 1 divided by the sum of
 *      the k chosen s (0 if that sum is 0).  The bias is not in the weights.
 * The choice is that of c computed in float64, also where float32 scores
 * coincide; without a bias (and group_best = 1 or one group) it is that of v.
 * Weights are float32, within 1e-6 relative, also where the scores themselves
 * are too small for float32.  A NaN logit or bias counts as -inf (as a score:
 * 0), +inf as the largest float32; sigma(v) below v = -709.78, where e^-v
 * leaves float64, counts as 0.
 * logits device float32 [T, E]; select_bias device float32 [E] or NULL;
 * topk_idx device int32 [T, k]; topk_w device float32 [T, k].
 * Limits: those of moe_route_topk; 1 <= n_group <= 32 divides E, 1 <=
 * topk_group <= n_group, k <= topk_group * E / n_group, group_best <= E /
 * n_group, scale finite.  No counterpart on the source pages. */
int moe_route_grouped(const float* logits, const float* select_bias, int T, int E, int k,
                      int n_group, int topk_group, int group_best, int score_fn, int renormalize, float scale,
                      int32_t* topk_idx, float* topk_w, cudaStream_t stream);

/* Products of at most 32 tokens with the weights of the grouped GEMM (packed
 * row-major or tiled, blocked scales), which then are read once and bound the
 * time; the activations keep their 16 bits (see below).  No counterpart on the
 * source pages, whose paths quantise activations at every batch size.
 *
 * moe_matvec_nvfp4: out[t, n] = w_gscale[0] * sum_k x[t, k] * W[n, k]
 *   (dequantised, float32 sums), rounded once to the type of x.
 * moe_matvec_mxfp4: the same without w_gscale.
 *   x device [T, K] of x_dtype, rows x_stride elements apart (a multiple of 8;
 *   0: the same row again; not read with T = 1); w_packed device uint8 [N, K/2]
 *   or its tiled copy, w_scales blocked; out device [T, N] contiguous.
 *   ws: moe_matvec_workspace_size(T, N, K) bytes (may be 0), 256-byte aligned.
 *
 * moe_experts_nvfp4: the expert layer after the router.  For the tokens routed
 *   to expert e: h = silu(x Wg^T) * (x Wu^T), Wg and Wu rows [0, I) and
 *   [I, 2I) of w_gu[e] (with w_gu_gscale[e]); out[t] = sum_j topk_w[t, j] *
 *   (h W_d[e]^T) over its k experts e = topk_idx[t, j] in ascending order,
 *   rounded to bf16 once.  h is held in float32 and multiplied as described
 *   below, in small calls as the sum of two float16 (22 bits: 2^-22 relative).
 * moe_experts_mxfp4: the same without the gscales.
 *   x_bf16 device [T, H], rows x_stride elements apart as above; topk_idx
 *   device int32 [T, k], topk_w device float32 [T, k]; w_gu [E, 2I, H], w_d
 *   [E, H, I]; out_bf16 device [T, H] contiguous.  An expert that a token
 *   names twice gets the sum of both weights.  An id outside [0, E) contributes
 *   nothing and raises NVFP4MOE_ERR_DEVICE_DATA.
 *   ws: moe_experts_workspace_size(T, k, H, I) bytes, 256-byte aligned, not
 *   initialised; calls that share one must not overlap on the GPU.
 *
 * How exact the operands are on the tensor core goes by the size of the call:
 *   small (T <= 8, and K <= 6144, T K <= 2^14, T K^2 N <= 2^37; for experts H <=
 *   6144, T H <= 2^14, T k 2 I H <= 2^24, (T k I)^2 2 H <= 2^36, T k ceil(I /
 *   256) <= 127): float16 with a power of two for 256 consecutive activations of
 *   a token: exact down to 2^-28 of their largest, below off by at most 2^-39 of
 *   it.  Infinities and NaN go through the sums (with MXFP4 an infinity may come
 *   out as NaN where scales of 256 consecutive weights of a row are more than
 *   2^27 apart).
 *   else: activations are sums of eight 4-bit terms with a scale for 16 (MXFP4:
 *   32) of them: off by at most 2^-18 of their largest, with NVFP4 also by 2^-34
 *   of the row's (of 2^-80 if that is larger).  An infinity or NaN makes all of
 *   its token's results NaN.
 * Either way a token's results do not depend on the others of the call beyond
 * float32 summation order, and a repeated call gives the same bits.
 * Limits: 0 <= T <= 32 (0 is a no-op), K, H and I multiples of 64 (NVFP4) or
 * 128 (MXFP4), N, H and I multiples of 128, 1 <= E <= 1024, 1 <= k <= 32. */
#define NVFP4MOE_X_BF16 0
#define NVFP4MOE_X_FP16 1
size_t moe_matvec_workspace_size(int T, int N, int K);
int moe_matvec_nvfp4(const void* x, int64_t x_stride, int T, int x_dtype,
                     const uint8_t* w_packed, const uint8_t* w_scales, const float* w_gscale,
                     int N, int K, int w_layout, void* out, void* ws, size_t ws_bytes, cudaStream_t stream);
int moe_matvec_mxfp4(const void* x, int64_t x_stride, int T, int x_dtype,
                     const uint8_t* w_packed, const uint8_t* w_scales,
                     int N, int K, int w_layout, void* out, void* ws, size_t ws_bytes, cudaStream_t stream);
size_t moe_experts_workspace_size(int T, int k, int H, int I);
/* Kernels that a call launches: 0 (T = 0), 2 or 4. */
int moe_experts_launches(int T, int k, int H, int I);
int moe_experts_nvfp4(const void* x_bf16, int64_t x_stride, const int32_t* topk_idx, const float* topk_w,
                      int T, int k, int E, int H, int I,
                      const uint8_t* w_gu_packed, const uint8_t* w_gu_scales, const float* w_gu_gscale,
                      const uint8_t* w_d_packed, const uint8_t* w_d_scales, const float* w_d_gscale,
                      int w_layout, void* out_bf16, void* ws, size_t ws_bytes, cudaStream_t stream);
int moe_experts_mxfp4(const void* x_bf16, int64_t x_stride, const int32_t* topk_idx, const float* topk_w,
                      int T, int k, int E, int H, int I,
                      const uint8_t* w_gu_packed, const uint8_t* w_gu_scales,
                      const uint8_t* w_d_packed, const uint8_t* w_d_scales,
                      int w_layout, void* out_bf16, void* ws, size_t ws_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4FEW_H */
