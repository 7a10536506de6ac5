// What the kernels of a few tokens' products share (few_tokens.cu,
// few_stream.cu): how 4-bit weights and 16-bit activations become the tensor
// core's float16, and which experts a batch hits.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace nvfp4moe {
namespace few {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kStep = 256;                // columns of a matrix in one step of a warp
constexpr int kUnitBytes = 2 * kStep;     // float16 activations of one token and step
constexpr int kMaxSegs = 1024;

enum Source { kBf16 = 0, kFp16 = 1, kF32 = 2 };
enum Mode { kDense = 0, kGateUp = 1, kDown = 2 };

// The experts that a batch hits, in their order: what the down product walks
// through.
struct Plan {
  int nseg;
  int pad[63];
  int expert[kMaxSegs];
  uint32_t tokens[kMaxSegs];  // bit t: token t is routed to it
  int base[kMaxSegs];         // first row of h; token t's is base + number of lower tokens
};

// The eight codes of a word as float16 pairs (in order).
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t ue4m3x2_to_half(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(two));
  return h;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Converts 8 values that the lane holds of a block of 256 to float16 as the
// header says; returns the factor that undoes it.  TWO: what the rounding
// leaves, as float16 of the same factor, to `rest` (none of an infinity or NaN).
template <bool TWO>
__device__ __forceinline__ float block_to_half(const float (&v)[8], uint4* out, uint4* rest) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  top = __reduce_max_sync(kFull, top) >> 23;
  const int e = top == 255 ? 127 : max(int(top) - 127, -112);
  const float m = exp2i(14 - e);
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = v[2 * i] * m, y = v[2 * i + 1] * m;
    const __half2 t = __floats2half2_rn(x, y);
    h[i] = *reinterpret_cast<const uint32_t*>(&t);
    if (TWO) {
      const float2 q = __half22float2(t);
      const float dx = x - q.x, dy = y - q.y;  // at most 8
      const __half2 u = __floats2half2_rn(fabsf(dx) <= 8.0f ? dx : 0.0f, fabsf(dy) <= 8.0f ? dy : 0.0f);
      l[i] = *reinterpret_cast<const uint32_t*>(&u);
    }
  }
  *out = make_uint4(h[0], h[1], h[2], h[3]);
  if (TWO) *rest = make_uint4(l[0], l[1], l[2], l[3]);
  return exp2i(e - 14);
}

// Values 8 lane .. 8 lane + 7 of step `step` of a row of K values (zeros past its end).
template <int SRC>
__device__ __forceinline__ void load_block(float (&v)[8], const void* row, int step, int K, int lane) {
  const int k = step * kStep + 8 * lane;
  if (k >= K) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    return;
  }
  if (SRC == kF32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(row) + k);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    return;
  }
  const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + k);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (SRC == kBf16) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// The experts that the batch hits, written by one block.  mask, count: E words
// of shared memory each.
template <int THREADS>
__device__ void write_plan(const int32_t* idx, int T, int k, int E, Plan* plan, unsigned* flags, uint32_t* mask,
                           int* count) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = T * k;
  __shared__ int sum_warp[2][THREADS / 32];
  for (int e = tid; e < E; e += THREADS) mask[e] = 0, count[e] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += THREADS) {
    const int e = idx[i];
    if (e >= 0 && e < E) {
      atomicOr(mask + e, 1u << (i / k));
      atomicAdd(count + e, 1);
    } else {
      atomicOr(flags, kFlagBadData);
    }
  }
  __syncthreads();
  const int per = (E + THREADS - 1) / THREADS, e0 = tid * per;
  int segs = 0, rows = 0;
  for (int e = e0; e < min(e0 + per, E); ++e) segs += mask[e] != 0, rows += count[e];
  int a = segs, b = rows;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int ua = __shfl_up_sync(kFull, a, d), ub = __shfl_up_sync(kFull, b, d);
    if (lane >= d) a += ua, b += ub;
  }
  if (lane == 31) sum_warp[0][warp] = a, sum_warp[1][warp] = b;
  __syncthreads();
  int seg = a - segs, row = b - rows;
  for (int w = 0; w < warp; ++w) seg += sum_warp[0][w], row += sum_warp[1][w];
  for (int e = e0; e < min(e0 + per, E); ++e) {
    if (mask[e]) {
      plan->expert[seg] = e;
      plan->tokens[seg] = mask[e];
      plan->base[seg] = row;
      ++seg;
    }
    row += count[e];
  }
  if (tid == THREADS - 1) plan->nseg = seg;
  __syncthreads();
}

}  // namespace few
}  // namespace nvfp4moe
