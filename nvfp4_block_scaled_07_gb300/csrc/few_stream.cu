// The products of a few tokens as one stream of weights over all SMs
// (moe_matvec_*, moe_experts_* beyond what few_tokens.cu takes), on the
// block-scaled tensor core.
//
// kind::mxf4nvf4 multiplies the 4-bit weights with their scales as they lie in
// memory, but takes 4-bit activations.  So an activation becomes a sum of eight
// 4-bit terms, each the rounding of what the terms before it left:
//   x = sum_r s_r b_r q_r + rest     q_r an E2M1 code, b_r the scale of its
//                                    block (16 values, ue4m3; MXFP4: 32, E8M0)
//   y[n, t] = s_0(t) sum_r 2^-shift_r (W q_r b_r)[n]
// Block scales are rounded up, so a term's largest value lies in 5.3 .. 6 of
// its step (E8M0: 3 .. 6) and the rest is at most 0.1875 (0.2) of it: after
// eight terms 2^-19 (2^-18) of the block's largest value.  NVFP4 terms share a
// power of two s_0 with their token's row, which grows smaller by 2^-shift_r from term
// to term as the rests do, so that ue4m3 reaches blocks 2^-14 of the row's
// largest; below, a value is off by 2^-34 of that.  The eight terms of a token are
// eight columns of the product: tokens x 8 columns of N, 128 weight rows M.
//
// The work is a list of stages in order: of a tile (128 rows of a matrix, or
// 64 of gate and the same 64 of up) the steps of 256 columns, of the down
// product all steps of all experts.  Every SM takes an equal range of it,
// whatever tiles that cuts.  One producer keeps a ring of weights in flight
// (tensor copies of 18 KB with their scales), another one of the tokens' terms
// (1.1 KB each; from L2, so fewer stages), four warps move the scales to tensor memory, one thread issues the
// MMAs, four warps sum the terms and join.  Where ranges cut a tile, each block
// leaves its sums in the workspace, and the one that is last adds them in the
// order of the ranges: a repeated call gives the same bits.
//
// 132 MB of weights take 25.5 us (one token) to 27.4 us (16), 5.2 to 4.8 TB/s with
// the launch that makes the terms.  19.5 us are the bytes; the rest, in which memory
// idles, are the starts of two launches and the last joins.  32 tokens take 35.8 us,
// bound by one accumulator and three stages of terms.  The
// same stream on mma.sync, with the codes widened to float16 in registers, was
// bound by those instructions: 31 us at 8 tokens, 79 us at 32, and 1390 us for 23
// tokens through a layer that takes 451 us here.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "../../include/nvfp4few.h"
#include "common.cuh"
#include "few_common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "mla_common.cuh"
#include "sm103_ptx.cuh"

namespace nvfp4moe {
using namespace few;
namespace {

__device__ unsigned g_stream_flags = 0;

constexpr int kTerms = 8;
constexpr int kCodeBytes = kTerms * kStep / 2;  // of a token and step: 8 rows of 128 bytes, swizzled as TMA would
constexpr int kTermScales = 128;                // their scales: [term][64 columns][4 bytes]
constexpr int kWeightBytes = 128 * 128;         // of a stage
constexpr int kScaleBytes = 2048;
constexpr int kStageBytes = kWeightBytes + kScaleBytes;
constexpr int kTileRows = 128;
constexpr int kMinShare = 4;                    // stages
constexpr int kMaxStages = 8;
constexpr int kJoinWarps = 4;
// warps: producers of weights and of terms, MMA, four that move scales, joiners
constexpr int kTermWarp = 1, kMmaWarp = 2, kScaleWarp = 3, kJoiner = 7, kThreads = 32 * (kJoiner + kJoinWarps);
// tensor memory: accumulators in columns 0 .. 255, then the stages' scales
constexpr int kTmemCols = 512, kScaleCol = 256;
constexpr int kSmemLimit = 227 * 1024;

// log2 of what term r's scale is smaller by than the first's: not more than
// the rests shrink (2.41 a term).
__host__ __device__ constexpr int shift_of(int r) { return r * 2415 / 1000; }

struct StreamParams {
  const float* gscale;       // null: 1
  const float* next_gscale;  // gate/up: of the down matrices
  const uint8_t* codes;      // terms of the activations: [step][row][kCodeBytes]
  const uint8_t* scales;     // [step][row][kTermScales]
  const float* row_scale;    // s_0 of each row
  int rows;
  int T, k, E, N, K, tiled, out_fp16;
  int stages, term_stages, term_bytes;         // of the weights' ring and the terms'; of a stage of terms
  const int32_t* idx;
  const float* topk_w;
  void* out;                 // [T, N], or h [T * k, N / 2] float32
  const Plan* plan;
  float* partial;            // [2 * grid][T][128]
  uint32_t* done;            // blocks that are through with a cut tile
  uint32_t wait_us;
};

// ---- activations, counters and plan beforehand ---------------------------------------
constexpr int kPrepThreads = 256, kPrepWarps = kPrepThreads / 32;

__device__ __forceinline__ float half_at(uint32_t low) { return __half2float(__ushort_as_half(uint16_t(low))); }

// Eight terms of a step's 256 values, of which the lane holds 8 lane .. 8 lane + 7.
template <bool MX>
__device__ __forceinline__ void write_terms(float (&v)[8], float s0, float inv_s0, int lane, uint8_t* codes, uint8_t* scales) {
#pragma unroll
  for (int r = 0; r < kTerms; ++r) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
    float step, inv;
    uint32_t sb;
    if (MX) {
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
      int x = max(mx_exponent(top), -126);
      if (top > 6.0f * exp2i(x)) ++x;          // at most 126
      sb = uint32_t(x + 127);
      step = exp2i(x);
      inv = exp2i(-x);
      const uint32_t next = __shfl_down_sync(kFull, sb, 4);
      if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(scales + r * 16 + (lane >> 3) * 4) = sb | next << 8;
    } else {
      const float s = s0 * (1.0f / float(1 << shift_of(r))), t = top * (inv_s0 * (float(1 << shift_of(r)) / 6.0f));
      uint16_t near;                           // the nearest scale, and the next where that is below t
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(near) : "f"(t));
      sb = near & 0xFFu;
      const float below = half_at(ue4m3x2_to_half(sb));
      if (below < t && sb < 0x7E) ++sb;
      step = half_at(ue4m3x2_to_half(sb)) * s;
      inv = sb ? ptx::rcp_approx(step) : 0.0f; // a code off by this is made good by the next term
      if ((lane & 1) == 0) scales[r * 16 + (lane >> 1)] = uint8_t(sb);
    }
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) word |= e2m1x2(v[2 * i] * inv, v[2 * i + 1] * inv) << (8 * i);
    *reinterpret_cast<uint32_t*>(codes + r * 128 + (((lane >> 2) ^ r) * 16) + (lane & 3) * 4) = word;
    uint32_t h[4];
    codes_to_half(word, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      v[2 * i] = fmaf(-q.x, step, v[2 * i]);
      v[2 * i + 1] = fmaf(-q.y, step, v[2 * i + 1]);
    }
  }
}

// A block converts eight steps of one row, whose largest value it finds first.
// An infinity or NaN makes the row's scale NaN, and so the results.
template <bool MX, int SRC>
__device__ __forceinline__ void convert_row(const void* x, int row, int rows, int group, int K, uint8_t* codes,
                                            uint8_t* scales, float* row_scale) {
  __shared__ uint32_t s_top[kPrepWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, steps = (K + kStep - 1) / kStep;
  const int step = group * kPrepWarps + warp;  // this warp's
  float v[8];
  load_block<SRC>(v, x, step, K, lane);
  uint32_t top = 0;
#pragma unroll 4
  for (int s = warp; s < steps; s += kPrepWarps) {
    float u[8];
    load_block<SRC>(u, x, s, K, lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(u[i]) & 0x7FFFFFFFu);
  }
  top = __reduce_max_sync(kFull, top);
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPrepWarps; ++w) top = max(top, s_top[w]);
  const bool finite = top < 0x7F800000u;
  const int e0 = max(int(top >> 23) - 127, -80) - 10;
  const float s0 = exp2i(e0);                  // the largest is 170 .. 342 times 6 of it
  if (group == 0 && threadIdx.x == 0) row_scale[row] = !finite ? __int_as_float(0x7FFFFFFF) : (MX ? 1.0f : s0);
  if (step >= steps) return;
  if (!finite) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
  const int64_t at = int64_t(step) * rows + row;
  write_terms<MX>(v, finite ? s0 : 1.0f, finite ? exp2i(-e0) : 1.0f, lane, codes + at * kCodeBytes, scales + at * kTermScales);
}

// Grid: (groups of eight steps, rows and, with a plan, one more).  Zeroes the counters as well.
template <bool MX, int SRC>
__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(const uint8_t* x, int64_t row_bytes, int rows, int K,
                                                               uint8_t* codes, uint8_t* scales, float* row_scale,
                                                               uint32_t* counters, int n_counters, const int32_t* idx, int T,
                                                               int k, int E, Plan* plan) {
  extern __shared__ uint32_t words[];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int row = blockIdx.y, block = blockIdx.y * gridDim.x + blockIdx.x;
  for (int i = block * kPrepThreads + threadIdx.x; i < n_counters; i += gridDim.x * gridDim.y * kPrepThreads) counters[i] = 0;
  if (row < rows)
    convert_row<MX, SRC>(x + row * row_bytes, row, rows, blockIdx.x, K, codes, scales, row_scale);
  else if (blockIdx.x == 0)
    write_plan<kPrepThreads>(idx, T, k, E, plan, &g_stream_flags, words, reinterpret_cast<int*>(words + E));
}

// The experts of at most 32 ids, in ascending order, by one warp: their number,
// and (unless null) the list and their tokens.  What the plan says, without waiting for it.
__device__ __forceinline__ int experts_of_warp(const int32_t* idx, int T, int k, int E, int lane, int* list, uint32_t* tokens) {
  const int n = T * k;
  const int e = lane < n ? __ldcg(idx + lane) : -1;
  const uint32_t same = __match_any_sync(kFull, e);
  const bool first = e >= 0 && e < E && __ffs(same) - 1 == lane;
  const uint32_t leaders = __ballot_sync(kFull, first);
  if (list) {
    int at = 0;
    for (int i = 0; i < n; ++i) {
      const int other = __shfl_sync(kFull, e, i);
      at += ((leaders >> i) & 1) && other < e;
    }
    uint32_t mine = 0;
    for (int t = 0; t < T; ++t) mine |= uint32_t((same & (((k < 32 ? 1u << k : 0u) - 1) << (t * k))) != 0) << t;
    if (first) list[at] = e, tokens[at] = mine;
    __syncwarp();
  }
  return __popc(leaders);
}

// Copies and MMAs issued by the elected lane of a converged warp (mla::elect_one).
__device__ __forceinline__ void tma_2d(uint32_t elected, uint32_t dst, const void* map, uint32_t bar, int c0, int c1,
                                       uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "l"(policy), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t elected, uint32_t dst, const void* map, uint32_t bar, int c0, int c1, int c2,
                                       int c3, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %8, 0;\n\t"
      "@q cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t elected, uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
      "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "r"(elected)
      : "memory");
}
// a, b: low words of the operands' descriptors (mla::desc_sw128)
template <bool MX>
__device__ __forceinline__ void mma_fp4(uint32_t elected, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
  if (MX)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %8};\n\tmov.b64 y, {%2, %8};\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], x, y, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(elected), "n"(mla::desc_hi(1024))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %8};\n\tmov.b64 y, {%2, %8};\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], x, y, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(elected), "n"(mla::desc_hi(1024))
        : "memory");
}

// A run of stages that share an accumulator: a tile's, of the down product one
// expert's of it.
struct Unit {
  int tile, seg, step, n;
  bool last;                                   // of the tile in this block's range
};

template <bool MX, int MODE, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) stream_kernel(const __grid_constant__ CUtensorMap weights,
                                                             const __grid_constant__ CUtensorMap scales,
                                                             const StreamParams p) {
  // WIDE: up to 256 columns, one accumulator; else up to 128 and two
  constexpr int kBuffers = WIDE ? 1 : 2, kScaleCols = WIDE ? 48 : 32;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t s_full[2 * kMaxStages], s_ready[kMaxStages], s_empty[2 * kMaxStages], s_acc[2 * kBuffers + 1];
  __shared__ mla::WaitCtl s_ctl;
  __shared__ uint32_t s_tmem;
  __shared__ int s_last, s_expert[2][32];      // of each producer
  __shared__ uint32_t s_tokens[32];
  uint8_t* smem = raw + ((1024 - (ptx::smem_u32(raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = mla::uniform(tid >> 5);
  const uint32_t full = ptx::smem_u32(s_full), ready = ptx::smem_u32(s_ready), empty = ptx::smem_u32(s_empty);
  const uint32_t t_full = full + 8 * kMaxStages, t_empty = empty + 8 * kMaxStages;          // of the terms
  const uint32_t terms = ptx::smem_u32(smem) + p.stages * kStageBytes;
  const uint32_t acc_full = ptx::smem_u32(s_acc), acc_empty = acc_full + 8 * kBuffers, drained = acc_empty + 8 * kBuffers;
  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      ptx::mbar_init(full + 8 * i, 1);
      ptx::mbar_init(ready + 8 * i, 4);        // the scale warps
      ptx::mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < p.term_stages; ++i) {
      ptx::mbar_init(t_full + 8 * i, 1);
      ptx::mbar_init(t_empty + 8 * i, 1);
    }
    for (int i = 0; i < kBuffers; ++i) {
      ptx::mbar_init(acc_full + 8 * i, 1);
      ptx::mbar_init(acc_empty + 8 * i, kJoinWarps);
    }
    ptx::mbar_init(drained, 1);
    ptx::fence_barrier_init();
    s_ctl.abort = 0;
    s_ctl.limit_us = p.wait_us;
    s_ctl.flags = &g_stream_flags;
    ptx::prefetch_tmap(&weights);
    ptx::prefetch_tmap(&scales);
  }
  if (warp == kScaleWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&s_tmem), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = s_tmem;

  // The kernel before is one of the same call, a prepare_kernel, which lets the
  // next be launched after its own wait: what was there before it (weights,
  // ids, for the down product the plan) can be read before this kernel's wait (from L2).
  const bool producer = warp <= kTermWarp;
  const bool early = MODE != kGateUp || p.T * p.k <= 32;   // the experts are known before the wait
  if (!producer || !early) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
  }
  const int nseg = MODE == kDense ? 1
                   : MODE == kGateUp && early ? experts_of_warp(p.idx, p.T, p.k, p.E, lane, producer ? s_expert[warp] : nullptr, s_tokens)
                                              : __ldcg(&p.plan->nseg);
  const int steps = (p.K + kStep - 1) / kStep, seg_tiles = MODE == kGateUp ? p.N / kTileRows : 1;
  const int tiles = MODE == kGateUp ? nseg * seg_tiles : p.N / kTileRows;
  const int length = MODE == kDown ? nseg * steps : steps;             // stages of a tile
  const int64_t all = int64_t(tiles) * length;
  const int per = int(max(int64_t(kMinShare), (all + gridDim.x - 1) / gridDim.x));
  const int64_t start = int64_t(blockIdx.x) * per, end = min(all, start + per);
  const int blocks = p.N / 128, k_blocks = p.K / 64;
  const int sf_at = p.term_bytes / (kCodeBytes + kTermScales) * kCodeBytes;   // the terms' scales in their stage
  // the units of this block's range, in order
  auto unit_at = [&](int64_t s) {
    Unit u;
    u.tile = int(s / length);
    const int at = int(s - int64_t(u.tile) * length);
    u.seg = MODE == kGateUp ? u.tile / seg_tiles : (MODE == kDown ? at / steps : 0);
    u.step = MODE == kDown ? at - u.seg * steps : at;
    u.n = int(min(end - s, int64_t(steps - u.step)));
    u.last = at + u.n == length || s + u.n == end;
    return u;
  };

  if (MODE == kDown && nseg == 0) {            // no token has an expert
    constexpr int kOthers = kThreads - 64;     // the producers have not waited
    if (!producer)
      for (int64_t i = int64_t(blockIdx.x) * kOthers + tid - 64; i < int64_t(p.T) * p.N; i += int64_t(gridDim.x) * kOthers)
        static_cast<uint16_t*>(p.out)[i] = 0;
  } else if (warp == 0) {
    // ---- weights and their scales, the first stages before the wait
    const uint32_t el = mla::elect_one();
    const uint64_t policy = ptx::policy_evict_first();
    const int kb_all = p.K / (MX ? 128 : 64);
    constexpr int kPerStep = MX ? 2 : 4;       // scale blocks of a step
    int st = 0, parity = 1;
    int64_t count = 0;
    bool ok = true;
    for (int64_t s = start; s < end && ok;) {
      const Unit u = unit_at(s);
      const int e = mla::uniform(MODE == kDense ? 0 : MODE == kGateUp && early ? s_expert[0][u.seg] : __ldcg(p.plan->expert + u.seg));
      const int in = MODE == kGateUp ? u.tile - u.seg * seg_tiles : u.tile;
      const int blk = mla::uniform(e * blocks + (MODE == kGateUp ? in >> 1 : in)), half = mla::uniform(in & 1);
      for (int i = 0; i < u.n; ++i, ++count) {
        ok = mla::wait_warp(empty + 8 * st, parity, &s_ctl);
        if (!ok) break;
        const int step = u.step + i;
        const uint32_t bar = full + 8 * st, dst = ptx::smem_u32(smem) + st * kStageBytes;
        mla::arrive_expect_tx(el, bar, kWeightBytes + kPerStep * 512);
        const int w0 = p.tiled ? 0 : step * 128, w1 = p.tiled ? blk * steps + step : blk, s1 = blk * kb_all + step * kPerStep;
        if (MODE == kGateUp) {                 // 16 rows of each 32 of a block of 128: gate's, then up's
          tma_4d(el, dst + kWeightBytes, &scales, bar, 64 * half, 0, step * kPerStep, blk, policy);
          tma_4d(el, dst, &weights, bar, w0, 16 * half, 0, w1 * 4, policy);
        } else {
          tma_2d(el, dst + kWeightBytes, &scales, bar, 0, s1, policy);
          tma_2d(el, dst, &weights, bar, w0, w1 * 128, policy);
        }
        if (++st == p.stages) st = 0, parity ^= 1;
      }
      s += u.n;
    }
    if (!ok)                                   // given up: the block's copies land before it leaves
      for (int64_t j = max(int64_t(0), count - p.stages); j < count; ++j)
        mla::drain_phase(full + 8 * int(j % p.stages), int(j / p.stages) & 1);
    __syncwarp();
  } else if (warp == kTermWarp) {
    // ---- the tokens' terms
    const uint32_t el = mla::elect_one();
    int st = 0, parity = 1;
    int64_t count = 0;
    bool ok = true;
    for (int64_t s = start; s < end && ok;) {
      const Unit u = unit_at(s);
      const uint32_t tokens = mla::uniform(MODE == kDense ? 0 : MODE == kGateUp && early ? s_tokens[u.seg]
                                                                                         : __ldcg(p.plan->tokens + u.seg));
      const int base = mla::uniform(MODE == kDown ? __ldcg(p.plan->base + u.seg) : 0), m = MODE == kDense ? p.T : __popc(tokens);
      if (s == start) ptx::grid_dep_wait();    // the terms are the kernel before's
      for (int i = 0; i < u.n; ++i, ++count) {
        ok = mla::wait_warp(t_empty + 8 * st, parity, &s_ctl);
        if (!ok) break;
        const uint32_t bar = t_full + 8 * st, dst = terms + st * p.term_bytes;
        const uint8_t* codes = p.codes + int64_t(u.step + i) * p.rows * kCodeBytes;
        const uint8_t* sf = p.scales + int64_t(u.step + i) * p.rows * kTermScales;
        mla::arrive_expect_tx(el, bar, m * (kCodeBytes + kTermScales));
        if (MODE == kGateUp && m < p.T) {
          uint32_t left = tokens;
          for (int slot = 0; slot < m; ++slot, left &= left - 1) {
            const int t = __ffs(left) - 1;
            bulk_copy(el, dst + slot * kCodeBytes, codes + t * kCodeBytes, kCodeBytes, bar);
            bulk_copy(el, dst + sf_at + slot * kTermScales, sf + t * kTermScales, kTermScales, bar);
          }
        } else {
          bulk_copy(el, dst, codes + int64_t(base) * kCodeBytes, m * kCodeBytes, bar);
          bulk_copy(el, dst + sf_at, sf + int64_t(base) * kTermScales, m * kTermScales, bar);
        }
        if (++st == p.term_stages) st = 0, parity ^= 1;
      }
      s += u.n;
    }
    if (!ok)
      for (int64_t j = max(int64_t(0), count - p.term_stages); j < count; ++j)
        mla::drain_phase(t_full + 8 * int(j % p.term_stages), int(j / p.term_stages) & 1);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---- MMAs: 128 rows x (8 columns a token), 64 columns of K each
    const uint32_t el = mla::elect_one();
    int st = 0, parity = 0, ts = 0;
    uint32_t n = 0;
    bool ok = true;
    for (int64_t s = start; s < end && ok; ++n) {
      const Unit u = unit_at(s);
      const int m = MODE == kDense ? p.T : __popc(p.plan->tokens[u.seg]);
      const uint32_t idesc = mla::uniform(ptx::idesc_nvfp4(128, (m * kTerms + 15) / 16 * 16, MX));
      const uint32_t buffer = n % kBuffers, d = tmem + buffer * 128;
      ok = mla::wait_warp(acc_empty + 8 * buffer, ((n / kBuffers) & 1) ^ 1, &s_ctl);
      for (int i = 0; i < u.n && ok; ++i) {
        ok = mla::wait_warp(ready + 8 * st, parity, &s_ctl);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t a = mla::desc_sw128(ptx::smem_u32(smem) + st * kStageBytes, 16);
        const uint32_t b = mla::desc_sw128(terms + ts * p.term_bytes, 16), sf = tmem + kScaleCol + st * kScaleCols;
        const int nk = min(4, k_blocks - 4 * (u.step + i));
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
          if (kb < nk)
            mma_fp4<MX>(el, d, a + 2 * kb, b + 2 * kb, idesc, sf + 4 * kb, sf + 16 + (WIDE ? 8 : 4) * kb, i > 0 || kb > 0);
        mla::tc_commit(el, empty + 8 * st);
        mla::tc_commit(el, t_empty + 8 * ts);
        if (++st == p.stages) st = 0, parity ^= 1;
        if (++ts == p.term_stages) ts = 0;
      }
      if (ok) mla::tc_commit(el, acc_full + 8 * buffer);
      s += u.n;
    }
    mla::tc_commit(el, drained);               // before the tensor memory is freed
    mla::drain_phase(drained, 0);
    __syncwarp();
  } else if (warp < kJoiner) {
    // ---- scales to tensor memory: lane i of each quarter holds rows i, 32 + i, 64 + i and 96 + i
    const uint32_t quarter = uint32_t(warp & 3) * 32 << 16;
    int st = 0, parity = 0, ts = 0, t_parity = 0;
    bool ok = true;
    for (int64_t s = start; s < end && ok;) {
      const Unit u = unit_at(s);
      const int m = MODE == kDense ? p.T : __popc(p.plan->tokens[u.seg]);
      for (int i = 0; i < u.n; ++i) {
        ok = __all_sync(kFull, mla::wait_phase(full + 8 * st, parity, &s_ctl) && mla::wait_phase(t_full + 8 * ts, t_parity, &s_ctl));
        if (!ok) break;
        const uint32_t at = ptx::smem_u32(smem) + st * kStageBytes + kWeightBytes, t_at = terms + ts * p.term_bytes + sf_at;
        const uint32_t sf = tmem + quarter + kScaleCol + st * kScaleCols;
        uint32_t c[16], t[WIDE ? 32 : 16];       // columns: [64 columns of K][32 rows]
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          uint4 w = ptx::lds128(at + (MX ? kb >> 1 : kb) * 512 + lane * 16);
          if (MX) {                            // a block's four scales are those of two K steps
            const int by = (kb & 1) * 16;
            w = make_uint4((w.x >> by) & 0xFFFFu, (w.y >> by) & 0xFFFFu, (w.z >> by) & 0xFFFFu, (w.w >> by) & 0xFFFFu);
          }
          c[4 * kb] = w.x, c[4 * kb + 1] = w.y, c[4 * kb + 2] = w.z, c[4 * kb + 3] = w.w;
        }
        // row 32 j + lane of the terms: term lane % 8 of token 4 j + lane / 8
#pragma unroll
        for (int j = 0; j < (WIDE ? 8 : 4); ++j) {
          const int token = 4 * j + (lane >> 3);
          uint4 w = make_uint4(0, 0, 0, 0);
          if (token < m) w = ptx::lds128(t_at + token * kTermScales + (lane & 7) * 16);
          constexpr int kRows = WIDE ? 8 : 4;
          t[j] = w.x, t[kRows + j] = w.y, t[2 * kRows + j] = w.z, t[3 * kRows + j] = w.w;
        }
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_st_32x32b_x16(sf, c);
        if constexpr (WIDE) ptx::tmem_st_32x32b_x32(sf + 16, t);
        else ptx::tmem_st_32x32b_x16(sf + 16, t);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::fence_proxy_async_smem();         // these reads before the copies that take the slot next
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ready + 8 * st);
        if (++st == p.stages) st = 0, parity ^= 1;
        if (++ts == p.term_stages) ts = 0, t_parity ^= 1;
      }
      s += u.n;
    }
  } else {
    // ---- joiners: a thread a row; sums over the terms, the experts (down) and the blocks
    const int quarter = warp & 3, row = 32 * quarter + lane, id = tid - 32 * kJoiner;
    const uint32_t lanes = tmem + (uint32_t(32 * quarter) << 16);
    float* total = reinterpret_cast<float*>(smem + p.stages * kStageBytes + p.term_stages * p.term_bytes) + row;   // [token or slot][128]
    uint32_t n = 0;
    int64_t tile_first = start;                // the block's first stage of the tile
    for (int64_t s = start; s < end; ++n) {
      const Unit u = unit_at(s);
      const uint32_t tokens = MODE == kDense ? 0 : p.plan->tokens[u.seg];
      const int base = MODE == kDense ? 0 : p.plan->base[u.seg], m = MODE == kDense ? p.T : __popc(tokens);
      // lane i: slot i's token and the scale of its row of activations
      const int token = MODE == kDense || lane >= m ? lane : int(__fns(tokens, 0, lane + 1));
      const float scale = lane < m ? p.row_scale[MODE == kDown ? base + lane : token] : 0.0f;
      float w = 0.0f, ws = 1.0f;               // lane i: slot i's weight of this expert, with the next matrix's scale
      if (MODE == kGateUp) {
        const int e = p.plan->expert[u.seg];
        if (p.gscale) ws = p.gscale[e];
        const float next = p.next_gscale ? p.next_gscale[e] : 1.0f;
        if (lane < m)
          for (int j = 0; j < p.k; ++j) {
            const int is = p.idx[token * p.k + j];
            const float x = p.topk_w[token * p.k + j];
            w += is == e ? x : 0.0f;
          }
        w *= next;
      } else if (MODE == kDense && p.gscale) {
        ws = p.gscale[0];
      }
      if (MODE == kDown && s == tile_first)
        for (int t = 0; t < p.T; ++t) total[t * kTileRows] = 0.0f;
      const uint32_t buffer = n % kBuffers;
      const bool ok = mla::wait_phase(acc_full + 8 * buffer, (n / kBuffers) & 1, &s_ctl);
      __syncwarp();
      if (__all_sync(kFull, ok)) {
        ptx::tc_fence_after();
        for (int slot = 0; slot < m; slot += 2) {
          uint32_t d[16];
          mla::tmem_ld_32x32b_x16(lanes + buffer * 128 + slot * kTerms, d);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float v = 0.0f;                    // the small terms first
#pragma unroll
            for (int r = kTerms - 1; r >= 0; --r)
              v += __uint_as_float(d[j * kTerms + r]) * (MX ? 1.0f : 1.0f / float(1 << shift_of(r)));
            const int i = (slot + j) & 31;
            v *= __shfl_sync(kFull, scale, i);
            const int t = __shfl_sync(kFull, token, i);
            if (slot + j < m) {
              if (MODE == kDown) total[t * kTileRows] += v;
              else total[(slot + j) * kTileRows] = v;
            }
          }
        }
        ptx::tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(acc_empty + 8 * buffer);
      s += u.n;
      if (!u.last) continue;

      // the tile's sums of this range are complete
      const int64_t tile_start = int64_t(u.tile) * length;
      const int first = int(tile_start / per), last = int((tile_start + length - 1) / per);
      const bool whole = first == last;
      const int width = MODE == kGateUp ? m : p.T;
      auto slot_of = [&](int block) {          // a block's first range of a cut tile, or its last
        return p.partial + int64_t(2 * block + (int64_t(block) * per > tile_start ? 0 : 1)) * p.T * kTileRows + row;
      };
      tile_first = s;
      if (!whole) {
        float* to = slot_of(blockIdx.x);
        for (int i = 0; i < width; ++i) to[i * kTileRows] = total[i * kTileRows];
        mla::bar_sync(1, 32 * kJoinWarps);
        if (id == 0) {                         // releases what the barrier ordered before it, acquires the others'
          uint32_t before;
          asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.done + u.tile) : "memory");
          s_last = before == uint32_t(last - first);
        }
        mla::bar_sync(1, 32 * kJoinWarps);
        if (!s_last) continue;
        // the ranges' sums in their order; eight tokens of four ranges on their way together
        for (int i = 0; i < width; i += 8) {
          float v[8] = {};
          for (int b = first; b <= last; b += 4) {
            float a[4][8];
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int j = 0; j < 8; ++j)
                a[c][j] = b + c <= last && i + j < width ? __ldcg(slot_of(b + c) + (i + j) * kTileRows) : 0.0f;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] += a[c][j];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (i + j < width) total[(i + j) * kTileRows] = v[j];
        }
      }
      if (MODE == kGateUp) {
        const int I = p.N / 2, in = u.tile - u.seg * seg_tiles;
        // rows 32 q + j are gate's, 32 q + 16 + j up's
        const int col = (in >> 1) * 128 + 32 * quarter + 16 * (in & 1) + lane;
        for (int i = 0; i < m; ++i) {
          const float gate = total[i * kTileRows] * ws, up = __shfl_xor_sync(kFull, gate, 16), wi = __shfl_sync(kFull, w, i);
          if (lane < 16) static_cast<float*>(p.out)[int64_t(base + i) * I + col] = gate / (1.0f + expf(-gate)) * up * wi;
        }
      } else {
        for (int t = 0; t < p.T; ++t) {
          const float v = total[t * kTileRows] * ws;
          const int64_t o = int64_t(t) * p.N + u.tile * kTileRows + row;
          if (MODE == kDense && p.out_fp16)
            static_cast<__half*>(p.out)[o] = __float2half_rn(v);
          else
            static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kScaleWarp) ptx::tmem_dealloc(tmem, kTmemCols);
}

int64_t steps_of(int K) { return (K + kStep - 1) / kStep; }
int64_t round256(int64_t b) { return (b + 255) & ~int64_t(255); }

// The parts of a workspace.
struct Layout {
  int64_t plan, counters, codes, scales, row_scale, h, h_codes, h_scales, h_row_scale, partial, bytes;
  int n_counters, n_done;
};
Layout layout_of(int T, int k, int E, int N, int K, int I) {  // I = 0: one matrix
  Layout l = {};
  const int64_t rows = int64_t(T) * k, segs = rows < E ? rows : E;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t a = at;
    at += round256(bytes);
    return a;
  };
  l.plan = take(I ? sizeof(Plan) : 0);
  l.n_done = int(I ? segs * (I / 64) : N / kTileRows);
  l.n_counters = l.n_done + (I ? N / kTileRows : 0);
  l.counters = take(int64_t(l.n_counters) * 4);
  l.codes = take(T * steps_of(K) * kCodeBytes);
  l.scales = take(T * steps_of(K) * kTermScales);
  l.row_scale = take(T * 4);
  if (I) {
    l.h = take(rows * I * 4);
    l.h_codes = take(rows * steps_of(I) * kCodeBytes);
    l.h_scales = take(rows * steps_of(I) * kTermScales);
    l.h_row_scale = take(rows * 4);
  }
  l.partial = take(int64_t(2) * kFewMaxGrid * T * kTileRows * 4);
  l.bytes = at;
  return l;
}

// The weights of all experts: boxes of 128 rows x 128 bytes (zeros past K/2)
// or, for the gated product, of 16 rows of each 32 of a block of 128, gate's and
// up's in turn; and the scales' blocks of 512 bytes, or their halves in turn.
bool weight_maps(CUtensorMap* weights, CUtensorMap* scales, const FewMatrix& w, int E, bool gate_up) {
  auto enc = mla::tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t steps = steps_of(w.K), row = w.tiled ? 128 : w.K / 2, rows = cuuint64_t(E) * w.N * (w.tiled ? steps : 1);
  const cuuint64_t up = cuuint64_t(w.N / 2) * row * (w.tiled ? steps : 1);    // bytes from gate to up
  const cuuint64_t dims[2] = {row, rows}, strides[1] = {row};
  const cuuint64_t g_dims[4] = {row, 32, 2, rows / 32}, g_strides[3] = {row, up, 32 * row};
  const cuuint32_t box[2] = {128, 128}, g_box[4] = {128, 16, 2, 4}, unit[4] = {1, 1, 1, 1};
  const cuuint32_t per_step = w.mx ? 2 : 4;
  const cuuint64_t kb = w.K / (w.mx ? 128 : 64), s_rows = cuuint64_t(E) * (w.N / 128) * kb;
  const cuuint64_t s_dims[2] = {128, s_rows}, s_strides[1] = {512};
  // gate's blocks of 128 rows and, as many further, up's; a step's blocks past the columns are not read
  const cuuint64_t gs_dims[4] = {128, 2, kb, cuuint64_t(E) * (w.N / 128)};
  const cuuint64_t gs_strides[3] = {cuuint64_t(w.N / 256) * kb * 512, 512, kb * 512};
  const cuuint32_t s_box[2] = {128, per_step}, gs_box[4] = {64, 2, per_step, 1};
  auto encode = [&](CUtensorMap* m, CUtensorMapDataType type, int rank, const uint8_t* base, const cuuint64_t* d,
                    const cuuint64_t* s, const cuuint32_t* b, CUtensorMapSwizzle swizzle) {
    return enc(m, type, cuuint32_t(rank), const_cast<uint8_t*>(base), d, s, b, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  return (gate_up ? encode(weights, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, w.packed, g_dims, g_strides, g_box, CU_TENSOR_MAP_SWIZZLE_128B) &&
                        encode(scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, w.scales, gs_dims, gs_strides, gs_box,
                               CU_TENSOR_MAP_SWIZZLE_NONE)
                  : encode(weights, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, w.packed, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) &&
                        encode(scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, w.scales, s_dims, s_strides, s_box,
                               CU_TENSOR_MAP_SWIZZLE_NONE));
}

template <bool MX, int MODE, bool WIDE>
cudaError_t launch_one(const FewMatrix& w, StreamParams p, int num_sms, cudaStream_t st) {
  auto kernel = stream_kernel<MX, MODE, WIDE>;
  CUtensorMap weights, scales;
  if (!weight_maps(&weights, &scales, w, p.E, MODE == kGateUp)) return cudaErrorInvalidValue;
  // Stages of weights as their scales have columns of tensor memory, of terms as fit beside them and the tile's
  // sums: the weights come from memory and wait longer.  (The terms' scales of T tokens in whole kilobytes, so
  // that every stage starts on one.)
  p.term_bytes = (p.T + 7) / 8 * 8 * (kCodeBytes + kTermScales);
  p.stages = WIDE ? 5 : kMaxStages;
  const int sums = p.T * kTileRows * 4, rest = kSmemLimit - 2048 - sums - p.stages * kStageBytes;
  p.term_stages = rest / p.term_bytes < p.stages ? rest / p.term_bytes : p.stages;
  const int smem = 1024 + p.stages * kStageBytes + p.term_stages * p.term_bytes + sums;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  return launch_kernel(kernel, dim3(unsigned(num_sms < kFewMaxGrid ? num_sms : kFewMaxGrid)), dim3(kThreads), smem, st, false,
                       weights, scales, p);
}

template <int MODE>
cudaError_t launch_stream(const FewMatrix& w, int E, StreamParams p, int num_sms, cudaStream_t st) {
  p.E = E;
  p.gscale = MODE == kDown ? nullptr : w.gscale;
  p.N = w.N, p.K = w.K, p.tiled = w.tiled;
  p.wait_us = wait_limit_us();
  // Up to 16 tokens two accumulators and eight stages: with WIDE 16 tokens x [32768, 7168] take 2 % longer, one
  // token through 8 experts of [6144, 2048] 6 %.
  if (p.T <= 16)
    return w.mx ? launch_one<true, MODE, false>(w, p, num_sms, st) : launch_one<false, MODE, false>(w, p, num_sms, st);
  return w.mx ? launch_one<true, MODE, true>(w, p, num_sms, st) : launch_one<false, MODE, true>(w, p, num_sms, st);
}

struct Terms {
  uint8_t* codes;
  uint8_t* scales;
  float* row_scale;
};

// idx: with a plan
template <int SRC>
cudaError_t launch_terms(const void* x, int64_t x_stride, int rows, int K, bool mx, const Terms& t, uint32_t* counters,
                         int n_counters, const int32_t* idx, int T, int k, int E, Plan* plan, cudaStream_t st) {
  const dim3 grid(unsigned((steps_of(K) + kPrepWarps - 1) / kPrepWarps), unsigned(rows + (plan ? 1 : 0)));
  return launch_kernel(mx ? prepare_kernel<true, SRC> : prepare_kernel<false, SRC>, grid, dim3(kPrepThreads),
                       plan ? size_t(E) * 8 : 0, st, false, static_cast<const uint8_t*>(x), x_stride * (SRC == kF32 ? 4 : 2),
                       rows, K, t.codes, t.scales, t.row_scale, counters, n_counters, idx, T, k, E, plan);
}

StreamParams params_of(uint8_t* ws, const Layout& l, int T, const Terms& t, int rows) {
  StreamParams p = {};
  p.T = T, p.rows = rows;
  p.codes = t.codes, p.scales = t.scales, p.row_scale = t.row_scale;
  p.partial = reinterpret_cast<float*>(ws + l.partial);
  p.done = reinterpret_cast<uint32_t*>(ws + l.counters);
  return p;
}

}  // namespace

size_t few_stream_matvec_bytes(int T, int N, int K) { return size_t(layout_of(T, 1, 1, N, K, 0).bytes); }
size_t few_stream_experts_bytes(int T, int k, int H, int I) { return size_t(layout_of(T, k, kMaxSegs, H, H, I).bytes); }

cudaError_t launch_stream_matvec(const void* x, int64_t x_stride, int T, bool fp16, const FewMatrix& w, void* out, void* ws,
                                 int num_sms, cudaStream_t st) {
  const Layout l = layout_of(T, 1, 1, w.N, w.K, 0);
  uint8_t* at = static_cast<uint8_t*>(ws);
  const Terms t = {at + l.codes, at + l.scales, reinterpret_cast<float*>(at + l.row_scale)};
  uint32_t* counters = reinterpret_cast<uint32_t*>(at + l.counters);
  const cudaError_t err = fp16 ? launch_terms<kFp16>(x, x_stride, T, w.K, w.mx, t, counters, l.n_counters, nullptr, T, 1, 0, nullptr, st)
                               : launch_terms<kBf16>(x, x_stride, T, w.K, w.mx, t, counters, l.n_counters, nullptr, T, 1, 0, nullptr, st);
  if (err != cudaSuccess) return err;
  StreamParams p = params_of(at, l, T, t, T);
  p.out = out, p.out_fp16 = fp16;
  return launch_stream<kDense>(w, 1, p, num_sms, st);
}

cudaError_t launch_stream_experts(const void* x, int64_t x_stride, const int32_t* idx, const float* topk_w, int T, int k,
                                  int E, const FewMatrix& gu, const FewMatrix& d, void* out, void* ws, int num_sms,
                                  cudaStream_t st) {
  const Layout l = layout_of(T, k, kMaxSegs, d.N, gu.K, d.K);
  uint8_t* at = static_cast<uint8_t*>(ws);
  Plan* plan = reinterpret_cast<Plan*>(at + l.plan);
  const Terms x_terms = {at + l.codes, at + l.scales, reinterpret_cast<float*>(at + l.row_scale)};
  const Terms h_terms = {at + l.h_codes, at + l.h_scales, reinterpret_cast<float*>(at + l.h_row_scale)};
  cudaError_t err = launch_terms<kBf16>(x, x_stride, T, gu.K, gu.mx, x_terms, reinterpret_cast<uint32_t*>(at + l.counters),
                                        l.n_counters, idx, T, k, E, plan, st);
  if (err != cudaSuccess) return err;
  StreamParams p = params_of(at, l, T, x_terms, T);
  p.k = k, p.idx = idx, p.topk_w = topk_w;
  p.plan = plan;
  p.next_gscale = d.gscale;
  p.out = at + l.h;
  if ((err = launch_stream<kGateUp>(gu, E, p, num_sms, st)) != cudaSuccess) return err;
  err = launch_terms<kF32>(at + l.h, d.K, T * k, d.K, d.mx, h_terms, nullptr, 0, nullptr, T, k, 0, nullptr, st);
  if (err != cudaSuccess) return err;
  StreamParams q = params_of(at, l, T, h_terms, T * k);
  q.k = k, q.plan = plan, q.out = out;
  q.done += l.n_done;
  return launch_stream<kDown>(d, E, q, num_sms, st);
}

cudaError_t stream_flags_address(unsigned** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_stream_flags); }

}  // namespace nvfp4moe
