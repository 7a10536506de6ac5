// The products of a few tokens as one stream of weights over all SMs
// (moe_matvec_*, moe_experts_* from few_stream_takes() on).
//
// The work is a list of stages in order: of a tile (128 rows of a matrix, or
// 64 of gate and the same 64 of up) the steps of 256 columns, of the down
// product all steps of all experts.  Every SM takes an equal range of it,
// whatever tiles that cuts.  A block's producer warp keeps a ring of stages in
// flight (weights by tensor copies, 18 KB, with the activations of the
// tokens that the step needs); its other warps form groups of four, which take
// the stages in turn, 32 rows a warp.  A tile's sums are joined over the
// groups in shared memory.  Where ranges cut a tile, each block leaves its sums
// in the workspace, and the one that is last adds them in the order of the
// ranges: a repeated call gives the same bits.
//
// The activations become float16 beforehand, and h when the blocks of its 256
// columns are complete: by the block that completed them.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "../../include/nvfp4few.h"
#include "few_common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "mla_common.cuh"
#include "sm103_ptx.cuh"

namespace nvfp4moe {
using namespace few;
namespace {

__device__ unsigned g_stream_flags = 0;

constexpr int kWeightBytes = 128 * 128;         // of a stage
constexpr int kScaleBytes = 2048;
constexpr int kTileRows = 128;
constexpr int kRedStride = kTileRows + 4;       // floats; of one token's sums, without bank conflicts
constexpr int kMinShare = 4;                    // stages
constexpr int kJoinWarps = 3;

template <int NB>
struct Shape {
  static constexpr int kWarps = NB == 1 ? 16 : 12;              // consumers; with 16 warps in all, 128 registers each
  static constexpr int kGroups = kWarps / 4;
  // A multiple of the groups, so that a slot of the ring is always the same
  // group's: with another number a group could come to a slot whose previous
  // stage, another group's, has not landed yet, and take that phase of its barrier for its own.
  static constexpr int kStages = NB == 1 ? 8 : 6;
  static constexpr int kProducer = kWarps, kJoiner = kWarps + 1;  // first warps of the other roles
  static constexpr int kStageBytes = kWeightBytes + kScaleBytes + 8 * NB * kUnitBytes;
  static constexpr int kThreads = 32 * (kWarps + 1 + kJoinWarps);
  static constexpr int kSmem = kStages * kStageBytes + kUnitBytes + 8 * NB * kRedStride * 4 + 1024;
  static_assert(kStages % kGroups == 0 && kSmem <= 227 * 1024);
};

struct StreamParams {
  const float* gscale;       // null: 1
  const float* next_gscale;  // gate/up: of the down matrices
  const uint8_t* frag;       // activations as float16: [step][row][kUnitBytes]
  const float* factor;       // [step][row]
  int rows;                  // of frag
  int T, k, E, N, K, tiled, out_fp16;
  const int32_t* idx;
  const float* topk_w;
  void* out;                 // [T, N], or h [T * k, N / 2] float32
  uint8_t* h_frag;
  float* h_factor;
  const Plan* plan;
  float* partial;            // [2 * grid][T][128]
  uint32_t* done;            // blocks that are through with a cut tile
  uint32_t* done_block;      // tiles of 256 columns of h that are complete
  uint32_t wait_us;
};

// Where piece j of a row's step lies in its kUnitBytes: odd rows swap pairs,
// so that two rows are read without bank conflicts.
__device__ __forceinline__ int piece_at(int j, int row) { return (j ^ (row & 1)) * 64; }

// ---- activations, counters and plan beforehand ---------------------------------------
constexpr int kPrepThreads = 256;

template <int SRC>
__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(const void* x, int64_t x_stride, int T, int K, uint8_t* frag,
                                                               float* factor, uint32_t* counters, int n_counters,
                                                               const int32_t* idx, int k, int E, Plan* plan) {
  extern __shared__ uint32_t words[];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  if (plan && blockIdx.x == 0) {
    write_plan<kPrepThreads>(idx, T, k, E, plan, &g_stream_flags, words, reinterpret_cast<int*>(words + E));
    return;
  }
  const int first = plan ? 1 : 0, lane = threadIdx.x & 31;
  const int block = blockIdx.x - first, blocks = gridDim.x - first;
  for (int i = block * kPrepThreads + threadIdx.x; i < n_counters; i += blocks * kPrepThreads) counters[i] = 0;
  const int items = T * ((K + kStep - 1) / kStep);
  for (int item = block * (kPrepThreads / 32) + (threadIdx.x >> 5); item < items; item += blocks * (kPrepThreads / 32)) {
    const int step = item / T, t = item - step * T;
    float v[8];
    load_block<SRC>(v, static_cast<const uint8_t*>(x) + t * x_stride * 2, step, K, lane);
    uint4 h;
    const float f = block_to_half(v, &h);
    *reinterpret_cast<uint4*>(frag + int64_t(item) * kUnitBytes + piece_at(lane & 7, t) + (lane >> 3) * 16) = h;
    if (lane == 0) factor[item] = f;
  }
}

// ---- the stream ---------------------------------------------------------------------
// The experts of at most 32 ids, in ascending order, by one warp: their number,
// and (unless null) the list.  What the plan says, without waiting for it.
__device__ __forceinline__ int experts_of_warp(const int32_t* idx, int n, int E, int lane, int* list) {
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
    if (first) list[at] = e;
    __syncwarp();
  }
  return __popc(leaders);
}

// Adds bytes that the current phase of a barrier waits for.
__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

template <bool MX, int MODE, int NB>
__global__ void __launch_bounds__(Shape<NB>::kThreads, 1) stream_kernel(const __grid_constant__ CUtensorMap weights,
                                                                        const __grid_constant__ CUtensorMap scales,
                                                                        const StreamParams p) {
  using S = Shape<NB>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t s_full[S::kStages], s_empty[S::kStages];
  __shared__ __align__(8) uint64_t s_red[S::kGroups + 1];
  __shared__ mla::WaitCtl s_ctl;
  __shared__ int s_last, s_token[32], s_expert[32];
  __shared__ float s_weight[32];
  uint8_t* smem = raw + ((1024 - (ptx::smem_u32(raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = mla::uniform(tid >> 5);
  const uint32_t full = ptx::smem_u32(s_full), empty = ptx::smem_u32(s_empty);
  // a tile's sums: barrier 0 opens them to the first group, each group opens them to the next, the last to the joiners
  const uint32_t red_bar = ptx::smem_u32(s_red);
  uint8_t* zeros = smem + S::kStages * S::kStageBytes;   // a step of a token that is not there
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      ptx::mbar_init(full + 8 * i, 1);
      ptx::mbar_init(empty + 8 * i, 4);        // the warps of a group
    }
    ptx::mbar_init(red_bar, kJoinWarps);
    for (int i = 1; i <= S::kGroups; ++i) ptx::mbar_init(red_bar + 8 * i, 4);
    ptx::fence_barrier_init();
    s_ctl.abort = 0;
    s_ctl.limit_us = p.wait_us;
    s_ctl.flags = &g_stream_flags;
    ptx::prefetch_tmap(&weights);
    ptx::prefetch_tmap(&scales);
  }
  if (tid < kUnitBytes / 4) reinterpret_cast<uint32_t*>(zeros)[tid] = 0;
  __syncthreads();

  // The kernel before is one of the same call: prepare_kernel, or before the
  // down product the gate/up one.  Both let the next be launched after their own wait, so what
  // was there before the call (weights, ids), and for the down product the
  // plan, can be read before this kernel's wait (from L2).
  const bool producer = warp == S::kProducer;
  const bool early = MODE != kGateUp || p.T * p.k <= 32;   // the experts are known before the wait
  if (!producer || !early) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
  }
  const int nseg = MODE == kDense ? 1
                   : MODE == kGateUp && early ? experts_of_warp(p.idx, p.T * p.k, p.E, lane, producer ? s_expert : nullptr)
                                              : __ldcg(&p.plan->nseg);
  if (MODE == kDown && nseg == 0) {            // no token has an expert
    ptx::grid_dep_wait();
    for (int64_t i = int64_t(blockIdx.x) * S::kThreads + tid; i < int64_t(p.T) * p.N; i += int64_t(gridDim.x) * S::kThreads)
      static_cast<uint16_t*>(p.out)[i] = 0;
    return;
  }
  const int steps = (p.K + kStep - 1) / kStep, seg_tiles = MODE == kGateUp ? p.N / kTileRows : 1;
  const int tiles = MODE == kGateUp ? nseg * seg_tiles : p.N / kTileRows;
  const int length = MODE == kDown ? nseg * steps : steps;             // stages of a tile
  const int64_t all = int64_t(tiles) * length;
  const int per = int(max(int64_t(kMinShare), (all + gridDim.x - 1) / gridDim.x));
  const int64_t start = int64_t(blockIdx.x) * per, end = min(all, start + per);
  if (start >= end) return;

  if (producer) {
    if (lane != 0) return;
    const uint64_t policy = ptx::policy_evict_first(), keep = ptx::policy_evict_normal();
    const int blocks = p.N / 128, kb_all = p.K / (MX ? 128 : 64);
    constexpr int kPerStep = MX ? 2 : 4;       // scale blocks of a step
    struct Place {                             // of a stage: its tile, of an expert's matrix, and step
      int tile, seg, in, step;
      int known, expert, base;                 // the expert's entries in the plan, read when it changes
      uint32_t tokens;
    };
    auto place_of = [&](int64_t s) {
      Place w;
      w.tile = int(s / length);
      const int at = int(s - int64_t(w.tile) * length);
      w.seg = MODE == kGateUp ? w.tile / seg_tiles : (MODE == kDown ? at / steps : 0);
      w.in = MODE == kGateUp ? w.tile - w.seg * seg_tiles : w.tile;
      w.step = MODE == kDown ? at - w.seg * steps : at;
      w.known = -1;
      return w;
    };
    auto advance = [&](Place& w) {
      if (++w.step < steps) return;
      w.step = 0;
      if (MODE == kDown && ++w.seg < nseg) return;
      if (MODE == kDown) w.seg = 0;
      ++w.tile, ++w.in;
      if (MODE == kGateUp && w.in == seg_tiles) w.in = 0, ++w.seg;
    };
    auto load_weights = [&](Place& w, int st) {
      if (MODE != kDense && w.seg != w.known) {
        w.known = w.seg;
        w.expert = MODE == kGateUp && early ? s_expert[w.seg] : __ldcg(p.plan->expert + w.seg);
        w.tokens = MODE == kGateUp && early ? 0 : __ldcg(p.plan->tokens + w.seg);
        w.base = MODE == kGateUp && early ? 0 : __ldcg(p.plan->base + w.seg);
      }
      const int e = MODE == kDense ? 0 : w.expert;
      const uint32_t bar = full + 8 * st, dst = ptx::smem_u32(smem + st * S::kStageBytes);
      expect_tx(bar, kWeightBytes + kPerStep * 512);
      if (MODE == kGateUp) {                   // 16 rows of each 32 of a block of 128, of gate and of up
        const int half = w.in & 1;
#pragma unroll
        for (int up = 0; up < 2; ++up) {
          const int blk = e * blocks + (w.in >> 1) + up * (blocks / 2);
          ptx::tma_load_3d(dst + up * (kWeightBytes / 2), &weights, bar, p.tiled ? 0 : w.step * 128, 16 * half,
                           (p.tiled ? blk * steps + w.step : blk) * 4, policy);
          ptx::tma_load_2d(dst + kWeightBytes + up * 1024, &scales, bar, 64 * half, blk * kb_all + w.step * kPerStep, policy);
        }
      } else {
        const int blk = e * blocks + w.in;
        ptx::tma_load_2d(dst, &weights, bar, p.tiled ? 0 : w.step * 128, (p.tiled ? blk * steps + w.step : blk) * 128, policy);
        ptx::tma_load_2d(dst + kWeightBytes, &scales, bar, 0, blk * kb_all + w.step * kPerStep, policy);
      }
    };
    int seen = -1;                             // the expert whose tokens these are
    uint32_t who = 0;
    int base = 0;
    auto load_activations = [&](const Place& w, int st) {
      if (MODE != kDense && w.seg != seen) {
        seen = w.seg;
        const bool have = w.known == w.seg && !(MODE == kGateUp && early);
        who = have ? w.tokens : p.plan->tokens[w.seg];
        base = have ? w.base : p.plan->base[w.seg];
      }
      const uint32_t bar = full + 8 * st, dst = ptx::smem_u32(smem + st * S::kStageBytes) + kWeightBytes + kScaleBytes;
      const uint8_t* from = p.frag + int64_t(w.step) * p.rows * kUnitBytes;
      uint32_t tokens = who;
      const int m = MODE == kDense ? p.T : __popc(tokens);
      ptx::mbar_arrive_expect_tx(bar, m * kUnitBytes);
      if (MODE == kGateUp && m < p.T) {
        for (int slot = 0; slot < m; ++slot) {
          ptx::bulk_load(dst + slot * kUnitBytes, from + (__ffs(tokens) - 1) * kUnitBytes, kUnitBytes, bar, keep);
          tokens &= tokens - 1;
        }
      } else {
        ptx::bulk_load(dst, from + (MODE == kDown ? base : 0) * kUnitBytes, m * kUnitBytes, bar, keep);
      }
    };
    Place w = place_of(start), b = w;
    const int n = int(end - start), ahead = n < S::kStages ? n : S::kStages;
    for (int i = 0; i < ahead; ++i) {
      load_weights(w, i);
      advance(w);
    }
    ptx::grid_dep_wait();
    for (int i = 0; i < ahead; ++i) {
      load_activations(b, i);
      advance(b);
    }
    int i = ahead, st = 0, parity = 0;
    for (; i < n; ++i) {
      if (!mla::wait_phase(empty + 8 * st, parity, &s_ctl)) break;
      load_weights(w, st);
      load_activations(w, st);
      advance(w);
      if (++st == S::kStages) st = 0, parity ^= 1;
    }
    if (i < n)                                 // given up: the block's copies land before it leaves
      for (int j = max(0, i - S::kStages); j < i; ++j) mla::drain_phase(full + 8 * (j % S::kStages), (j / S::kStages) & 1);
    return;
  }

  float* red = reinterpret_cast<float*>(zeros + kUnitBytes);   // a tile's sums: [token][row]

  if (warp >= S::kJoiner) {
    // ---- joiners: sums over the groups and the blocks, results
    constexpr int kThreads = 32 * kJoinWarps;
    const int id = tid - 32 * S::kJoiner, my_warp = warp - S::kJoiner;
    int parity = 0;
    for (int tile = int(start / length); int64_t(tile) * length < end; ++tile, parity ^= 1) {
      const int64_t tile_start = int64_t(tile) * length;
      const int seg = MODE == kGateUp ? tile / seg_tiles : 0;
      const uint32_t tokens = MODE == kGateUp ? p.plan->tokens[seg] : 0;
      const int m = MODE == kGateUp ? __popc(tokens) : p.T;
      auto token_of = [&](int slot) { return MODE == kGateUp ? s_token[slot] : slot; };
      if (MODE == kGateUp) {
        const int e = p.plan->expert[seg];
        if (my_warp == 0 && ((tokens >> lane) & 1)) s_token[__popc(tokens & ((1u << lane) - 1))] = lane;
        mla::bar_sync(1, kThreads);
        for (int i = my_warp; i < m; i += kJoinWarps) {      // the tokens' weights of this expert
          const int t = s_token[i];
          float w = lane < p.k && p.idx[t * p.k + lane] == e ? p.topk_w[t * p.k + lane] : 0.0f;
#pragma unroll
          for (int d = 16; d; d >>= 1) w += __shfl_xor_sync(kFull, w, d);
          if (lane == 0) s_weight[i] = w;
        }
        mla::bar_sync(1, kThreads);
      }
      mla::wait_phase(red_bar + 8 * S::kGroups, parity, &s_ctl);
      auto joined = [&](int row, int t) { return *reinterpret_cast<const float4*>(red + t * kRedStride + row); };
      auto release = [&] {                     // the consumers may write the next tile's sums
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(red_bar);
      };
      const int first = int(tile_start / per), last = int((tile_start + length - 1) / per);
      const bool whole = first == last;
      auto slot_of = [&](int block) {          // a block's first range of a cut tile, or its last
        return p.partial + int64_t(2 * block + (int64_t(block) * per > tile_start ? 0 : 1)) * p.T * kTileRows;
      };
      if (!whole) {
        float* to = slot_of(blockIdx.x);
        for (int i = id; i < m * (kTileRows / 4); i += kThreads) {
          const int row = 4 * (i % (kTileRows / 4)), t = token_of(i / (kTileRows / 4));
          *reinterpret_cast<float4*>(to + t * kTileRows + row) = joined(row, t);
        }
        release();
        __threadfence();
        mla::bar_sync(1, kThreads);
        if (id == 0) {
          s_last = atomicAdd(p.done + tile, 1u) == uint32_t(last - first);
          __threadfence();
        }
        mla::bar_sync(1, kThreads);
        if (!s_last) continue;
      }
      auto value = [&](int row, int t) {       // four rows
        if (whole) return joined(row, t);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int b = first; b <= last; ++b) {
          const float4 a = __ldcg(reinterpret_cast<const float4*>(slot_of(b) + t * kTileRows + row));
          v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
        }
        return v;
      };
      if (MODE == kGateUp) {
        const int I = p.N / 2, in = tile - seg * seg_tiles, e = p.plan->expert[seg], base = p.plan->base[seg];
        const float scale = p.gscale ? p.gscale[e] : 1.0f, next = p.next_gscale ? p.next_gscale[e] : 1.0f;
        float* h = static_cast<float*>(p.out);
        for (int i = id; i < 16 * m; i += kThreads) {
          const int r = 4 * (i & 15), slot = i >> 4, t = s_token[slot];
          const float4 gate = value(r, t), up = value(64 + r, t);
          const float w = s_weight[slot] * next;
          auto gated = [&](float a, float b) {
            a *= scale;
            return a / (1.0f + expf(-a)) * (b * scale) * w;
          };
          const int col = (in >> 1) * 128 + 32 * (r >> 4) + 16 * (in & 1) + (r & 15);
          *reinterpret_cast<float4*>(h + int64_t(base + slot) * I + col) =
              make_float4(gated(gate.x, up.x), gated(gate.y, up.y), gated(gate.z, up.z), gated(gate.w, up.w));
        }
        if (whole) release();
        // the block that completes 256 columns converts them
        const int block = in >> 2, in_block = min(4, seg_tiles - 4 * block);
        __threadfence();
        mla::bar_sync(1, kThreads);
        if (id == 0) {
          s_last = atomicAdd(p.done_block + seg * ((seg_tiles + 3) / 4) + block, 1u) == uint32_t(in_block - 1);
          __threadfence();
        }
        mla::bar_sync(1, kThreads);
        if (s_last) {
          const int64_t rows = int64_t(p.T) * p.k;
          for (int i = my_warp; i < m; i += kJoinWarps) {
            const int row = base + i, c = block * kStep + 8 * lane;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
              const float4 a = c < I ? __ldcg(reinterpret_cast<const float4*>(h + int64_t(row) * I + c + j))
                                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              v[j] = a.x, v[j + 1] = a.y, v[j + 2] = a.z, v[j + 3] = a.w;
            }
            uint4 x;
            const float fac = block_to_half(v, &x);
            *reinterpret_cast<uint4*>(p.h_frag + (block * rows + row) * kUnitBytes + piece_at(lane & 7, row) + (lane >> 3) * 16) = x;
            if (lane == 0) p.h_factor[block * rows + row] = fac;
          }
        }
      } else {
        const float scale = MODE == kDense && p.gscale ? p.gscale[0] : 1.0f;
        for (int i = id; i < p.T * (kTileRows / 4); i += kThreads) {
          const int row = 4 * (i % (kTileRows / 4)), t = i / (kTileRows / 4);
          const float4 v = value(row, t);
          uint2 r;
          if (MODE == kDense && p.out_fp16) {
            const __half2 lo = __floats2half2_rn(v.x * scale, v.y * scale), hi = __floats2half2_rn(v.z * scale, v.w * scale);
            r = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * scale, v.y * scale),
                                 hi = __floats2bfloat162_rn(v.z * scale, v.w * scale);
            r = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          }
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + int64_t(t) * p.N + tile * kTileRows + row) = r;
        }
        if (whole) release();
      }
    }
    return;
  }

  // ---- consumers: warp q of group `group`
  const int q = warp & 3, group = warp >> 2, g = lane >> 2, tg = lane & 3;
  // byte offsets within a stage: the lane's rows (g of tile 0) and 16-byte pieces (swizzled), its scales
  const int row0 = (MODE == kGateUp ? 16 : 32) * q, tile_rows = MODE == kGateUp ? 64 : 16;
  const int w_at = (row0 + g) * 128, w_lo = ((2 * tg) ^ g) * 16, w_hi = ((2 * tg + 1) ^ g) * 16;
  const int kb = MX ? tg >> 1 : tg;
  const int s_at = kWeightBytes + kb * (MODE == kGateUp ? 256 : 512) + g * 16 + q * 4 + (MX ? (tg & 1) * 2 : 0);
  const int s_tile = MODE == kGateUp ? 1024 : 256;

  int tile = int(start / length), at = int(start - int64_t(tile) * length);
  int turn = 0, st = 0, parity = 0, red_parity = 1;
  float total[2][NB][4];
  int seen = -1, base = 0;                     // down: the expert whose plan entries these are
  uint32_t mine = 0;

  for (int64_t s = start; s < end;) {
    const int64_t tile_start = int64_t(tile) * length;
    const int stop = int(min(int64_t(length), end - tile_start));     // of this tile
    uint32_t tokens = p.T == 32 ? kFull : (1u << p.T) - 1;
    int seg = 0, step = at;
    if (MODE == kGateUp) {
      seg = tile / seg_tiles;
      tokens = p.plan->tokens[seg];
    } else if (MODE == kDown) {
      seg = at / steps;
      step = at - seg * steps;
    }
#pragma unroll
    for (int i = 0; i < 2 * NB * 4; ++i) (&total[0][0][0])[i] = 0.0f;

    for (; at < stop; ++at, ++s) {
      if (turn == group) {
        if (MODE == kDown && seg != seen) seen = seg, mine = p.plan->tokens[seg], base = p.plan->base[seg];
        if (MODE == kDown) tokens = mine;
        // the factors of this lane's columns, for the end
        float f[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int t = 8 * b + 2 * tg + c;
            const int row = MODE == kDown ? base + __popc(tokens & ((1u << t) - 1)) : t;
            f[b][c] = (tokens >> t) & 1 ? p.factor[int64_t(step) * p.rows + row] : 0.0f;
          }
        mla::wait_phase(full + 8 * st, parity, &s_ctl);
        __syncwarp();
        const uint8_t* stage = smem + st * S::kStageBytes;
        // where the lane's token of each eight lies: pieces 2i and 2i + 1 (piece_at)
        const uint8_t *even[NB], *odd[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int t = 8 * b + g, slot = __popc(tokens & ((1u << t) - 1));
          const int swap = ((MODE == kDown ? base + slot : t) & 1) * 64;
          const uint8_t* from = ((tokens >> t) & 1 ? stage + kWeightBytes + kScaleBytes + slot * kUnitBytes : zeros) + tg * 16;
          even[b] = from + swap;
          odd[b] = from + (64 - swap);
        }
        const bool inside = step * kStep + tg * 64 < p.K;
        uint32_t sw[4], ref[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {          // (tile i / 2, rows g or g + 8)
          const uint8_t* sp = stage + s_at + (i >> 1) * s_tile + (i & 1) * 128;
          sw[i] = MX ? uint32_t(*reinterpret_cast<const uint16_t*>(sp)) : *reinterpret_cast<const uint32_t*>(sp);
          if (!inside) sw[i] = 0;
          if (MX) {
            uint32_t top = max(sw[i] & 255u, sw[i] >> 8);
            top = max(top, __shfl_xor_sync(kFull, top, 1));
            ref[i] = max(top, __shfl_xor_sync(kFull, top, 2));
          }
        }
        float acc[2][NB][4];
#pragma unroll
        for (int i = 0; i < 2 * NB * 4; ++i) (&acc[0][0][0])[i] = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {          // the lane's two 16-byte pieces of each row
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = *reinterpret_cast<const uint4*>(stage + w_at + ((i >> 1) * tile_rows + (i & 1) * 8) * 128 + (h ? w_hi : w_lo));
          uint32_t sc[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (!MX && (j & 1) == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t two = ue4m3x2_to_half(h ? sw[i] >> 16 : sw[i]);
                sc[i] = __byte_perm(two, two, j ? 0x3232 : 0x1010);
              }
            }
            if (MX && j == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int x = int(h ? sw[i] >> 8 : sw[i] & 255u) - int(ref[i]) + 28;
                sc[i] = uint32_t(max(x, 0)) * 0x04000400u;   // exponent fields of 2^(scale - reference + 13), or 0
              }
            }
            uint32_t a[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              codes_to_half(j == 0 ? w[i].x : (j == 1 ? w[i].y : (j == 2 ? w[i].z : w[i].w)), a[i]);
#pragma unroll
              for (int c = 0; c < 4; ++c) a[i][c] = hmul2(a[i][c], sc[i]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              if (NB > 1 && ((tokens >> (8 * b)) & 255u) == 0) continue;
              const uint4 x = *reinterpret_cast<const uint4*>((j & 1 ? odd[b] : even[b]) + (4 * h + (j & 2)) * 64);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                mma(acc[i][b], a[2 * i][0], a[2 * i + 1][0], a[2 * i][1], a[2 * i + 1][1], x.x, x.y);
                mma(acc[i][b], a[2 * i][2], a[2 * i + 1][2], a[2 * i][3], a[2 * i + 1][3], x.z, x.w);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(empty + 8 * st);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if ((tokens >> (8 * b + 2 * tg + c)) & 1) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float v = acc[i >> 1][b][(i & 1) * 2 + c];
                if (MX) {
                  const int x = int(ref[i]) - 140;   // 2^(ref - 127 - 13) as two factors of float32's normal range
                  v = ref[i] == 255 ? __int_as_float(0x7FFFFFFF) : v * exp2i(x >> 1);
                  total[i >> 1][b][(i & 1) * 2 + c] += v * f[b][c] * exp2i(x - (x >> 1));
                } else {
                  total[i >> 1][b][(i & 1) * 2 + c] += v * f[b][c];
                }
              }
            }
      }
      if (++turn == S::kGroups) turn = 0;
      if (++st == S::kStages) st = 0, parity ^= 1;
      if (++step == steps) step = 0, ++seg;
    }

    // ---- the tile's sums: a group after the other, so in a fixed order
    mla::wait_phase(red_bar + 8 * group, red_parity ^ (group ? 1 : 0), &s_ctl);
    red_parity ^= 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = row0 + (i >> 1) * tile_rows + (i & 1) * 8 + g;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float* to = red + (8 * b + 2 * tg + c) * kRedStride + row;
          const float v = total[i >> 1][b][(i & 1) * 2 + c];
          *to = group ? *to + v : v;
        }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(red_bar + 8 * (group + 1));
    at = 0;
    ++tile;
  }
}

int64_t steps_of(int K) { return (K + kStep - 1) / kStep; }
int64_t round256(int64_t b) { return (b + 255) & ~int64_t(255); }

// The parts of a workspace.
struct Layout {
  int64_t plan, counters, frag, factor, h, h_frag, h_factor, partial, bytes;
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
  l.n_counters = l.n_done + int(I ? segs * ((I / 64 + 3) / 4) + N / kTileRows : 0);
  l.counters = take(int64_t(l.n_counters) * 4);
  l.frag = take(T * steps_of(K) * kUnitBytes);
  l.factor = take(T * steps_of(K) * 4);
  if (I) {
    l.h = take(rows * I * 4);
    l.h_frag = take(rows * steps_of(I) * kUnitBytes);
    l.h_factor = take(rows * steps_of(I) * 4);
  }
  l.partial = take(int64_t(2) * kFewMaxGrid * T * kTileRows * 4);
  l.bytes = at;
  return l;
}

// The weights of all experts: boxes of 128 rows x 128 bytes (zeros past K/2)
// or, for the gated product, of 16 rows of each 32 of them; and the scales'
// blocks of 512 bytes, or their halves.
bool weight_maps(CUtensorMap* weights, CUtensorMap* scales, const FewMatrix& w, int E, bool gate_up) {
  auto enc = mla::tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t row = w.tiled ? 128 : w.K / 2, rows = cuuint64_t(E) * w.N * (w.tiled ? steps_of(w.K) : 1);
  const cuuint64_t dims[3] = {row, gate_up ? 32 : rows, rows / 32}, strides[2] = {row, 32 * row};
  const cuuint32_t box[3] = {128, cuuint32_t(gate_up ? 16 : 128), 4}, unit[3] = {1, 1, 1};
  const int per_step = w.mx ? 2 : 4;
  const cuuint64_t s_dims[2] = {128, cuuint64_t(E) * (w.N / 128) * (w.K / (w.mx ? 128 : 64))}, s_strides[1] = {512};
  const cuuint32_t s_box[2] = {cuuint32_t(gate_up ? 64 : 128), cuuint32_t(per_step)};
  return enc(weights, CU_TENSOR_MAP_DATA_TYPE_UINT8, gate_up ? 3 : 2, const_cast<uint8_t*>(w.packed), dims, strides, box, unit,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
         enc(scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(w.scales), s_dims, s_strides, s_box, unit,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool MX, int MODE, int NB>
cudaError_t launch_one(const FewMatrix& w, const StreamParams& p, int num_sms, cudaStream_t st) {
  auto kernel = stream_kernel<MX, MODE, NB>;
  CUtensorMap weights, scales;
  if (!weight_maps(&weights, &scales, w, p.E, MODE == kGateUp)) return cudaErrorInvalidValue;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NB>::kSmem);
  if (err != cudaSuccess) return err;
  return launch_kernel(kernel, dim3(unsigned(num_sms < kFewMaxGrid ? num_sms : kFewMaxGrid)), dim3(Shape<NB>::kThreads),
                       Shape<NB>::kSmem, st, false, weights, scales, p);
}

template <int MODE>
cudaError_t launch_stream(const FewMatrix& w, int E, StreamParams p, int num_sms, cudaStream_t st) {
  p.E = E;
  p.gscale = MODE == kDown ? nullptr : w.gscale;
  p.N = w.N, p.K = w.K, p.tiled = w.tiled;
  p.wait_us = wait_limit_us();
  if (p.T <= 8) return w.mx ? launch_one<true, MODE, 1>(w, p, num_sms, st) : launch_one<false, MODE, 1>(w, p, num_sms, st);
  if (p.T <= 16) return w.mx ? launch_one<true, MODE, 2>(w, p, num_sms, st) : launch_one<false, MODE, 2>(w, p, num_sms, st);
  return w.mx ? launch_one<true, MODE, 4>(w, p, num_sms, st) : launch_one<false, MODE, 4>(w, p, num_sms, st);
}

template <int SRC>
cudaError_t launch_prepare_few(const void* x, int64_t x_stride, int T, int K, uint8_t* ws, const Layout& l, const int32_t* idx,
                               int k, int E, cudaStream_t st) {
  const int64_t items = T * steps_of(K);
  const int64_t warps = kPrepThreads / 32;
  int64_t blocks = (items + warps - 1) / warps;
  if (blocks > 304) blocks = 304;
  return launch_kernel(prepare_kernel<SRC>, dim3(unsigned(blocks + (idx ? 1 : 0))), dim3(kPrepThreads), idx ? size_t(E) * 8 : 0, st,
                       false, x, x_stride, T, K, ws + l.frag, reinterpret_cast<float*>(ws + l.factor),
                       reinterpret_cast<uint32_t*>(ws + l.counters), l.n_counters, idx, k, E,
                       idx ? reinterpret_cast<Plan*>(ws + l.plan) : nullptr);
}

StreamParams params_of(uint8_t* ws, const Layout& l, int T) {
  StreamParams p = {};
  p.T = T, p.rows = T;
  p.frag = ws + l.frag;
  p.factor = reinterpret_cast<float*>(ws + l.factor);
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
  const cudaError_t err = fp16 ? launch_prepare_few<kFp16>(x, x_stride, T, w.K, at, l, nullptr, 1, 0, st)
                               : launch_prepare_few<kBf16>(x, x_stride, T, w.K, at, l, nullptr, 1, 0, st);
  if (err != cudaSuccess) return err;
  StreamParams p = params_of(at, l, T);
  p.out = out, p.out_fp16 = fp16;
  return launch_stream<kDense>(w, 1, p, num_sms, st);
}

cudaError_t launch_stream_experts(const void* x, int64_t x_stride, const int32_t* idx, const float* topk_w, int T, int k,
                                  int E, const FewMatrix& gu, const FewMatrix& d, void* out, void* ws, int num_sms,
                                  cudaStream_t st) {
  const Layout l = layout_of(T, k, kMaxSegs, d.N, gu.K, d.K);
  uint8_t* at = static_cast<uint8_t*>(ws);
  cudaError_t err = launch_prepare_few<kBf16>(x, x_stride, T, gu.K, at, l, idx, k, E, st);
  if (err != cudaSuccess) return err;
  StreamParams p = params_of(at, l, T);
  p.k = k, p.idx = idx, p.topk_w = topk_w;
  p.plan = reinterpret_cast<const Plan*>(at + l.plan);
  p.next_gscale = d.gscale;
  p.out = at + l.h;
  p.h_frag = at + l.h_frag;
  p.h_factor = reinterpret_cast<float*>(at + l.h_factor);
  const int blocks = d.K / 64;                // tiles of an expert's h
  p.done_block = p.done + l.n_done;
  if ((err = launch_stream<kGateUp>(gu, E, p, num_sms, st)) != cudaSuccess) return err;
  p.rows = T * k;
  p.frag = p.h_frag;
  p.factor = p.h_factor;
  p.out = out;
  const int64_t segs = int64_t(T) * k < kMaxSegs ? int64_t(T) * k : kMaxSegs;
  p.done = p.done_block + segs * ((blocks + 3) / 4);
  return launch_stream<kDown>(d, E, p, num_sms, st);
}

cudaError_t stream_flags_address(unsigned** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_stream_flags); }

}  // namespace nvfp4moe
