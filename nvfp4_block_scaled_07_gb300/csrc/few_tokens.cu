// Products of a few tokens with 4-bit matrices (moe_matvec_*, moe_experts_*):
// 16-bit activations against NVFP4 or MXFP4 weights in the layouts of the
// grouped GEMM.
//
//   y[t, n] = s sum_k x[t, k] code[n, k] scale[n, k / B]          B = 16 or 32
//   experts:  h = silu(x Wg^T) * (x Wu^T) for each routed token, then
//   out[t] = sum over its experts of weight * h Wd^T
//
// This is the kernel of small products; few_stream.cu takes the rest (the rule
// stands at takes_matvec).  What bounds these is latency: a launch (two for the
// experts), one read of the activations and a few steps of weights.  One token x
// [512, 2048] takes 2.7 us, three tokens through two of 8 experts each (H 256, I
// 128) 7.7 us with the plan.  mma.sync takes the codes as float16: a code times its ue4m3 scale has at most 6 significant bits and
// lies in 2^-10 .. 2688, so the product is exact.  E8M0 scales do not fit that
// range: of the 256 values of a row that a step takes, the largest scale is
// the reference 2^X, codes are multiplied by 2^(scale - X + 13), and the sum
// by 2^(X - 13).  Scales below 2^-27 of that reference, which hardly ever are, take
// another pass over the step with the largest of them as its reference.
// Activations become float16 too, in blocks of 256 values of a token that are
// multiplied by the power of two which brings the largest into 2^14 .. 2^15:
// exact for every bf16 or fp16 value above 2^-28 of its block's largest, and
// smaller ones are off by at most 2^-39 of it.  The gated products h (float32)
// become two such numbers, the second what the rounding to the first leaves:
// 22 bits, off by 2^-22 of themselves, as four float32 roundings.  (One number,
// 11 bits, took 7.4 us instead of 7.7 for the three tokens, but differences of
// nearly equal products were lost in it, and the bf16 results were 8e-4 off in
// norm where they now are those of float32.)  Sums are float32.
//
// A warp takes 32 rows of a matrix as two 16-row tiles (of gate and of up in
// the gated product) and steps of 256 of its columns, a lane 32 bytes of four
// rows a step.  The rows of a tile are four of each 32, because the blocked
// scale layout keeps the scales of rows r, r + 32, r + 64 and r + 96 together:
// so a tile's scales are whole sectors.  Eight columns of a tile's product are
// tokens.  The warps of a block take the steps of the same rows in turn, their
// sums are joined in shared memory in a fixed order (with warps on rows of
// their own 8 tokens x [512, 1024] took 6.1 us instead of 3.9).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/nvfp4few.h"
#include "few_common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "sm103_ptx.cuh"

namespace nvfp4moe {
using namespace few;
namespace {

__device__ unsigned g_few_flags = 0;

constexpr int kThreads = 256, kWarps = 8;
constexpr int kMaxRows = 256;             // routed rows, T * k

struct FewParams {
  const void* x;             // [T, K] of Source, or h [T * k, K] float32
  int64_t x_stride;
  int T, k, E;
  const int32_t* idx;        // [T, k]
  const float* topk_w;
  const uint8_t* packed;
  const uint8_t* scales;
  const float* gscale;       // null: 1
  const float* next_gscale;  // gate/up: the down matrices' scales, null: 1
  int N, K;                  // rows (gate and up together) and columns of one matrix
  int tiled, wide;           // wide: rows start on 32-byte boundaries
  int out_fp16;
  void* out;
  Plan* plan;
};

constexpr int kReach = 27;  // float16 takes scales down to 2^-27 of the largest

// 32 bytes of each of a lane's four rows, and their scale words.
struct Rows {
  uint32_t w[4][8];
  uint32_t s[4];
};

__device__ __forceinline__ void load32(uint32_t (&r)[8], const uint8_t* p, bool wide) {
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w, r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
  }
}

// Where a lane's weights lie: rows g and g + 8 of two tiles, its 32 bytes of a step.
struct Lane {
  int64_t w0, w_tile, w_half, w_step, w_matrix;  // byte offsets
  int64_t s0, s_tile, s_step, s_matrix;
  int tg;
};

template <bool MX>
__device__ __forceinline__ Lane lane_of(const FewParams& p, int rb, int st, int64_t tile_rows, int lane) {
  Lane l;
  const int g = lane >> 2;
  l.tg = lane & 3;
  const int64_t half = p.K / 2, kc = (p.K + 255) / 256, kb = p.K / (MX ? 128 : 64);
  const int r = 4 * st + (g & 3) + 32 * (g >> 2);
  // tile_rows: rows between the two tiles, a multiple of 128 (gate and up) or 4
  if (p.tiled) {
    l.w0 = int64_t(rb) * kc * 16384 + r * 128 + l.tg * 32;
    l.w_tile = (tile_rows / 128) * kc * 16384 + (tile_rows % 128) * 128;
    l.w_half = 64 * 128;
    l.w_step = 16384;
    l.w_matrix = int64_t(p.N / 128) * kc * 16384;
  } else {
    l.w0 = (int64_t(rb) * 128 + r) * half + l.tg * 32;
    l.w_tile = tile_rows * half;
    l.w_half = 64 * half;
    l.w_step = 128;
    l.w_matrix = int64_t(p.N) * half;
  }
  l.s0 = int64_t(rb) * kb * 512 + (4 * st + (g & 3)) * 16 + (g >> 2) * 4 + (MX ? (l.tg >> 1) * 512 + (l.tg & 1) * 2 : l.tg * 512);
  l.s_tile = (tile_rows / 128) * kb * 512 + (tile_rows % 128) * 16;
  l.s_step = MX ? 1024 : 2048;
  l.s_matrix = int64_t(p.N / 128) * kb * 512;
  return l;
}

template <bool MX>
__device__ __forceinline__ void load_rows(Rows& r, const FewParams& p, const Lane& l, int e, int step) {
  if (step * kStep + l.tg * 64 < p.K) {
    const uint8_t* w = p.packed + e * l.w_matrix + l.w0 + step * l.w_step;
    const uint8_t* s = p.scales + e * l.s_matrix + l.s0 + step * l.s_step;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // (tile i / 2, rows g or g + 8)
      load32(r.w[i], w + (i >> 1) * l.w_tile + (i & 1) * l.w_half, p.wide);
      const uint8_t* sp = s + (i >> 1) * l.s_tile + (i & 1) * 8;
      r.s[i] = MX ? uint32_t(__ldg(reinterpret_cast<const uint16_t*>(sp))) : __ldg(reinterpret_cast<const uint32_t*>(sp));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.s[i] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) r.w[i][j] = 0;
    }
  }
}

// The products of a step's weights with the tokens' activations, in two tiles: `from` is this lane's part of them, m tokens'
// pieces apart.  MX: scale(i, half) is a block's scale less its row's reference, as a power of two.
template <bool MX, bool TWO, typename Scale>
__device__ __forceinline__ void multiply(float (&acc)[2][4], const Rows& r, const Scale& scale, const uint8_t* from, int m,
                                         int second, bool has) {
  uint32_t sc[4];                       // the rows' scales of this word as float16 pairs
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!MX && (j & 1) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t two = ue4m3x2_to_half(j < 4 ? r.s[i] : r.s[i] >> 16);
        sc[i] = __byte_perm(two, two, (j & 2) ? 0x3232 : 0x1010);
      }
    }
    if (MX && (j & 3) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)       // exponent fields of 2^(scale - reference + 13), or 0
        sc[i] = uint32_t(max(scale(i, j >> 2) + kReach + 1, 0)) * 0x04000400u;
    }
    uint32_t a[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      codes_to_half(r.w[i][j], a[i]);
#pragma unroll
      for (int q = 0; q < 4; ++q) a[i][q] = hmul2(a[i][q], sc[i]);
    }
#pragma unroll
    for (int part = 0; part < (TWO ? 2 : 1); ++part) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (has) x = *reinterpret_cast<const uint4*>(from + part * second + j * m * 64);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mma(acc[i], a[2 * i][0], a[2 * i + 1][0], a[2 * i][1], a[2 * i + 1][1], x.x, x.y);
        mma(acc[i], a[2 * i][2], a[2 * i + 1][2], a[2 * i][3], a[2 * i + 1][3], x.z, x.w);
      }
    }
  }
}

// The largest of the four lanes that hold a row.
__device__ __forceinline__ int row_max(int v) {
  v = max(v, __shfl_xor_sync(kFull, v, 1));
  return max(v, __shfl_xor_sync(kFull, v, 2));
}

// Whether a lane's block (half of its 32 bytes of a row) has codes other than 0.
__device__ __forceinline__ bool has_codes(const uint32_t (&w)[8], int half) {
  return ((w[4 * half] | w[4 * half + 1] | w[4 * half + 2] | w[4 * half + 3]) & 0x77777777u) != 0;
}

template <bool MX, int SRC, int MODE>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(const FewParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_or[kWarps];
  __shared__ int s_sum[kWarps], s_first[kWarps];
  __shared__ float s_weight[32];
  __shared__ int s_expert[MODE == kDown ? kMaxRows : 1], s_base[MODE == kDown ? kMaxRows : 1];  // the plan
  __shared__ uint32_t s_tokens[MODE == kDown ? kMaxRows : 1];
  __shared__ int s_of_row[MODE == kDown ? kMaxRows : 1];   // the plan's entry of a row of h, or -1
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int steps = (p.K + kStep - 1) / kStep;

  // The experts of this block, the tokens of each and their rows of activations.
  int e = 0, base = 0, nseg = 1;
  uint32_t tokens = p.T == 32 ? kFull : (1u << p.T) - 1;
  if (MODE == kGateUp) {
    const int f = blockIdx.y, n = p.T * p.k;
    if (f == n) {                              // blocks of their own for the down product's plan: one works
      if (blockIdx.x == 0)
        write_plan<kThreads>(p.idx, p.T, p.k, p.E, p.plan, &g_few_flags, reinterpret_cast<uint32_t*>(smem),
                             reinterpret_cast<int*>(smem) + p.E);
      return;
    }
    e = p.idx[f];
    if (e < 0 || e >= p.E) return;             // write_plan raises the flag
    uint32_t bits = 0;
    int below = 0, first = n;
    for (int i = tid; i < n; i += kThreads) {
      const int v = p.idx[i];
      if (v == e) {
        bits |= 1u << (i / p.k);
        first = min(first, i);
      }
      below += v >= 0 && v < e;
    }
    bits = __reduce_or_sync(kFull, bits);
    below = __reduce_add_sync(kFull, below);
    first = __reduce_min_sync(kFull, first);
    if (lane == 0) s_or[warp] = bits, s_sum[warp] = below, s_first[warp] = first;
    __syncthreads();
    tokens = 0;
    for (int w = 0; w < kWarps; ++w) {
      tokens |= s_or[w];
      base += s_sum[w];
      first = min(first, s_first[w]);
    }
    if (first != f) return;                    // the block of the expert's first token has it
    for (int t = warp; t < p.T; t += kWarps) { // a token's weight of this expert
      const bool mine = lane < p.k && p.idx[t * p.k + lane] == e;
      float w = mine ? p.topk_w[t * p.k + lane] : 0.0f;
#pragma unroll
      for (int d = 16; d; d >>= 1) w += __shfl_xor_sync(kFull, w, d);
      if (lane == 0) s_weight[t] = w;
    }
  } else if (MODE == kDown) {
    nseg = p.plan->nseg;
    s_of_row[tid] = -1;
    if (tid < nseg) s_expert[tid] = p.plan->expert[tid], s_base[tid] = p.plan->base[tid], s_tokens[tid] = p.plan->tokens[tid];
    __syncthreads();
    if (tid < nseg)
      for (int i = 0; i < __popc(s_tokens[tid]); ++i) s_of_row[s_base[tid] + i] = tid;
    __syncthreads();
  }
  const int units = nseg * steps;

  // This warp's tiles.
  const int sub = blockIdx.x;
  const int rb = MODE == kGateUp ? sub >> 3 : sub >> 2, st = MODE == kGateUp ? sub & 7 : 2 * (sub & 3);
  const Lane l = lane_of<MX>(p, rb, st, MODE == kGateUp ? p.N / 2 : 4, lane);

  int step = warp, seg = 0;                    // the warps take the columns' steps in turn
  while (step >= steps) step -= steps, ++seg;
  Rows cur;
  if (warp < units) load_rows<MX>(cur, p, l, MODE == kDown ? s_expert[seg] : e, step);

  // Activations as float16: [step][piece j][token of the expert][16 bytes of 4 lane groups]; the
  // second parts of h lie `second` bytes further.
  constexpr bool kTwo = SRC == kF32;
  const int rows = MODE == kDown ? p.T * p.k : p.T;   // an upper bound, also of a gate/up block's tokens
  const int second = rows * steps * kUnitBytes;
  float* factor = reinterpret_cast<float*>(smem + (kTwo ? 2 : 1) * second);
  const int held = MODE == kDown ? rows : __popc(tokens);
  for (int i = warp; i < held * steps; i += kWarps) {
    const int r = i / steps, at = i - r * steps;
    int row = r, slot = r, first = 0, m = held;
    if (MODE == kDown) {
      const int s = s_of_row[r];
      if (s < 0) continue;
      first = s_base[s], slot = r - first, m = __popc(s_tokens[s]);
    } else if (MODE == kGateUp) {
      row = int(__fns(tokens, 0, slot + 1));
    }
    float v[8];
    load_block<SRC>(v, static_cast<const uint8_t*>(p.x) + row * p.x_stride * (SRC == kF32 ? 4 : 2), at, p.K, lane);
    uint4 h, rest;
    const float f = block_to_half<kTwo>(v, &h, &rest);
    uint8_t* dst = smem + (first * steps + at * m) * kUnitBytes + ((lane & 7) * m + slot) * 64 + (lane >> 3) * 16;
    *reinterpret_cast<uint4*>(dst) = h;
    if (kTwo) *reinterpret_cast<uint4*>(dst + second) = rest;
    if (lane == 0) factor[r * steps + at] = f;
  }
  __syncthreads();

  float total[2][4] = {};
  const int g = lane >> 2;

  // A step's products into the totals, tokens of this expert only.
  auto add = [&](const float (&acc)[2][4], const int (&ref)[4]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int t = 2 * l.tg + c;
      if ((tokens >> t) & 1) {
        const int slot = __popc(tokens & ((1u << t) - 1));
        const float f = factor[(MODE == kDown ? base + slot : slot) * steps + step];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = acc[i >> 1][(i & 1) * 2 + c];
          if (MX) {
            if (ref[i] < 0) continue;          // nothing is left of this row
            // 2^(ref - 127 - 13) as two factors of float32's normal range
            const int x = ref[i] - 140;
            v = ref[i] == 255 ? __int_as_float(0x7FFFFFFF) : v * exp2i(x >> 1);
            total[i >> 1][(i & 1) * 2 + c] += v * f * exp2i(x - (x >> 1));
          } else {
            total[i >> 1][(i & 1) * 2 + c] += v * f;
          }
        }
      }
    }
  };

  bool again = false;                   // MX: scales were out of reach
  for (int u = warp; u < units; u += kWarps) {
    // the next step's weights on their way
    int nstep = step + kWarps, next = seg;
    while (nstep >= steps) nstep -= steps, ++next;
    Rows nxt;
    if (u + kWarps < units) load_rows<MX>(nxt, p, l, MODE == kDown ? s_expert[next] : e, nstep);

    if (MODE == kDown) tokens = s_tokens[seg], base = s_base[seg];
    const int m = __popc(tokens);
    // this lane's column: token g
    const bool has = (tokens >> g) & 1;
    const uint8_t* from = smem + ((MODE == kDown ? base : 0) * steps + step * m) * kUnitBytes +
                          __popc(tokens & ((1u << g) - 1)) * 64 + l.tg * 16;

    int ref[4];                         // MX: a row's largest scale of this step
    if (MX) {
      bool far = false;                 // and whether others are out of its reach
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int x = cur.s[i] & 255u, y = cur.s[i] >> 8;
        ref[i] = row_max(max(x, y));
        far |= min(x, y) < ref[i] - kReach;
      }
      if (__any_sync(kFull, far)) {
        far = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          far |= (int(cur.s[i] & 255u) < ref[i] - kReach && has_codes(cur.w[i], 0)) ||
                 (int(cur.s[i] >> 8) < ref[i] - kReach && has_codes(cur.w[i], 1));
        again |= __any_sync(kFull, far);
      }
    }
    float acc[2][4] = {};
    multiply<MX, kTwo>(acc, cur, [&](int i, int half) { return int(half ? cur.s[i] >> 8 : cur.s[i] & 255u) - ref[i]; }, from, m,
                       second, has);
    add(acc, ref);
    cur = nxt;
    step = nstep;
    seg = next;
  }

  // MX: the blocks whose scales were out of reach, pass by pass, each with the largest scale that is left as a reference.
  if (MX && again) {
    constexpr int kDone = -512;         // below every scale and its reach
    step = warp, seg = 0;
    for (int u = warp; u < units; u += kWarps, step += kWarps) {
      while (step >= steps) step -= steps, ++seg;
      load_rows<MX>(cur, p, l, MODE == kDown ? s_expert[seg] : e, step);
      if (MODE == kDown) tokens = s_tokens[seg], base = s_base[seg];
      const int m = __popc(tokens);
      const bool has = (tokens >> g) & 1;
      const uint8_t* from = smem + ((MODE == kDown ? base : 0) * steps + step * m) * kUnitBytes +
                            __popc(tokens & ((1u << g) - 1)) * 64 + l.tg * 16;
      int s[4][2], ref[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i][0] = has_codes(cur.w[i], 0) ? int(cur.s[i] & 255u) : kDone;
        s[i][1] = has_codes(cur.w[i], 1) ? int(cur.s[i] >> 8) : kDone;
        ref[i] = row_max(max(cur.s[i] & 255u, cur.s[i] >> 8));
      }
#pragma unroll 1
      for (int pass = 0; pass < 8; ++pass) {   // a row has eight blocks in a step, of which a pass ends one or more
        bool left = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (s[i][h] >= ref[i] - kReach) s[i][h] = kDone;
          ref[i] = row_max(max(s[i][0], s[i][1]));
          left |= ref[i] != kDone;
        }
        if (!__any_sync(kFull, left)) break;
        float acc[2][4] = {};
        multiply<MX, kTwo>(acc, cur, [&](int i, int half) { return s[i][half] - ref[i]; }, from, m, second, has);
        add(acc, ref);
      }
    }
  }

  // Joins the warps along the columns: [warp][tile][row 0..15][8 tokens].
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float* at = red + (warp * 2 + i) * 128 + 2 * l.tg;
    *reinterpret_cast<float2*>(at + g * 8) = make_float2(total[i][0], total[i][1]);
    *reinterpret_cast<float2*>(at + (g + 8) * 8) = make_float2(total[i][2], total[i][3]);
  }
  __syncthreads();
  auto joined = [&](int tile, int row, int t) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[(w * 2 + tile) * 128 + row * 8 + t];
    return v;
  };
  if (MODE == kGateUp) {
    const int m = __popc(tokens), I = p.N / 2;
    const float s = p.gscale ? p.gscale[e] : 1.0f, s_next = p.next_gscale ? p.next_gscale[e] : 1.0f;
    float* h = static_cast<float*>(p.out);
    for (int i = tid; i < 16 * m; i += kThreads) {
      const int row = i & 15, slot = i >> 4, t = int(__fns(tokens, 0, slot + 1));
      const float gate = joined(0, row, t) * s, up = joined(1, row, t) * s;
      const int col = (sub >> 3) * 128 + (sub & 7) * 4 + (row & 3) + 32 * (row >> 2);
      h[int64_t(base + slot) * I + col] = gate / (1.0f + expf(-gate)) * up * s_weight[t] * s_next;
    }
  } else {
    const float s = MODE == kDense && p.gscale ? p.gscale[0] : 1.0f;
    for (int i = tid; i < 32 * p.T; i += kThreads) {
      const int r = i & 31, t = i >> 5;
      // rows 8 (sub % 4) + 0..7 of each 32 of the 128: the first four of tile 0, the others of tile 1
      const float v = joined((r >> 2) & 1, (r & 3) + 4 * (r >> 3), t) * s;
      const int64_t o = int64_t(t) * p.N + (sub >> 2) * 128 + (sub & 3) * 8 + (r & 7) + 32 * (r >> 3);
      if (MODE == kDense && p.out_fp16)
        static_cast<__half*>(p.out)[o] = __float2half_rn(v);
      else
        static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
    }
  }
}

int64_t steps_of(int K) { return (K + kStep - 1) / kStep; }
int64_t round256(int64_t b) { return (b + 255) & ~int64_t(255); }
int64_t self_bytes(int64_t rows, int K, bool two) { return rows * steps_of(K) * ((two ? 2 : 1) * kUnitBytes + 4); }

// What this file takes; few_stream.cu takes the rest.  Every block converts
// all activations that it needs, so the work grows with them twice: with the
// steps of a block and with the blocks.  Measured (us here, us there): one
// token x [512, 2048] 2.7, 6.5, x [8192, 4096] 8.5, 10.3, x [2048, 7168] 8.8,
// 8.0; three x [4096, 4096] 8.2, 7.8; eight x [2048, 2048] 5.6, 7.4, x [8192,
// 2048] 9.2, 8.0.  Experts (tokens, of them, H, I): 1, 2, 2048, 2048 15.4,
// 16.6; 1, 8, 1024, 1024 19.7, 15.6; 8, 4, 512, 256 12.4, 18.3; 4, 4, 1024,
// 512 15.9, 16.3.
constexpr int64_t kSelfBytes = 128 * 1024;      // of shared memory
constexpr int kSmallTokens = 8, kSmallK = 6144;
constexpr int64_t kValues = int64_t(1) << 14;   // activations that a block converts
bool takes_matvec(int T, int N, int K) {
  return T <= kSmallTokens && K <= kSmallK && int64_t(T) * K <= kValues && int64_t(T) * K * K * N <= int64_t(1) << 37;
}
bool takes_experts(int T, int k, int H, int I) {
  if (T > kSmallTokens || T * k > kMaxRows || H > kSmallK || int64_t(T) * H > kValues ||
      self_bytes(int64_t(T) * k, I, true) > kSelfBytes)
    return false;
  const int64_t h = int64_t(T) * k * I, work = h * 2 * H;
  return work <= int64_t(1) << 24 && h * work <= int64_t(1) << 36;
}

template <bool MX, int SRC, int MODE>
cudaError_t launch_few(const FewParams& p, int64_t rows, dim3 grid, cudaStream_t st) {
  auto kernel = few_kernel<MX, SRC, MODE>;
  size_t smem = size_t(self_bytes(rows, p.K, SRC == kF32));
  if (smem < size_t(kWarps) * 1024) smem = size_t(kWarps) * 1024;
  if (MODE == kGateUp && smem < size_t(p.E) * 8) smem = size_t(p.E) * 8;
  if (smem > 48 * 1024) {
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (err != cudaSuccess) return err;
  }
  return launch_kernel(kernel, grid, dim3(kThreads), smem, st, false, p);
}

void set_matrix(FewParams* p, const FewMatrix& w) {
  p->packed = w.packed;
  p->scales = w.scales;
  p->gscale = w.gscale;
  p->N = w.N;
  p->K = w.K;
  p->tiled = w.tiled;
  p->wide = (reinterpret_cast<uintptr_t>(w.packed) & 31) == 0;
}

}  // namespace

size_t few_matvec_workspace_bytes(int T, int N, int K) { return takes_matvec(T, N, K) ? 0 : few_stream_matvec_bytes(T, N, K); }

size_t few_experts_workspace_bytes(int T, int k, int H, int I) {
  if (!takes_experts(T, k, H, I)) return few_stream_experts_bytes(T, k, H, I);
  return size_t(round256(sizeof(Plan)) + int64_t(T) * k * I * 4);
}

int few_experts_launches(int T, int k, int H, int I) { return takes_experts(T, k, H, I) ? 2 : 4; }

cudaError_t launch_few_matvec(const void* x, int64_t x_stride, int T, bool fp16, const FewMatrix& w, void* out, void* ws,
                              int num_sms, cudaStream_t st) {
  if (!takes_matvec(T, w.N, w.K)) return launch_stream_matvec(x, x_stride, T, fp16, w, out, ws, num_sms, st);
  FewParams p = {};
  p.x = x, p.x_stride = x_stride;
  p.T = T, p.k = 1, p.E = 1;
  set_matrix(&p, w);
  p.out_fp16 = fp16;
  p.out = out;
  const dim3 grid(unsigned(w.N / 32));
  if (w.mx) return fp16 ? launch_few<true, kFp16, kDense>(p, T, grid, st) : launch_few<true, kBf16, kDense>(p, T, grid, st);
  return fp16 ? launch_few<false, kFp16, kDense>(p, T, grid, st) : launch_few<false, kBf16, kDense>(p, T, grid, st);
}

cudaError_t launch_few_experts(const void* x, int64_t x_stride, const int32_t* idx, const float* topk_w, int T, int k,
                               int E, const FewMatrix& gu, const FewMatrix& d, void* out, void* ws, int num_sms,
                               cudaStream_t st) {
  if (!takes_experts(T, k, gu.K, d.K))
    return launch_stream_experts(x, x_stride, idx, topk_w, T, k, E, gu, d, out, ws, num_sms, st);
  FewParams p = {};
  p.plan = static_cast<Plan*>(ws);
  float* h = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + round256(sizeof(Plan)));
  p.x = x, p.x_stride = x_stride;
  p.T = T, p.k = k, p.E = E;
  p.idx = idx, p.topk_w = topk_w;
  set_matrix(&p, gu);
  p.next_gscale = d.gscale;
  p.out = h;
  dim3 grid(unsigned(d.K / 16), unsigned(T * k + 1));
  const cudaError_t err = gu.mx ? launch_few<true, kBf16, kGateUp>(p, T, grid, st) : launch_few<false, kBf16, kGateUp>(p, T, grid, st);
  if (err != cudaSuccess) return err;

  set_matrix(&p, d);
  p.gscale = p.next_gscale = nullptr;     // in h already
  p.x = h, p.x_stride = d.K;
  p.out = out;
  grid = dim3(unsigned(d.N / 32));
  return d.mx ? launch_few<true, kF32, kDown>(p, int64_t(T) * k, grid, st)
              : launch_few<false, kF32, kDown>(p, int64_t(T) * k, grid, st);
}

cudaError_t few_flags_address(unsigned** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_few_flags); }

}  // namespace nvfp4moe
