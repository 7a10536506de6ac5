// Absorbed latent attention over the paged cache (decode), on the
// 5th-generation tensor core.
//
// With q [rows, 576] the queries of one sequence (row = new token x head) and
// c [keys, 576] its cached rows,
//   S = q c^T * scale,  P = softmax(S),  out = P c[:, :512].
// One pass over the keys with a running maximum m and sum l per row:
//   p = exp2(S * scale * log2 e - m),  l = l * a + sum p,  O = O * a + p c,
// a = exp2(m_old - m_new).
//
// A CTA holds 64 rows: their accumulator (64 x 512 float32) is half of the
// SM's tensor memory, and a wider block would leave no room for S.  Keys come
// in tiles of 64; a tile is read once from the cache into shared memory (72
// KB, two tiles in flight) and serves both products:
//   S [64 rows x 64 keys]     = Q (64 x 576, K-major) x C^T (K-major)
//   O^T [512 x 64 rows] +=  C^T (512 x 64 keys, M-major) x P^T (K-major)
// O is kept transposed so that the cached values are the 128-row operand in
// four blocks and the rows the N side: few rows then cost little, and the 64
// rows run at the full rate that M = 64 would not reach.
//
// Work is a list of (sequence, row block) items, each of ceil(len / 64)
// tiles; every CTA takes an equal, contiguous range of the tile list, found
// from the lengths on the device.  An item cut by a range border leaves
// partial results (normalised float32 rows and their log-sums) in the
// workspace, which a second kernel joins.
//
// Bound by the cache's bytes: a tile takes 2800 cycles in the middle of a range,
// the rate at which HBM feeds an SM (S takes 1400 of them, P V 650 to 1000, the
// softmax 1000).  Ten calls in a graph (a loop of calls takes 1 us more), 128
// sequences x 16 heads of 300 to 4100 keys (340 MB): 66 us, 5.1 TB/s; 32 x 64 heads of 1000 to 8191 (172 MB): 47.7 us, where a range is only
// 16 tiles and pays 5000 cycles to its first copy (lengths, pages), 4000 for its
// last tile, 5800 to store its rows, and the join 8 us.
//
// Warp roles: warps 0-7 softmax and epilogue, 8-11 TMA producers, warp 12
// tensor-memory owner and issuer of S, warp 13 issuer of P V.  Every wait is
// bounded.
#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstdint>

#include "../../include/nvfp4mla.h"
#include "internal.h"
#include "launch.cuh"
#include "mla_decode.cuh"
#include "mla_decode_pair.cuh"
#include "sm103_ptx.cuh"

namespace nvfp4moe {
namespace {

using namespace mla;

constexpr int kKeys = 64;                     // keys of a tile
constexpr int kChunk = 64 * 128;              // 64 rows x 64 values, 128-byte rows
constexpr int kTile = 9 * kChunk;
constexpr int kPieces = 4;                    // of a tile: 16 keys each, freed one by one
constexpr int kStages = 2;
constexpr int kProducer = 8, kIssuer = 12;    // first producer warp; the MMA warps, S and P V
constexpr int kThreads = 448;
constexpr int kSoftmaxThreads = 256;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;               // S buffers after the 4 x 64 columns of O^T

// Shared memory after the 1024-byte control block.
constexpr int kCtrl = 1024;
constexpr int kQOff = kCtrl;
constexpr int kKvOff = kQOff + kTile;
constexpr int kPOff = kKvOff + kStages * kTile;
constexpr int kSmem = kPOff + kChunk;

struct Control {
  uint64_t full[kStages], empty[kStages][kPieces];
  uint64_t q_full, q_empty, s_full[2], s_free[2], p_full, pv_done, o_free, drain;
  uint32_t tmem, pad;
  WaitCtl wait;
  float half[2][kRows];                       // per row: maxima, later sums, of the two halves of a tile's keys
  alignas(16) float col[kRows];               // per-row factors for the transposed accumulator
};
static_assert(sizeof(Control) <= kCtrl, "control block");
static_assert(kSmem <= 232448, "shared memory");

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kv_map,
                  const DecodeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Control* ctl = reinterpret_cast<Control*>(smem);
  volatile WaitCtl* wctl = &ctl->wait;
  const uint32_t base = ptx::smem_u32(smem);
  const int warp = __shfl_sync(kFull, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  auto bar = [&](const uint64_t& b) { return base + uint32_t(reinterpret_cast<const uint8_t*>(&b) - smem); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar(ctl->full[s]), kPieces);
      for (int i = 0; i < kPieces; ++i) ptx::mbar_init(bar(ctl->empty[s][i]), 1);
    }
    ptx::mbar_init(bar(ctl->q_full), 1);
    ptx::mbar_init(bar(ctl->q_empty), 1);
    ptx::mbar_init(bar(ctl->s_full[0]), 1);
    ptx::mbar_init(bar(ctl->s_full[1]), 1);
    ptx::mbar_init(bar(ctl->p_full), kSoftmaxThreads);
    ptx::mbar_init(bar(ctl->pv_done), 1);
    ptx::mbar_init(bar(ctl->o_free), kSoftmaxThreads);
    ptx::mbar_init(bar(ctl->s_free[0]), kSoftmaxThreads);
    ptx::mbar_init(bar(ctl->s_free[1]), kSoftmaxThreads);
    ptx::mbar_init(bar(ctl->drain), 2);
    ptx::fence_barrier_init();
    ctl->wait.abort = 0;
    ctl->wait.limit_us = p.wait_us;
    ctl->wait.flags = &g_decode_flags;
  }
  if (warp == kProducer && lane == 0) {
    ptx::prefetch_tmap(&q_map);
    ptx::prefetch_tmap(&kv_map);
  }
  if (warp == kIssuer) {
    ptx::tmem_alloc(base + uint32_t(offsetof(Control, tmem)), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  Cursor<kKeys> cur;                          // its loads run while tensor memory is allocated
  const int share = cur.init(p, blockIdx.x, gridDim.x);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, ctl->tmem, 0);

  if (warp >= kProducer && warp < kProducer + kPieces) {
    // ---- producers: one warp for each piece of 16 keys, so that a tile's
    // copies are issued in the time of two ----
    const int piece = warp - kProducer;
    if (piece == 0 && blockIdx.x == 0)        // lengths that are not served as they are
      for (int b = lane; b < p.B; b += 32)
        if (__ldg(p.lens + b) != seq_len(p, b)) atomicOr(&g_decode_flags, kFlagBadData);
    const uint32_t el = elect_one();
    const int oob = p.num_pages * p.page;
    uint32_t g = 0, seg = 0;
    // First cache row of the piece.
    auto look_up = [&](const Cursor<kKeys>& c) {
      const int row = c.tile * kKeys + 16 * piece;
      if (row >= c.len) return oob;
      const int id = __ldg(p.tables + c.b * p.table_stride + (row >> p.log_page));
      if (id >= 0 && id < p.num_pages) return id * p.page + (row & (p.page - 1));
      if (lane == 0) atomicOr(&g_decode_flags, kFlagBadData);  // zero rows instead of a page that does not exist
      return oob;
    };
    int mine = cur.valid() ? look_up(cur) : 0;
    while (cur.valid()) {
      if (piece == 0 && cur.is_first()) {
        if (!wait_warp(bar(ctl->q_empty), (seg & 1u) ^ 1u, wctl)) break;
        arrive_expect_tx(el, bar(ctl->q_full), kTile);
#pragma unroll
        for (int c = 0; c < 9; c += 3)
          tma_load_3d(el, base + kQOff + c * kChunk, &q_map, bar(ctl->q_full), 0, cur.b * p.rows + cur.block * kRows, c);
        ++seg;
      }
      const uint32_t s = g & 1u, fb = bar(ctl->full[s]);
      const uint32_t dst = base + kKvOff + s * kTile + 2 * piece * kGroup;
      const int groups = min(2, max(0, (cur.keys() - 16 * piece + 7) / 8));
      if (!wait_warp(bar(ctl->empty[s][piece]), ((g >> 1) & 1u) ^ 1u, wctl)) break;
      arrive_expect_tx(el, fb, uint32_t(groups * kGroup));
      if (groups > 0) tma_load_3d(el, dst, &kv_map, fb, 0, mine, 0);
      if (groups > 1) tma_load_3d(el, dst + kGroup, &kv_map, fb, 0, min(mine, oob - 8) + 8, 0);
      ++g;
      cur.next(p);
      if (cur.valid()) {
        // Shared memory holds two tiles, too few to cover the latency of HBM:
        // the next piece is requested into L2 while its buffer is still in
        // use.  One tile ahead measured best (three ahead: 6 % slower).
        mine = look_up(cur);
        const int rows = min(16, cur.len - cur.tile * kKeys - 16 * piece);
        if (rows > 0 && mine != oob)
          prefetch_l2(el, p.cache + int64_t(mine) * (2 * kRow), uint32_t(rows) * (2 * kRow));
      }
    }
    // Every copy that this warp issued has landed before the CTA leaves: the
    // barrier's phase also needs the other pieces, which after an abort may
    // not come, so the wait is bounded.
    if (seg) drain_phase(bar(ctl->q_full), (seg - 1) & 1u);
    for (uint32_t s = 0; s < kStages; ++s) {
      const uint32_t n = (g + 1 - s) / 2;     // uses of the stage
      if (n) drain_phase(bar(ctl->full[s]), (n - 1) & 1u);
    }
    __syncwarp();
  } else if (warp >= kIssuer) {
    // ---- MMA issuers: one warp for S, one for P V.  A single one that took
    // what was ready put an S in front of the P V that frees a buffer in most
    // rounds (3500 cycles a tile). ----
    const uint32_t el = elect_one();
    const int n = uniform(cur.end - cur.pos);
    uint32_t seg = 0;
    if (warp == kIssuer) {
      const uint32_t idesc = idesc_f16(Elem<T>::kFormat, 64, kKeys, false, false);
      const uint32_t a = desc_sw128(base + kQOff, 16);
      for (int g = 0; g < n; ++g) {
        const uint32_t s = g & 1u, ph = (g >> 1) & 1u, d = tmem + kSCol + s * kKeys;
        const bool first = uniform(cur.is_first()), last = uniform(cur.is_last());
        cur.next(p);
        if (first && !wait_warp(bar(ctl->q_full), seg++ & 1u, wctl)) break;
        if (!wait_warp(bar(ctl->s_free[s]), ph ^ 1u, wctl)) break;
        if (!wait_warp(bar(ctl->full[s]), ph, wctl)) break;
        ptx::tc_fence_after();
        const uint32_t b = desc_sw128(base + kKvOff + s * kTile, 16);
#pragma unroll
        for (int c = 0; c < 9; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16<1024, kGroup>(el, d, a + c * (kChunk >> 4) + 2 * k, b + c * (1024 >> 4) + 2 * k, idesc, c + k > 0);
        tc_commit(el, bar(ctl->s_full[s]));
        if (last) tc_commit(el, bar(ctl->q_empty));
      }
    } else {
      const uint32_t b = desc_sw128(base + kPOff, 16);
      for (int g = 0; g < n; ++g) {
        const uint32_t s = g & 1u;
        const bool first = uniform(cur.is_first());
        const uint32_t idesc = idesc_f16(Elem<T>::kFormat, 128, uniform((cur.rows(p) + 15) / 16 * 16), true, false);
        cur.next(p);
        if (!wait_warp(bar(ctl->p_full), g & 1u, wctl)) break;
        // the previous segment's accumulator has been read
        if (first && seg++ && !wait_warp(bar(ctl->o_free), seg & 1u, wctl)) break;
        ptx::tc_fence_after();
        const uint32_t more = first ? 0u : 1u;
        const uint32_t a = desc_sw128(base + kKvOff + s * kTile, 1024);
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {   // 16 keys: two groups of C, 32 bytes of P
#pragma unroll
          for (int m = 0; m < 4; ++m)         // 128 values: two chunks
            mma_f16<kGroup, 1024>(el, tmem + m * kRows, a + k * (2 * kGroup >> 4) + m * (2 * 1024 >> 4), b + 2 * k, idesc,
                    k ? 1u : more);
          tc_commit(el, bar(ctl->empty[s][k]));
        }
        tc_commit(el, bar(ctl->pv_done));
      }
    }
    tc_commit(el, bar(ctl->drain));
    drain_phase(bar(ctl->drain), 0);
    __syncwarp();
  } else {
    // ---- softmax and epilogue ----
    if (threadIdx.x == 0) {
      Head h;
      h.share = share;
      h.start = cur.valid() ? cur.pos - cur.tile : 0;
      h.tiles = cur.valid() ? cur.tiles : 0;
      h.b = cur.valid() ? cur.b : 0;
      h.block = cur.valid() ? cur.block : 0;
      p.heads[blockIdx.x] = h;
    }
    // Two warps share a quarter of the lanes: each takes half of a tile's keys
    // in the softmax and half of the accumulator's values.
    const int half = warp >> 2, lanes = 32 * (warp & 3);
    const uint32_t quarter = uint32_t(lanes) << 16;
    const int r0 = lanes / 2 + (lane >> 2);         // this thread's rows: r0 and r0 + 8
    float m[2], l[2];                               // running maximum (log2 domain) less kLift, and half's sum
    uint32_t g = 0;
    // A failed wait is remembered and ends the loop for all warps at the
    // next tile's vote, so that no thread leaves others at a barrier.
    bool dead = false;
    auto wait = [&](uint32_t b, uint32_t parity) {
      dead |= !wait_phase(b, parity, wctl);
      __syncwarp();
    };
    int behind[2] = {0, 0};                         // keys of the sequence that come after the rows' tokens
    while (cur.valid()) {
      if (cur.is_first()) {
#pragma unroll
        for (int i = 0; i < 2; ++i) behind[i] = p.Sq - 1 - (cur.block * kRows + r0 + 8 * i) / p.H;
      }
      const bool first = cur.is_first(), last = cur.is_last();
      const int keys = cur.keys(), rows = cur.rows(p);
      wait(bar(ctl->s_full[g & 1u]), (g >> 1) & 1u);
      ptx::tc_fence_after();
      uint32_t sr[16];
      tmem_ld_16x256b_x4(tmem + quarter + kSCol + (g & 1u) * kKeys + 32 * half, sr);
      ptx::tmem_ld_wait();
      ptx::tc_fence_before();
      ptx::mbar_arrive(bar(ctl->s_free[g & 1u]));
      // keys of this half that row r0 + 8 i sees: query token s of Sq sees len - Sq + s + 1
      int sees[2];
      bool masked = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + 8 * i;
        sees[i] = r < rows ? cur.len - behind[i] - cur.tile * kKeys - 32 * half : 0;
        masked |= sees[i] < 32;
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (8 * (i >> 2) + 2 * (lane & 3) + (i & 1) >= sees[(i >> 1) & 1]) sr[i] = 0xFF800000u;
      }
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 16; ++i) top[(i >> 1) & 1] = fmaxf(top[(i >> 1) & 1], __uint_as_float(sr[i]));
      bool grew = first;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(kFull, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(kFull, top[i], 2));
        top[i] *= p.scale_log2;
        if (first) m[i] = -INFINITY, l[i] = 0.0f;
        grew |= top[i] - m[i] > kGrow + Elem<T>::kLift;  // also from -inf
        if ((lane & 3) == 0) ctl->half[half][r0 + 8 * i] = top[i];
      }
      // The reference maximum moves only when some row's maximum grew by 2^8:
      // until then weights of up to 2^8 are as exact as weights of up to 1.
      if (bar_any(1, kSoftmaxThreads, grew || dead)) {
        if (bar_any(2, kSoftmaxThreads, dead)) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mn = fmaxf(m[i], fmaxf(top[i], ctl->half[half ^ 1][r0 + 8 * i]) - Elem<T>::kLift);
          const float a = mn == m[i] ? 1.0f : exp2_approx(m[i] - mn);
          m[i] = mn;
          l[i] *= a;
          if (half == 0 && (lane & 3) == 0) ctl->col[r0 + 8 * i] = a;
        }
        bar_sync(2, kSoftmaxThreads);
        if (!first) {
          wait(bar(ctl->pv_done), (g - 1) & 1u);
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 2 * half * kRows; c < 2 * (half + 1) * kRows; c += 32) {
            if ((c & (kRows - 1)) >= rows) continue;
            uint32_t o[32];
            ptx::tmem_ld_32x32b_x32(tmem + quarter + c, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * ctl->col[(c & (kRows - 1)) + i]);
            ptx::tmem_st_32x32b_x32(tmem + quarter + c, o);
          }
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
        }
      }
      // the weights, rounded to 16 bits for the second product; their sum stays float32
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int k = (i >> 1) & 1;
        const float e = exp2_approx(fmaf(__uint_as_float(sr[i]), p.scale_log2, m[k] == -INFINITY ? 0.0f : -m[k]));
        l[k] += e;
        sr[i] = __float_as_uint(e);
      }
      if (g) wait(bar(ctl->pv_done), (g - 1) & 1u);  // P is free
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const int r = r0 + 8 * ((i >> 1) & 1);
        sts32(base + kPOff + r * 128 + ((((i >> 2) + 4 * half) ^ (r & 7)) << 4) + (lane & 3) * 4,
              Elem<T>::pack(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])));
      }
      // Rows of the tile past the last key may hold anything, and 0 * NaN is
      // NaN: they are zeroed before the second product reads them as values.
      if (keys < kKeys) {
        const int from = max(keys, 0);
        const uint32_t kv = base + kKvOff + (g & 1u) * kTile;
        for (int i = threadIdx.x; i < (kKeys - from) * 64; i += kSoftmaxThreads) {
          const int k = from + (i >> 6);      // 64 pieces of 16 bytes a key: eight in each of eight chunks
          ptx::sts128(kv + (k >> 3) * kGroup + ((i >> 3) & 7) * 1024 + (k & 7) * 128 + (i & 7) * 16, 0, 0, 0, 0);
        }
      }
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      ptx::mbar_arrive(bar(ctl->p_full));
      if (last) {
        const bool whole = cur.first == 0 && cur.tile + 1 == cur.tiles;
        const int64_t part = 2 * blockIdx.x + (cur.pos - cur.tile + cur.first == int(share * blockIdx.x) ? 0 : 1);
        const int64_t row0 = whole ? int64_t(cur.b) * p.rows + cur.block * kRows : part * kRows;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[i] += __shfl_xor_sync(kFull, l[i], 1);
          l[i] += __shfl_xor_sync(kFull, l[i], 2);
          if ((lane & 3) == 0) ctl->half[half][r0 + 8 * i] = l[i];
        }
        bar_sync(2, kSoftmaxThreads);
        bool empty = false;                   // some row saw no key
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = r0 + 8 * i;
          const float sum = l[i] + ctl->half[half ^ 1][r];
          empty |= sum == 0.0f;
          if (half == 0 && (lane & 3) == 0) {
            ctl->col[r] = sum == 0.0f ? 0.0f : 1.0f / sum;
            const float e = sum == 0.0f ? -INFINITY : m[i] + log2f(sum);
            if (r < rows) (whole ? p.lse : p.part_lse)[row0 + r] = whole ? e * kLn2 : e;
          }
        }
        empty = bar_any(2, kSoftmaxThreads, empty);
        wait(bar(ctl->pv_done), g & 1u);
        ptx::tc_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < rows; c0 += 32) {
          float f[32];                        // the factors of 32 rows, for both blocks of values
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(f + i) = *reinterpret_cast<const float4*>(ctl->col + c0 + i);
#pragma unroll 1
          for (int v = 0; v < 2; ++v) {
            uint32_t o[32];
            ptx::tmem_ld_32x32b_x32(tmem + quarter + (2 * half + v) * kRows + c0, o);
            ptx::tmem_ld_wait();
            const int dim = (2 * half + v) * 128 + lanes + lane, n = min(32, rows - c0);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f[i]);
            if (empty) {                      // zeros, also where masked values were not finite
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (f[i] == 0.0f) o[i] = 0u;
            }
            if (whole) {
              T* out = reinterpret_cast<T*>(p.out) + (row0 + c0) * kLatent + dim;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i < n) out[i * kLatent] = Elem<T>::from(__uint_as_float(o[i]));
            } else {
              float* out = p.part_o + (row0 + c0) * kLatent + dim;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i < n) out[i * kLatent] = __uint_as_float(o[i]);
            }
          }
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(ctl->o_free));
      }
      cur.next(p);
      ++g;
    }
  }

  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kIssuer) ptx::tmem_dealloc(tmem, kTmemCols);
}

// Joins the partial results of the items that a range border cut.  With e_i
// the log2-sum of piece i and o_i its normalised rows, out = sum 2^(e_i - e)
// o_i, e = log2 sum 2^e_i, the pieces always in the same order.
// SHARE warps share the pieces of a row.  With one, a warp takes a whole row
// and block (c, .) serves the item that the border between ranges c and c + 1
// is the first to cut.  With more (few items of many pieces), block (item, .)
// serves an item; eight take 128 of a row's values, one block for each.
constexpr int kJoinThreads = 256;
template <typename T, int SHARE>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const DecodeParams p) {
  constexpr bool kByItem = SHARE > 1;
  constexpr int kWarps = kJoinThreads / 32, kParts = SHARE == 8 ? 4 : 1, kVecs = 4 / kParts;
  __shared__ float4 s_sum[kByItem ? kWarps : 1][kVecs][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, set = warp % SHARE;
  int start, tiles, share, b, block;
  // The lengths are older than the kernel before this one, which waited for
  // them before it let this one begin: they need no wait here.
  if (kByItem) find_item<kKeys>(p, blockIdx.x, b, block, start, tiles, share);
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  if (!kByItem) {
    const Head h = p.heads[blockIdx.x + 1];
    start = h.start, tiles = h.tiles, share = h.share, b = h.b, block = h.block;
    if (!border_joins(int(blockIdx.x), start, tiles, share)) return;
  }
  const int first = start / share, last = (start + tiles - 1) / share;
  if (first == last) return;                  // whole: written by its CTA
  const int pieces = last - first + 1;
  const int row = int(blockIdx.y) / kParts * (kWarps / SHARE) + warp / SHARE, part = int(blockIdx.y) % kParts;
  const bool live = row < min(kRows, p.rows - block * kRows);
  // piece 0 is the last segment of range `first` unless the range begins with it
  const int lead = start != first * share ? 1 : 0;
  auto piece_row = [&](int i) {
    return int64_t(2 * (first + i) + (i == 0 ? lead : 0)) * kRows + row;
  };
  constexpr int kPer = (kMlaDecodeMaxGrid + 31) / 32;
  float w[kPer];                              // the weights of pieces lane, lane + 32, ...
  float top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    w[k] = live && lane + 32 * k < pieces ? p.part_lse[piece_row(lane + 32 * k)] : -INFINITY;
    top = fmaxf(top, w[k]);
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
  const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
  for (int k = 0; k < kPer; ++k) sum += w[k] = exp2_approx(w[k] - ref);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  float4 acc[kVecs] = {};                     // values 128 (part * kVecs + j) + 4 lane ..
  if (live) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int n = min(32, pieces - 32 * k);
#pragma unroll 4 / kVecs * 2
      for (int i = set; i < n; i += SHARE) {
        const float* at = p.part_o + piece_row(32 * k + i) * kLatent + 128 * kVecs * part + 4 * lane;
        const float a = __shfl_sync(kFull, w[k], i) * inv;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          const float4 o = *reinterpret_cast<const float4*>(at + 128 * j);
          acc[j].x += a * o.x, acc[j].y += a * o.y, acc[j].z += a * o.z, acc[j].w += a * o.w;
        }
      }
    }
  }
  const int64_t at = int64_t(b) * p.rows + block * kRows + row;
  auto store = [&](int j, float4 v) {
    *reinterpret_cast<uint2*>(p.out + 2 * (at * kLatent + 128 * (part * kVecs + j) + 4 * lane)) =
        make_uint2(Elem<T>::pack(v.x, v.y), Elem<T>::pack(v.z, v.w));
  };
  if (live && lane == 0 && set == 0 && part == 0) p.lse[at] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * kLn2;
  if (kByItem) {                              // warp j of a row adds up the j-th of its vectors
#pragma unroll
    for (int j = 0; j < kVecs; ++j) s_sum[warp][j][lane] = acc[j];
    __syncthreads();
    if (set >= kVecs) return;
    float4 v = s_sum[warp - set][set][lane];
#pragma unroll
    for (int i = 1; i < SHARE; ++i) {
      const float4 o = s_sum[warp - set + i][set][lane];
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    if (live) store(set, v);
  } else if (live) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) store(j, acc[j]);
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of a range at least, of 64 keys with one CTA and of 128 with a pair:
// below this, splitting a sequence costs more than it gains.  A sequence of
// 1024 keys with 16 heads takes 10.5 us (9.6 with 1, 12.6 with 4), of 4096 keys
// 11.4 (12.1 with 1, 13.2 with 4); with 128 heads 14.5 (15.0 and 16.5), of 8192
// keys 15.7 (18.7 and 16.7); eight of 1024 keys with 16 heads 10.9 (11.9 and 13.2).
constexpr int kMinShare = 2;

// Most tiles the call can have.
int64_t most_tiles(const MlaDecodeArgs& a, int ctas, int keys) {
  const int64_t longest = std::max<int64_t>(1, ceil_div(int64_t(a.max_pages) * a.page, keys));
  return int64_t(a.B) * ceil_div(int64_t(a.Sq) * a.H, kRows * ctas) * longest;
}

// CTA pairs that can be resident at once, per device, looked up once.
template <typename K>
int max_pairs(K kernel) {
  static std::atomic<int> cached[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if ((n = cached[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pair::kSmem) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(pair::kThreads);
  cfg.dynamicSmemBytes = pair::kSmem;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <typename T>
int launch(const MlaDecodeArgs& a, int num_sms, cudaStream_t st) {
  if (most_tiles(a, 1, kKeys) >= (int64_t(1) << 31)) {
    set_error_detail("B = %d, Sq * H = %d and max_pages * page_size = %lld keys exceed 2^31 tiles of 64 rows x 64 keys",
                     a.B, a.Sq * a.H, (long long)a.max_pages * a.page);
    return NVFP4MOE_ERR_UNSUPPORTED;
  }
  const int rows = a.Sq * a.H;
  // A pair of CTAs shares each tile between 128 rows, in the time that one CTA
  // needs for 64: from 65 rows on it halves the passes over the cache (sequences
  // of some 3500 keys, with pairs and with single CTAs: 32 x 66 heads 43.3 and 51.7
  // us, 32 x 96 43.7 and 52.9, 128 x 66 108 and 172, 128 x 128 113 and 178; 2 of
  // 28000 x 72 28.2 and 32.5).  With at most 64 rows half of its rows would be
  // padding, and single CTAs are faster (32 x 64 heads: 47.8 us, with pairs 50.8;
  // 128 x 16 heads 66 and 79).
  const bool pair = rows > kRows;
  CUtensorMap q_map, kv_map;
  if (!encode_rows<T>(&q_map, a.q, int64_t(a.B) * rows, kRows, 3) ||
      !encode_rows<T>(&kv_map, a.cache, int64_t(a.num_pages) * a.page, 8, pair ? 9 / pair::kParts : 9)) {
    set_error_detail("cuTensorMapEncodeTiled failed or is unavailable");
    return NVFP4MOE_ERR_CUDA;
  }
  const int ctas = pair ? 2 : 1;
  int most_ranges = std::min(num_sms, kMlaDecodeMaxGrid);
  if (pair) {
    most_ranges = std::min(max_pairs(decode_pair_kernel<T>), most_ranges / 2);
    if (most_ranges < 1) {
      set_error_detail("no CTA pair of the absorbed attention fits on this device");
      return NVFP4MOE_ERR_SMEM;
    }
  }
  const int ranges = int(std::min<int64_t>(most_ranges, ceil_div(most_tiles(a, ctas, pair ? pair::kKeys : kKeys), kMinShare)));
  DecodeParams p;
  p.tables = a.tables;
  p.table_stride = a.table_stride;
  p.lens = a.lens;
  p.B = a.B, p.Sq = a.Sq, p.H = a.H;
  p.rows = rows;
  p.ctas = ctas;
  p.blocks = int(ceil_div(rows, kRows * ctas));
  p.cache = static_cast<const uint8_t*>(a.cache);
  p.num_pages = a.num_pages;
  p.page = a.page;
  p.log_page = 0;
  while ((1 << p.log_page) < a.page) ++p.log_page;
  p.max_pages = a.max_pages;
  p.scale_log2 = a.scale * kLog2e;
  p.out = static_cast<uint8_t*>(a.out);
  p.lse = a.lse;
  p.ranges = ranges;
  p.min_share = kMinShare;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.heads = reinterpret_cast<Head*>(ws);
  p.part_lse = reinterpret_cast<float*>(ws + kMlaDecodeHeadBytes);
  p.part_o = p.part_lse + int64_t(kMlaDecodeMaxGrid) * 2 * kRows;
  p.wait_us = wait_limit_us();
  static_assert(sizeof(Head) * kMlaDecodeMaxGrid <= kMlaDecodeHeadBytes, "workspace header");
  cudaError_t err;
  if (pair) {
    CUtensorMap v_map;
    if (!encode_values<T>(&v_map, a.cache, int64_t(a.num_pages) * a.page)) {
      set_error_detail("cuTensorMapEncodeTiled failed");
      return NVFP4MOE_ERR_CUDA;
    }
    err = cudaFuncSetAttribute(decode_pair_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, pair::kSmem);
    if (err == cudaSuccess)
      err = launch_kernel(decode_pair_kernel<T>, dim3(2 * ranges), dim3(pair::kThreads), pair::kSmem, st, false, q_map,
                          kv_map, v_map, p);
  } else {
    err = cudaFuncSetAttribute(decode_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (err == cudaSuccess)
      err = launch_kernel(decode_kernel<T>, dim3(ranges), dim3(kThreads), kSmem, st, false, q_map, kv_map, p);
  }
  const int64_t items = int64_t(a.B) * p.blocks;
  if (err == cudaSuccess && ranges > 1) {
    // Few items of many pieces are joined by item, several warps a row; more items
    // by the borders that cut them, a warp a row.  Single CTAs (152 ranges), calls
    // in a graph, by item and by borders: 8 sequences of 8192 keys x 64 heads 25.6
    // and 29.1 us, 20 45.1 and 46.4, 36 of 4096 x 16 heads 36.3 and 37.2, 38 x 64
    // heads 45.9 and 44.7, 76 75.6 and 68.2: a quarter of the ranges.  Pairs (76
    // ranges), whose items have half as many pieces of twice the rows, x 128 heads:
    // 2 of 32768 keys 28.3 and 43.1, 5 of 16384 38.3 and 40.5, 6 43.4 and 42.9, 8
    // 50.2 and 48.0, 12 of 4096 36.7 and 29.2, 19 of 8192 63.7 and 49.9: a twelfth.
    const int most = std::min(kRows * ctas, rows);
    const bool by_item = items * (pair ? 12 : 4) <= ranges;
    // From 16 pieces on, and while the blocks are resident at once, eight warps
    // share a quarter of a row: one sequence of 32768 keys with 16 heads takes
    // 21.2 us, 33.8 with four warps a row, eight with 16 heads 46.9 and 48.7; but
    // eight with 64 heads (2048 blocks) 56.7 and 52.6, eight of 1024 keys (eight
    // pieces each) 11.8 and 10.6.
    const bool wide = items * 16 <= ranges && items * most * 4 <= num_sms * 8;
    const int across = by_item ? int(items) : ranges - 1;
    if (pair)  // a task is eight rows x 128 values
      err = launch_kernel(by_item ? join_pair_kernel<T, true> : join_pair_kernel<T, false>,
                          dim3(across, by_item ? (most + 7) / 8 * 4 : (most + 7) / 8), dim3(by_item ? 2 * kPairJoinThreads : kPairJoinThreads), 0, st, false, p);
    else if (wide)
      err = launch_kernel(join_kernel<T, 8>, dim3(across, most * 4), dim3(kJoinThreads), 0, st, false, p);
    else
      err = launch_kernel(by_item ? join_kernel<T, 4> : join_kernel<T, 1>,
                          dim3(across, by_item ? (most + 1) / 2 : (most + 7) / 8), dim3(kJoinThreads), 0, st, false, p);
  }
  if (err != cudaSuccess) {
    set_error_detail("mla_decode launch: %s", cudaGetErrorString(err));
    return NVFP4MOE_ERR_CUDA;
  }
  return NVFP4MOE_OK;
}

}  // namespace

size_t mla_decode_workspace_bytes() {
  return kMlaDecodeHeadBytes + size_t(kMlaDecodeMaxGrid) * 2 * kRows * (kLatent + 1) * sizeof(float);
}

int launch_mla_decode(const MlaDecodeArgs& a, int num_sms, cudaStream_t st) {
  return a.fp16 ? launch<__half>(a, num_sms, st) : launch<__nv_bfloat16>(a, num_sms, st);
}

cudaError_t mla_decode_flags_address(unsigned** at) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_decode_flags);
}

}  // namespace nvfp4moe
