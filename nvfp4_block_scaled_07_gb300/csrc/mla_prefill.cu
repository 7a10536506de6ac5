// Expanded latent attention over ragged batches (prefill), on the
// 5th-generation tensor core.
//
// For each head, with keys of 128 own values and 64 that all heads share:
//   S = (q_nope k_nope^T + q_rope k_rope^T) * scale,  P = softmax(S),  out = P v,
// one pass over the keys with a running maximum and sum per row, as in the
// absorbed kernel (p = exp2(S * scale * log2 e - m)).
//
// Bound by the tensor core: 2 * (192 + 128) operations a score.  One sequence
// of 16384 tokens x 16 heads takes 826 to 871 us as ten calls in a graph, 1.58 to
// 1.66 PFLOP/s, at about 1.55 GHz under the power limit, and 874 to 890 us in a
// loop of calls; a tile of keys with two tiles of rows takes 3400 cycles, of
// which the MMAs need 2700.  Short sequences pay for the ends of a block, 16000
// cycles (place 3000, first copies 2700, softmax and output of the last tile
// 8000, the next block's start 2000): seven of 101 to 2500 tokens take 133 us,
// 0.88 PFLOP/s.
//
// A CTA takes 256 queries of a head as two tiles of 128 rows, keys come in
// tiles of 128:
//   S_t [128 x 128] = Q_t (smem) x K^T (smem)         12 MMAs of 68 cycles
//   O_t [128 x 128] += P_t (tensor memory) x V (smem)  8 MMAs of 67 cycles
// Tensor memory holds S and O of both tiles (4 x 128 columns); P_t overwrites
// S_t, so S_t of the next keys follows P_t V.  The MMAs of one tile run under
// the softmax of the other:  P_a V, S_a', P_b V, S_b', ...  Each softmax
// thread owns a row, so that no statistics cross threads.
// Shared memory: Q 96 KB, two K tiles of 48 KB, one V tile of 32 KB whose
// halves are reloaded one by one.
//
// The parts of a key come from three tensors (k_nope and v usually slices of
// one projection's output), so nothing is concatenated in memory.
// Blocks are ordered by the keys that they see, most first, and by head among
// those: the hardware hands them out in this order, and short blocks fill the
// end (by head and sequence instead: 16384 tokens of one sequence 883 us
// instead of 834, seven ragged sequences 150 instead of 144).
//
// Warp roles: warps 0-3 and 4-7 softmax and epilogue of the two tiles, warp 8
// TMA producer, warp 9 tensor-memory owner and MMA issuer.  Every wait is
// bounded.
#include <climits>
#include <cstddef>
#include <cstdint>

#include "../../include/nvfp4mla.h"
#include "internal.h"
#include "launch.cuh"
#include "mla_common.cuh"
#include "sm103_ptx.cuh"

namespace nvfp4moe {
namespace {

using namespace mla;

__device__ unsigned g_prefill_flags = 0;

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kM = 128;                       // rows of a tile
constexpr int kKeys = 128;                    // keys of a tile
constexpr int kChunk = 128 * 128;             // 128 rows x 64 values
constexpr int kNopeDim = 128, kValueDim = 128;
constexpr int kQTile = 3 * kChunk, kKTile = 3 * kChunk, kVTile = 2 * kChunk;
constexpr int kProducer = 8, kIssuer = 9;
constexpr int kThreads = 320;
constexpr int kStageRow = 2 * kValueDim + 16; // bytes of an output row on its way out; 16 more against bank conflicts
constexpr uint32_t kTmemCols = 512;
constexpr float kGrow = 8.0f;                 // rescale O only when a maximum grew by 2^8

constexpr int kCtrl = 1024;
constexpr int kQOff = kCtrl;
constexpr int kKOff = kQOff + 2 * kQTile;
constexpr int kVOff = kKOff + 2 * kKTile;
constexpr int kSmem = kVOff + kVTile;

struct Control {
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2];  // v: halves of 64 keys
  uint64_t s_full[2], p_half[2], p_full[2], pv_done[2], drain;       // per tile of rows
  uint32_t tmem, pad;
  WaitCtl wait;
};
static_assert(sizeof(Control) <= kCtrl && kSmem <= 232448, "shared memory");

struct PrefillParams {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, Tq, Tk, H, most;                     // most: upper bound of the blocks of a head
  int causal;
  float scale_log2;
  uint8_t* out;                               // [Tq, H, 128]
  float* lse;                                 // [Tq, H]
  uint32_t wait_us;
};

// A sequence's range in `cu`, kept inside [0, total].
__device__ __forceinline__ int2 range_of(const int32_t* cu, int b, int total) {
  const int from = min(max(__ldg(cu + b), 0), total), to = min(max(__ldg(cu + b + 1), from), total);
  return make_int2(from, to - from);
}

// Scores of columns from `sees` on become -inf.
__device__ __forceinline__ void mask_from(uint32_t (&s)[32], int sees) {
  const uint32_t seen = sees >= 32 ? 0xFFFFFFFFu : sees <= 0 ? 0u : (1u << sees) - 1u;
#pragma unroll
  for (int k = 0; k < 32; ++k)
    if (!(seen >> k & 1u)) s[k] = 0xFF800000u;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kn_map,
                   const __grid_constant__ CUtensorMap kr_map, const __grid_constant__ CUtensorMap v_map,
                   const PrefillParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Control* ctl = reinterpret_cast<Control*>(smem);
  volatile WaitCtl* wctl = &ctl->wait;
  const uint32_t base = ptx::smem_u32(smem);
  const int warp = __shfl_sync(kFull, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  auto bar = [&](const uint64_t& b) { return base + uint32_t(reinterpret_cast<const uint8_t*>(&b) - smem); };

  ptx::grid_dep_wait();
  // The block's place: head, sequence b, its 256 queries from q0 on (q0 < 0:
  // none, the grid is sized by what the lengths could need).  All warps find it.
  const int head = int(blockIdx.x) % p.H;
  int b = 0, at_q = 0, at_k = 0, nq = 0, nk = 0, q0 = -1;
  {
    // Level of a block: the keys that its last row sees, in units of 256.  The
    // blocks of a sequence have consecutive levels from `low` on (causal), or
    // all the same.
    struct Levels {
      int blocks, low;
    };
    auto levels = [&](int k) {
      Levels v = {0, 0};
      if (k < p.B) {
        const int2 rq = range_of(p.cu_q, k, p.Tq), rk = range_of(p.cu_k, k, p.Tk);
        v.blocks = (rq.y + 2 * kM - 1) / (2 * kM);
        v.low = p.causal ? (rk.y - rq.y + 4 * kM - 1) >> 8 : (rk.y + 2 * kM - 1) >> 8;
      }
      return v;
    };
    const Levels mine = levels(lane);         // of the first 32 sequences
    auto at_least = [&](const Levels& v, int level) {  // a sequence's blocks of this level or above
      if (p.causal) return min(max(v.low + v.blocks - level, 0), v.blocks);
      return v.low >= level ? v.blocks : 0;
    };
    auto count = [&](int level) {
      int n = at_least(mine, level);
      for (int k = 32 + lane; k < p.B; k += 32) n += at_least(levels(k), level);
      return int(__reduce_add_sync(kFull, unsigned(n)));
    };
    int lo = INT_MAX, hi = INT_MIN;
    for (int k = lane; k < p.B; k += 32) {
      const Levels v = k == lane ? mine : levels(k);
      if (v.blocks) lo = min(lo, v.low), hi = max(hi, v.low + (p.causal ? v.blocks - 1 : 0));
    }
    lo = __reduce_min_sync(kFull, lo), hi = __reduce_max_sync(kFull, hi);
    const int i = int(blockIdx.x) / p.H;      // the i-th block from the highest level down
    if (lo <= hi && i < count(lo)) {
      while (lo < hi) {                       // the highest level with more than i blocks at or above it
        const int mid = lo + (hi - lo + 1) / 2;
        if (count(mid) > i) lo = mid;
        else hi = mid - 1;
      }
      int left = i - count(lo + 1);           // among the blocks of this level, by sequence
      for (int b0 = 0; b0 < p.B && q0 < 0; b0 += 32) {
        const Levels v = b0 ? levels(b0 + lane) : mine;
        const int here = at_least(v, lo) - at_least(v, lo + 1);
        int upto = here;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int n = __shfl_up_sync(kFull, upto, d);
          if (lane >= d) upto += n;
        }
        const unsigned hit = __ballot_sync(kFull, upto > left);
        if (hit) {
          const int src = __ffs(hit) - 1;
          b = b0 + src;
          q0 = 2 * kM * (p.causal ? lo - __shfl_sync(kFull, v.low, src) : left - __shfl_sync(kFull, upto - here, src));
          const int2 rq = range_of(p.cu_q, b, p.Tq), rk = range_of(p.cu_k, b, p.Tk);
          at_q = rq.x, nq = rq.y, at_k = rk.x, nk = rk.y;
        }
        left -= __shfl_sync(kFull, upto, 31);
      }
    }
  }
  if (blockIdx.x == 0 && warp == kProducer)   // offsets that are not served as they are
    for (int k = lane; k < p.B; k += 32)
      if (range_of(p.cu_q, k, p.Tq).x != __ldg(p.cu_q + k) || __ldg(p.cu_q + k + 1) < __ldg(p.cu_q + k) ||
          range_of(p.cu_k, k, p.Tk).x != __ldg(p.cu_k + k) || __ldg(p.cu_k + k + 1) < __ldg(p.cu_k + k) ||
          __ldg(p.cu_q + k + 1) > p.Tq || __ldg(p.cu_k + k + 1) > p.Tk)
        atomicOr(&g_prefill_flags, kFlagBadData);
  if (q0 < 0) return;

  // Row r of tile t is query q0 + 128 t + r; it sees keys 0 .. shift + its index.
  const int shift = p.causal ? nk - nq : nk;
  int n[2];                                   // key tiles that tile t takes part in
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(nq, q0 + (t + 1) * kM) - 1;  // last row's index
    const int sees = last < q0 + t * kM ? 0 : min(nk, p.causal ? shift + last + 1 : nk);
    n[t] = sees > 0 ? (sees + kKeys - 1) / kKeys : 0;
  }
  const int tiles = max(n[0], n[1]);

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(bar(ctl->q_full[t]), 1);
      ptx::mbar_init(bar(ctl->k_full[t]), 1);
      ptx::mbar_init(bar(ctl->k_empty[t]), 1);
      ptx::mbar_init(bar(ctl->v_full[t]), 1);
      ptx::mbar_init(bar(ctl->v_empty[t]), 1);
      ptx::mbar_init(bar(ctl->s_full[t]), 1);
      ptx::mbar_init(bar(ctl->p_half[t]), 128);
      ptx::mbar_init(bar(ctl->p_full[t]), 128);
      ptx::mbar_init(bar(ctl->pv_done[t]), 1);
    }
    ptx::mbar_init(bar(ctl->drain), 1);
    ptx::fence_barrier_init();
    ctl->wait.abort = 0;
    ctl->wait.limit_us = p.wait_us;
    ctl->wait.flags = &g_prefill_flags;
  }
  if (warp == kProducer && lane == 0) {
    ptx::prefetch_tmap(&q_map);
    ptx::prefetch_tmap(&kn_map);
    ptx::prefetch_tmap(&kr_map);
    ptx::prefetch_tmap(&v_map);
  }
  if (warp == kIssuer) {
    ptx::tmem_alloc(base + uint32_t(offsetof(Control, tmem)), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, ctl->tmem, 0);
  ptx::grid_dep_launch();

  if (warp == kProducer) {
    // ---- producer ----
    const uint32_t el = elect_one();
    uint32_t done_k = 0, done_v = 0;          // K tiles and V halves begun
    if (tiles) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (n[t] == 0) continue;
        arrive_expect_tx(el, bar(ctl->q_full[t]), kQTile);
#pragma unroll
        for (int c = 0; c < 3; ++c)
          tma_load_3d(el, base + kQOff + t * kQTile + c * kChunk, &q_map, bar(ctl->q_full[t]), 64 * c, head,
                      at_q + q0 + t * kM);
      }
    }
    for (int j = 0; j < tiles; ++j) {
      const uint32_t s = j & 1;
      const int row = at_k + j * kKeys;
      if (!wait_warp(bar(ctl->k_empty[s]), ((j >> 1) & 1u) ^ 1u, wctl)) break;
      ++done_k;
      const uint32_t kb = bar(ctl->k_full[s]), kd = base + kKOff + s * kKTile;
      arrive_expect_tx(el, kb, kKTile);
      tma_load_3d(el, kd, &kn_map, kb, 0, head, row);
      tma_load_3d(el, kd + kChunk, &kn_map, kb, 64, head, row);
      tma_load_3d(el, kd + 2 * kChunk, &kr_map, kb, 0, 0, row);
      bool ok = true;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ok = ok && wait_warp(bar(ctl->v_empty[h]), (j & 1u) ^ 1u, wctl);
        if (!ok) break;
        ++done_v;
        const uint32_t vb = bar(ctl->v_full[h]), vd = base + kVOff + h * (kChunk / 2);
        arrive_expect_tx(el, vb, kVTile / 2);
        tma_load_3d(el, vd, &v_map, vb, 0, head, row + 64 * h);
        tma_load_3d(el, vd + kChunk, &v_map, vb, 64, head, row + 64 * h);
      }
      if (!ok) break;
    }
    // every copy that was issued has landed before the CTA leaves
#pragma unroll
    for (uint32_t t = 0; t < 2; ++t) {
      if (n[t]) drain_phase(bar(ctl->q_full[t]), 0);
      const uint32_t k = (done_k + 1 - t) / 2, v = (done_v + 1 - t) / 2;
      if (k) drain_phase(bar(ctl->k_full[t]), (k - 1) & 1u);
      if (v) drain_phase(bar(ctl->v_full[t]), (v - 1) & 1u);
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // ---- MMA issuer ----
    const uint32_t el = elect_one();
    const uint32_t idesc_s = idesc_f16(Elem<T>::kFormat, kM, kKeys, false, false);
    const uint32_t idesc_o = idesc_f16(Elem<T>::kFormat, kM, kValueDim, false, true);
    auto issue_s = [&](int t, int j) {
      const uint32_t a = desc_sw128(base + kQOff + t * kQTile, 16);
      const uint32_t k = desc_sw128(base + kKOff + (j & 1) * kKTile, 16);
#pragma unroll
      for (int c = 0; c < 3; ++c)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_f16<1024, 1024>(el, tmem + t * kKeys, a + c * (kChunk >> 4) + 2 * s, k + c * (kChunk >> 4) + 2 * s, idesc_s, c + s > 0);
      tc_commit(el, bar(ctl->s_full[t]));
    };
    // V is stored with its values contiguous: 16 keys are 2048 bytes, the second 64 values a chunk further.
    // The first 64 keys go out as soon as their weights are there.
    auto issue_pv = [&](int t, int j, bool last_user) {
      const uint32_t v = desc_sw128(base + kVOff, kChunk);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!wait_warp(bar(ctl->v_full[h]), j & 1u, wctl) ||
            !wait_warp(bar(h ? ctl->p_full[t] : ctl->p_half[t]), j & 1u, wctl))
          return false;
        ptx::tc_fence_after();
#pragma unroll
        for (int s = 4 * h; s < 4 * h + 4; ++s)
          mma_f16_ts<1024>(el, tmem + 256 + t * kValueDim, tmem + t * kKeys + 8 * s, v + s * (2048 >> 4), idesc_o,
                     s ? 1u : uint32_t(j > 0));
        if (last_user) tc_commit(el, bar(ctl->v_empty[h]));
      }
      tc_commit(el, bar(ctl->pv_done[t]));
      return true;
    };
    bool ok = true;
    for (int j = -1; ok && j < tiles; ++j) {
      // P V of keys j, then S of keys j + 1, first tile a, then tile b
#pragma unroll
      for (int t = 0; t < 2 && ok; ++t) {
        if (j >= 0 && j < n[t]) {
          ok = issue_pv(t, j, t == 1 || j >= n[1]);
          if (!ok) break;
        }
        if (j + 1 < n[t]) {
          if (j < 0) ok = wait_warp(bar(ctl->q_full[t]), 0, wctl);
          ok = ok && wait_warp(bar(ctl->k_full[(j + 1) & 1]), ((j + 1) >> 1) & 1u, wctl);
          if (!ok) break;
          ptx::tc_fence_after();
          issue_s(t, j + 1);
          if (t == 1 || j + 1 >= n[1]) tc_commit(el, bar(ctl->k_empty[(j + 1) & 1]));
        }
      }
    }
    tc_commit(el, bar(ctl->drain));
    drain_phase(bar(ctl->drain), 0);
    __syncwarp();
  } else {
    // ---- softmax and epilogue: thread = row ----
    const int t = warp >> 2, quarter = warp & 3;
    const int r = 32 * quarter + lane, index = q0 + t * kM + r;  // the row, its query's index
    const uint32_t lanes = uint32_t(32 * quarter) << 16;
    const uint32_t s_col = tmem + lanes + t * kKeys, o_col = tmem + lanes + 256 + t * kValueDim;
    const int limit = index < nq ? min(nk, p.causal ? shift + index + 1 : nk) : 0;
    float m = -INFINITY, l = 0.0f;            // running maximum (log2 domain) less kLift, and sum
    bool ok = true;                           // the same for all lanes of a warp
    for (int j = 0; j < n[t]; ++j) {
      ok = __all_sync(kFull, wait_phase(bar(ctl->s_full[t]), j & 1u, wctl));
      if (!ok) break;
      ptx::tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) ptx::tmem_ld_32x32b_x32(s_col + 32 * c, s[c]);
      ptx::tmem_ld_wait();
      const int sees = limit - j * kKeys;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (__any_sync(kFull, sees < 32 * c + 32)) mask_from(s[c], sees - 32 * c);
      float top[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {           // four chains of three-way maxima
        top[c] = __uint_as_float(s[c][0]);
#pragma unroll
        for (int k = 1; k < 31; k += 2)
          top[c] = fmaxf(fmaxf(top[c], __uint_as_float(s[c][k])), __uint_as_float(s[c][k + 1]));
        top[c] = fmaxf(top[c], __uint_as_float(s[c][31]));
      }
      const float mn = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2 - Elem<T>::kLift);
      // The reference maximum moves only when it grew by 2^8 in some row of
      // the warp: until then weights of up to 2^8 are as exact as of up to 1.
      if (__any_sync(kFull, j == 0 || mn - m > kGrow)) {
        const float a = mn == m ? 1.0f : exp2_approx(m - mn);
        m = mn;
        l *= a;
        if (j) {
          ok = __all_sync(kFull, wait_phase(bar(ctl->pv_done[t]), (j - 1) & 1u, wctl));
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kValueDim; c += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(o_col + c, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
            ptx::tmem_st_32x32b_x16(o_col + c, o);
          }
        }
      }
      // Rows of V past the last key belong to another sequence or lie beyond
      // the tensor, and 0 * NaN is NaN: they are zeroed before P V reads them.
      const int keys = nk - j * kKeys;
      if (keys < kKeys) {
        ok = __all_sync(kFull, wait_phase(bar(ctl->v_full[0]), j & 1u, wctl) &&
                                   wait_phase(bar(ctl->v_full[1]), j & 1u, wctl));
        if (!ok) break;
        for (int k = int(threadIdx.x & 127); k < (kKeys - keys) * 16; k += 128)
          ptx::sts128(base + kVOff + (k & 1) * kChunk + (keys + (k >> 4)) * 128 + ((k >> 1) & 7) * 16, 0, 0, 0, 0);
        ptx::fence_proxy_async_smem();
      }
      // the weights, rounded to 16 bits for the second product; their sum stays float32
      float neg = m == -INFINITY ? 0.0f : -m;
      float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
        weights<T>(s[c], w, p.scale_log2, neg, sum0, sum1);
        ptx::tmem_st_32x32b_x16(s_col + 16 * c, w);
        if (c & 1) {                          // 64 keys are complete
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          ptx::mbar_arrive(bar(c == 1 ? ctl->p_half[t] : ctl->p_full[t]));
          asm volatile("" : "+f"(neg)::"memory");  // the other half's weights stay behind the arrival
        }
      }
      l += sum0 + sum1;
    }
    if (n[t] && ok) ok = __all_sync(kFull, wait_phase(bar(ctl->pv_done[t]), (n[t] - 1) & 1u, wctl));
    ptx::tc_fence_after();
    if (ok) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      // Rows go through the tile's Q, which no product reads any more, so that
      // a store covers two whole rows and not 16 bytes of 32 (this part of a
      // block 4500 -> 2600 cycles, a ragged batch 136.6 -> 133.1 us).
      uint8_t* stage = smem + kQOff + t * kQTile + 32 * quarter * kStageRow;
      // a row that saw no key gets zeros, also where masked values were not finite
      const bool zero = __any_sync(kFull, l == 0.0f);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (n[t]) {
          ptx::tmem_ld_32x32b_x32(o_col + 32 * c, o);
          ptx::tmem_ld_wait();
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * inv);
        if (zero)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (l == 0.0f) o[k] = 0u;
#pragma unroll
        for (int k = 0; k < 32; k += 8)
          *reinterpret_cast<uint4*>(stage + lane * kStageRow + 64 * c + 2 * k) =
              make_uint4(Elem<T>::pack(__uint_as_float(o[k]), __uint_as_float(o[k + 1])),
                         Elem<T>::pack(__uint_as_float(o[k + 2]), __uint_as_float(o[k + 3])),
                         Elem<T>::pack(__uint_as_float(o[k + 4]), __uint_as_float(o[k + 5])),
                         Elem<T>::pack(__uint_as_float(o[k + 6]), __uint_as_float(o[k + 7])));
      }
      __syncwarp();
      const int first = q0 + t * kM + 32 * quarter;  // the warp's first row
      uint8_t* out = p.out + 2 * (((int64_t(at_q) + first) * p.H + head) * kValueDim) + 16 * (lane & 15);
#pragma unroll
      for (int k = lane >> 4; k < 32; k += 2) {
        const uint4 v = *reinterpret_cast<const uint4*>(stage + k * kStageRow + 16 * (lane & 15));
        if (first + k < nq) *reinterpret_cast<uint4*>(out + int64_t(k) * p.H * (2 * kValueDim)) = v;
      }
      if (index < nq) p.lse[(int64_t(at_q) + index) * p.H + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kIssuer) ptx::tmem_dealloc(tmem, kTmemCols);
}

// 16-bit [tokens, heads, values] with strides in elements, in boxes of 64 values x 1 head x `rows` tokens.
template <typename T>
bool encode_heads(CUtensorMap* m, const void* base, int64_t values, int64_t heads, int64_t tokens, int64_t head_stride,
                  int64_t token_stride, int rows) {
  const int64_t dims[3] = {values, heads, tokens}, strides[2] = {2 * head_stride, 2 * token_stride};
  const int box[3] = {64, 1, rows};
  return encode_map(m, Elem<T>::kMap, 3, base, dims, strides, box);
}

template <typename T>
int launch(const MlaPrefillArgs& a, cudaStream_t st) {
  CUtensorMap q, kn, kr, v;
  const int64_t tk = a.Tk ? a.Tk : 1;         // no keys: nothing is loaded through the maps
  if (!encode_heads<T>(&q, a.q, kNopeDim + kRope, a.H, a.Tq, a.q_head_stride, a.q_token_stride, kM) ||
      !encode_heads<T>(&kn, a.k_nope, kNopeDim, a.H, tk, a.kn_head_stride, a.kn_token_stride, kKeys) ||
      !encode_heads<T>(&kr, a.k_rope, kRope, 1, tk, kRope, a.kr_token_stride, kKeys) ||
      !encode_heads<T>(&v, a.v, kValueDim, a.H, tk, a.v_head_stride, a.v_token_stride, kKeys / 2)) {
    set_error_detail("cuTensorMapEncodeTiled failed or is unavailable (strides?)");
    return NVFP4MOE_ERR_CUDA;
  }
  PrefillParams p;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.B = a.B, p.Tq = a.Tq, p.Tk = a.Tk, p.H = a.H;
  p.most = a.Tq / (2 * kM) + a.B;             // each sequence leaves at most one block that is not full
  p.causal = a.causal;
  p.scale_log2 = a.scale * kLog2e;
  p.out = static_cast<uint8_t*>(a.out);
  p.lse = a.lse;
  p.wait_us = wait_limit_us();
  auto kernel = prefill_kernel<T>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (err == cudaSuccess)
    err = launch_kernel(kernel, dim3(unsigned(int64_t(p.most) * a.H)), dim3(kThreads), kSmem, st, false, q, kn, kr, v, p);
  if (err != cudaSuccess) {
    set_error_detail("mla_prefill launch: %s", cudaGetErrorString(err));
    return NVFP4MOE_ERR_CUDA;
  }
  return NVFP4MOE_OK;
}

}  // namespace

int launch_mla_prefill(const MlaPrefillArgs& a, cudaStream_t st) {
  return a.fp16 ? launch<__half>(a, st) : launch<__nv_bfloat16>(a, st);
}

cudaError_t mla_prefill_flags_address(unsigned** at) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_prefill_flags);
}

}  // namespace nvfp4moe
