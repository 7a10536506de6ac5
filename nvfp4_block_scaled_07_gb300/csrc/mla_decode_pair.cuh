// Absorbed latent attention on CTA pairs: 128 rows (new token x head) share
// one pass over the keys.
//
// The mathematics is that of the one-CTA kernel.  A pair issues cta_group::2
// MMAs of M = 128 rows, 64 in each CTA, so that O (64 x 512 float32 a CTA)
// leaves room for S, and each operand byte of the cache is staged by one CTA
// for both:
//   S [128 x 128 keys]    = Q x C^T     N = 128: each CTA stages 64 keys x 576
//   O [128 x 512] += P x C[:, :512]     N = 256, twice: each CTA stages 256 of
//                                       the values of all 128 keys
// 36 MMAs of 36 cycles and 16 of 68 a tile of 128 keys, 2360 cycles, against
// the 2820 in which HBM delivers it to a pair.  Measured: about 3400.  128
// sequences x 128 heads of 2048 to 8192 keys (803 MB) take 155 us, 5.2 TB/s, as ten
// calls in a graph, and 160 to 173 us in a loop of calls, where the power limit
// lowers the clock; the tensor pipe is active for 57 % of the time, DRAM for 71 %
// and shared memory's banks for 43 %: what bounds is the way of the rows through
// one buffer, MMAs of a part 430 cycles, its release 850, its copy 2000.  (Times
// below are of ten calls in a graph.)  Two stages of 64 keys
// fit as well, but read Q twice as often: 187 us where 128 keys took 182.
// A CTA's share of a tile is 72 KB for S and 64 KB for P V (its own keys'
// values twice, so that both CTAs use the same descriptors).  S frees its rows
// in three parts of 192 values, so that the next tile's are copied while it
// still reads the others and while softmax and P V of the tile run (whole rows:
// 168 us where parts took 159; nine parts, boxes of 1 KB: 339).
// All roles share the instruction cache: loops whose bodies are not unrolled
// gave another 4 us.
//
// Warp roles in each CTA: warps 0-7 softmax and epilogue of its 64 rows, 8-9
// TMA producers of whole rows, 10-13 of values, warp 14 tensor-memory owner
// and, in the even CTA, issuer of S, warp 15 issuer of P V there.
// The even CTA's barriers count both CTAs' copies of whole rows, the arrivals of
// both CTAs' row warps (with and without rows to copy) and of their softmax
// warps; commits arrive in both.  The copies of values count in their own
// CTA, whose softmax warps wait for them before they arrive: rows past the
// last key are zeroed after their copy.
#pragma once

#include "../../include/nvfp4mla.h"
#include "internal.h"
#include "mla_decode.cuh"

namespace nvfp4moe {
namespace {

namespace pair {
constexpr int kKeys = 128;                    // keys of a tile
constexpr int kPieces = 8;                    // of a tile: 16 keys each
constexpr int kParts = 3;                     // of a row: 192 values each
constexpr int kProducer = 8, kIssuer = 14;    // first producer warp; the MMA warps, S and P V
constexpr int kThreads = 512;
constexpr int kSoftmaxThreads = 256;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256, kSCols = 64;  // S buffers after the 256 columns of O
constexpr int kQBytes = 64 * 2 * kRow;
constexpr int kKBytes = 8 * kGroup;           // 64 keys
constexpr int kVGroup = 4 * 1024;             // 8 keys: four atoms (two of each half of the values)
constexpr int kVBytes = 16 * kVGroup;         // 128 keys
constexpr int kPBytes = 64 * 128;             // 64 rows x 64 keys
constexpr int kCtrl = 2048;
constexpr int kQOff = kCtrl;
constexpr int kKOff = kQOff + kQBytes;
constexpr int kVOff = kKOff + kKBytes;
constexpr int kPOff = kVOff + kVBytes;
constexpr int kSmem = kPOff + 2 * kPBytes;

struct Control {
  // counted in the even CTA only: k_full, q_full, s_free, p_full, o_free
  uint64_t k_full[kParts], v_full, k_empty[kParts], v_empty[kPieces];
  uint64_t q_full, q_empty, s_full[2], s_free[2], p_full, pv_done, o_free, drain;
  uint32_t tmem, pad;
  WaitCtl wait;
  float part[4][kRows];                       // per row: maxima, later sums, of the four quarters of a tile's keys
};
static_assert(sizeof(Control) <= kCtrl && kSmem <= 232448, "shared memory");
}  // namespace pair

// The values of the cached rows for P V: boxes of 8 rows x two chunks of 64
// values x both halves (values 0 .. 255 and 256 .. 511), which land as four
// atoms of 8 rows x 128 bytes, half by half.
template <typename T>
bool encode_values(CUtensorMap* m, const void* base, int64_t rows) {
  const int64_t dims[4] = {64, rows, 4, 2}, strides[3] = {2 * kRow, 128, 512};
  const int box[4] = {64, 8, 2, 2};
  return encode_map(m, Elem<T>::kMap, 4, base, dims, strides, box);
}

// Place of four values of a partial row (floats): row r of 64, values 256
// half + 128 upper + 4 q .. + 3.  32 rows' pieces of 16 bytes are contiguous.
__device__ __forceinline__ int part_offset(int r, int half, int upper, int q) {
  return (((half * 32 + q) * 4 + 2 * upper + (r >> 5)) * 32 + (r & 31)) * 4;
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair::kThreads, 1)
    decode_pair_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kv_map,
                       const __grid_constant__ CUtensorMap v_map, const DecodeParams p) {
  using namespace pair;
  extern __shared__ __align__(1024) uint8_t smem[];
  Control* ctl = reinterpret_cast<Control*>(smem);
  volatile WaitCtl* wctl = &ctl->wait;
  const uint32_t base = ptx::smem_u32(smem);
  const int warp = __shfl_sync(kFull, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1u;      // of the cluster (2, 1, 1); from blockIdx, so that branches on it count as uniform
  const int range = int(blockIdx.x >> 1), ranges = int(gridDim.x >> 1);
  auto bar = [&](const uint64_t& b) { return base + uint32_t(reinterpret_cast<const uint8_t*>(&b) - smem); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kParts; ++i) {
      ptx::mbar_init(bar(ctl->k_full[i]), 4);
      ptx::mbar_init(bar(ctl->k_empty[i]), 1);
    }
    ptx::mbar_init(bar(ctl->v_full), 4);
    for (int i = 0; i < kPieces; ++i) ptx::mbar_init(bar(ctl->v_empty[i]), 1);
    ptx::mbar_init(bar(ctl->q_full), 1);
    ptx::mbar_init(bar(ctl->q_empty), 1);
    ptx::mbar_init(bar(ctl->s_full[0]), 1);
    ptx::mbar_init(bar(ctl->s_full[1]), 1);
    ptx::mbar_init(bar(ctl->p_full), 2 * kSoftmaxThreads / 32);
    ptx::mbar_init(bar(ctl->pv_done), 1);
    ptx::mbar_init(bar(ctl->o_free), 2 * kSoftmaxThreads / 32);
    ptx::mbar_init(bar(ctl->s_free[0]), 2 * kSoftmaxThreads / 32);
    ptx::mbar_init(bar(ctl->s_free[1]), 2 * kSoftmaxThreads / 32);
    ptx::mbar_init(bar(ctl->drain), 2);
    ptx::fence_barrier_init();
    ctl->wait.abort = 0;
    ctl->wait.limit_us = p.wait_us;
    ctl->wait.flags = &g_decode_flags;
  }
  if (warp == kProducer && lane == 0) {
    ptx::prefetch_tmap(&q_map);
    ptx::prefetch_tmap(&kv_map);
    ptx::prefetch_tmap(&v_map);
  }
  if (warp == kIssuer) {
    ptx::tmem_alloc_pair(base + uint32_t(offsetof(Control, tmem)), kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  Cursor<kKeys> cur;                          // its loads run while tensor memory is allocated
  const int share = cur.init(p, range, ranges);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();                        // both CTAs' barriers exist before either signals one
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, ctl->tmem, 0);

  if (warp >= kProducer && warp < kIssuer) {
    // ---- producers: two warps copy whole rows (32 of the CTA's 64 keys
    // each), four copy values (32 of the tile's 128 keys each), so that rows,
    // whose buffers S frees early, never wait behind values.  A tile's pages
    // are looked up while the tile before it waits for its buffers. ----
    const bool rows_role = warp < kProducer + 2;
    const int sub = rows_role ? warp - kProducer : warp - kProducer - 2;
    const uint32_t el = elect_one(), el0 = rank == 0 ? el : 0u, el1 = rank ? el : 0u;  // the even CTA tells its barriers what to expect
    const int oob = p.num_pages * p.page;
    // First cache row of piece `piece` (16 keys) of the cursor's tile.
    auto look_up = [&](const Cursor<kKeys>& c, int piece) {
      const int row = c.tile * kKeys + 16 * piece;
      if (row >= c.len) return oob;
      const int id = __ldg(p.tables + c.b * p.table_stride + (row >> p.log_page));
      if (id >= 0 && id < p.num_pages) return id * p.page + (row & (p.page - 1));
      atomicOr(&g_decode_flags, kFlagBadData);  // zero rows instead of a page that does not exist
      return oob;
    };
    uint32_t g = 0;                           // tiles begun
    if (rows_role) {
      if (sub == 0 && blockIdx.x == 0)        // lengths that are not served as they are
        for (int b = lane; b < p.B; b += 32)
          if (__ldg(p.lens + b) != seq_len(p, b)) atomicOr(&g_decode_flags, kFlagBadData);
      const int piece0 = 4 * int(rank) + 2 * sub;  // the warp's two pieces, one looked up by even lanes, one by odd
      const uint32_t kf = ptx::mapa(bar(ctl->k_full[0]), 0), qf = ptx::mapa(bar(ctl->q_full), 0);
      const uint32_t dst = base + kKOff + 4 * sub * kGroup;
      uint32_t seg = 0, begun = 0;            // parts begun
      int row = cur.valid() ? look_up(cur, piece0 + (lane & 1)) : 0;
      while (cur.valid()) {
        if (sub == 0 && cur.is_first()) {
          if (!wait_warp(bar(ctl->q_empty), (seg & 1u) ^ 1u, wctl)) break;
          arrive_expect_tx(el0, bar(ctl->q_full), 2 * kQBytes);
#pragma unroll
          for (int c = 0; c < 9; c += 3)
            tma_load_3d_pair(el, base + kQOff + c * 64 * 128, &q_map, qf, 0,
                             cur.b * p.rows + (2 * cur.block + int(rank)) * kRows, c);
          ++seg;
        }
        const int groups = (max(cur.keys(), 0) + 7) / 8;  // of 8 keys, in the tile
        Cursor<kKeys> nxt = cur;
        nxt.next(p);
        const int next = nxt.valid() ? look_up(nxt, piece0 + (lane & 1)) : 0;
        // both CTAs' groups 4 sub .. 4 sub + 3 of their eight
        const int mine = min(4, max(0, groups - 4 * sub)), theirs = min(4, max(0, groups - 8 - 4 * sub));
        const int n = rank ? theirs : mine;
        const int from0 = uniform(row), from1 = __shfl_sync(kFull, row, 1);
        bool ok = true;
#pragma unroll 1
        for (int part = 0; part < kParts; ++part) {
          ok = ok && wait_warp(bar(ctl->k_empty[part]), (g & 1u) ^ 1u, wctl);
          if (!ok) break;
          ++begun;
          arrive_expect_tx(el0, bar(ctl->k_full[part]), uint32_t((mine + theirs) * (kGroup / kParts)));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int from = i < 2 ? from0 : from1;
            if (i < n)
              tma_load_3d_pair(el, dst + i * kGroup + part * (kGroup / kParts), &kv_map, kf + 8 * part, 0,
                               min(from, oob - 8 * (i & 1)) + 8 * (i & 1), part * (9 / kParts));
          }
          // The odd CTA's warps arrive too, also where they have no keys to copy:
          // otherwise a slow one could miss a phase of k_empty, whose parity then
          // repeats, and the pair would wait until the limit.  (Behind the copies:
          // ahead of them 128 x 128 took 157 us and not 155.)
          arrive_peer(el1, kf + 8 * part);
        }
        if (!ok) break;
        ++g;
        cur = nxt;
        row = next;
        if (cur.valid()) {                    // the next rows are requested into L2 while their buffers are in use
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int from = __shfl_sync(kFull, row, i);
            const int ahead = min(16, cur.len - cur.tile * kKeys - 16 * (piece0 + i));
            if (ahead > 0 && from != oob)
              prefetch_l2(el, p.cache + int64_t(from) * (2 * kRow), uint32_t(ahead) * (2 * kRow));
          }
        }
      }
      // Every copy has landed before the pair leaves: the even CTA's barriers
      // count both CTAs' (bounded, since an abort may leave a phase incomplete).
      if (rank == 0 && seg) drain_phase(bar(ctl->q_full), (seg - 1) & 1u);
#pragma unroll
      for (uint32_t part = 0; part < kParts; ++part) {
        const uint32_t n = (begun + kParts - 1 - part) / kParts;
        if (rank == 0 && n) drain_phase(bar(ctl->k_full[part]), (n - 1) & 1u);
      }
      // After an abort the odd CTA may have begun a part that the even one did
      // not, and it cannot wait on the other's barriers: 10 ms cover the copy.
      if (rank == 1 && cur.valid()) {
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < 10000000ull) {
        }
      }
    } else {
      bool ok = true;
      const uint32_t vf = bar(ctl->v_full), dst = base + kVOff + 4 * sub * kVGroup;
      int row = cur.valid() ? look_up(cur, 2 * sub + (lane & 1)) : 0;  // of the warp's two pieces
      while (ok && cur.valid()) {
        const int n = min(4, max(0, (cur.keys() + 7) / 8 - 4 * sub));  // groups of 8 keys
        Cursor<kKeys> nxt = cur;
        nxt.next(p);
        const int next = nxt.valid() ? look_up(nxt, 2 * sub + (lane & 1)) : 0;
        const int from0 = uniform(row), from1 = __shfl_sync(kFull, row, 1);
        ok = wait_warp(bar(ctl->v_empty[2 * sub]), (g & 1u) ^ 1u, wctl);
        if (!ok) break;
        arrive_expect_tx(el, vf, uint32_t(n * kVGroup));
        ++g;
        if (n > 0) tma_load_4d(el, dst, &v_map, vf, 0, from0, 2 * int(rank), 0);
        if (n > 1) tma_load_4d(el, dst + kVGroup, &v_map, vf, 0, min(from0, oob - 8) + 8, 2 * int(rank), 0);
        // The second piece's buffer is waited for only where it is copied: without
        // bytes of it the tile does not wait for this warp any more, which could
        // then miss a phase, whose parity repeats.  After an abort the piece still
        // comes: a phase that was begun has to end.
        if (n > 2) ok = wait_warp(bar(ctl->v_empty[2 * sub + 1]), (g & 1u), wctl);
        if (n > 2) tma_load_4d(el, dst + 2 * kVGroup, &v_map, vf, 0, from1, 2 * int(rank), 0);
        if (n > 3) tma_load_4d(el, dst + 3 * kVGroup, &v_map, vf, 0, min(from1, oob - 8) + 8, 2 * int(rank), 0);
        cur = nxt;
        row = next;
      }
      if (g) drain_phase(bar(ctl->v_full), (g - 1) & 1u);
    }
    __syncwarp();
  } else if (warp >= kIssuer) {
    // ---- MMA issuers, in the even CTA: one warp for S, one for P V.  A single
    // warp's waits, commits and list walking between the two products took as
    // long as the MMAs themselves (2600 cycles a tile). ----
    const uint32_t el = elect_one();
    if (rank == 0 && warp == kIssuer) {
      const uint32_t idesc = idesc_f16(Elem<T>::kFormat, 128, kKeys, false, false);
      const uint32_t a = desc_sw128(base + kQOff, 16);
      for (uint32_t g = 0, seg = 0; cur.valid(); ++g) {
        const uint32_t s = g & 1u;
        if (cur.is_first() && !wait_warp(bar(ctl->q_full), seg++ & 1u, wctl)) break;
        if (!wait_warp(bar(ctl->s_free[s]), ((g >> 1) & 1u) ^ 1u, wctl)) break;
        const uint32_t b = desc_sw128(base + kKOff, 16);
        bool ok = true;
#pragma unroll 1
        for (int part = 0; part < kParts; ++part) {
          ok = ok && wait_warp(bar(ctl->k_full[part]), g & 1u, wctl);
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int c = 0; c < 9 / kParts; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16_pair<1024, kGroup>(el, tmem + kSCol + s * kSCols,
                                         a + part * (9 / kParts * 64 * 128 >> 4) + c * (64 * 128 >> 4) + 2 * k,
                                         b + part * (9 / kParts * 1024 >> 4) + c * (1024 >> 4) + 2 * k, idesc,
                                         c + k ? 1u : uint32_t(part));
          tc_commit_pair(el, bar(ctl->k_empty[part]));
        }
        if (!ok) break;
        tc_commit_pair(el, bar(ctl->s_full[s]));
        if (cur.is_last()) tc_commit_pair(el, bar(ctl->q_empty));
        cur.next(p);
      }
    } else if (rank == 0) {
      const uint32_t idesc = idesc_f16(Elem<T>::kFormat, 128, 256, false, true);
      const uint32_t a = desc_sw128(base + kPOff, 16), b = desc_sw128(base + kVOff, 1024);
      for (uint32_t g = 0, seg = 0; cur.valid(); ++g) {
        if (!wait_warp(bar(ctl->p_full), g & 1u, wctl)) break;
        ptx::mbar_acquire_smem(bar(ctl->p_full), g & 1u);
        // the previous segment's accumulator has been read
        if (cur.is_first() && seg++ && !wait_warp(bar(ctl->o_free), seg & 1u, wctl)) break;
        ptx::tc_fence_after();
        const uint32_t more = cur.is_first() ? 0u : 1u;
#pragma unroll 1
        for (int k = 0; k < kPieces; ++k) {   // 16 keys: 32 bytes of P, two groups of values
#pragma unroll
          for (int h = 0; h < 2; ++h)         // 256 values
            mma_f16_pair<1024, kVGroup>(el, tmem + 128 * h, a + (k >> 2) * (kPBytes >> 4) + 2 * (k & 3), b + k * (2 * kVGroup >> 4) + h * (2048 >> 4), idesc,
                         k ? 1u : more);
          tc_commit_pair(el, bar(ctl->v_empty[k]));
        }
        tc_commit_pair(el, bar(ctl->pv_done));
        cur.next(p);
      }
    }
    if (rank == 0) tc_commit_pair(el, bar(ctl->drain));
    // Both CTAs stay until the pair's last MMAs are done and their commits have
    // arrived (the odd one waits here from the start).
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar(ctl->drain), 0))
      if (ptx::globaltimer_ns() - t0 > 30000000000ull) break;
    __syncwarp();
  } else if (warp < kProducer) {
    // ---- softmax and epilogue: this CTA's 64 rows ----
    if (threadIdx.x == 0 && rank == 0) {
      Head h;
      h.share = share;
      h.start = cur.valid() ? cur.pos - cur.tile : 0;
      h.tiles = cur.valid() ? cur.tiles : 0;
      h.b = cur.valid() ? cur.b : 0;
      h.block = cur.valid() ? cur.block : 0;
      p.heads[range] = h;
    }
    // Lane quarters 0 and 1 hold the rows' first 64 keys, 2 and 3 the others;
    // two warps share a quarter, each takes 32 of its columns: a thread has one
    // row and 32 keys, four threads share a row.
    const int quarter = warp & 3, half = warp >> 2, upper = quarter >> 1;
    const uint32_t lanes = uint32_t(32 * quarter) << 16;
    const int r = 32 * (quarter & 1) + lane, key0 = 64 * upper + 32 * half, who = 2 * upper + half;
    const uint32_t p_full = ptx::mapa(bar(ctl->p_full), 0), o_free = ptx::mapa(bar(ctl->o_free), 0);
    const uint32_t s_free = ptx::mapa(bar(ctl->s_free[0]), 0);
    float m = 0.0f, l = 0.0f;                 // running maximum (log2 domain) less kLift, and this quarter's sum
    uint32_t g = 0;
    int behind = 0;                           // keys of the sequence that come after the row's token
    // A failed wait is remembered and ends the loop for all warps at the next
    // tile's vote, so that no thread leaves others at a barrier.
    bool dead = false;
    auto wait = [&](uint32_t b, uint32_t parity) {
      dead |= !wait_phase(b, parity, wctl);
      __syncwarp();
    };
    while (cur.valid()) {
      const bool first = cur.is_first(), last = cur.is_last();
      const int keys = cur.keys(), rows = cur.rows(p, int(rank));
      if (first) {
        behind = p.Sq - 1 - ((2 * cur.block + int(rank)) * kRows + r) / p.H;
        m = -INFINITY, l = 0.0f;
      }
      wait(bar(ctl->s_full[g & 1u]), (g >> 1) & 1u);
      ptx::tc_fence_after();
      uint32_t s[32];
      ptx::tmem_ld_32x32b_x32(tmem + lanes + kSCol + (g & 1u) * kSCols + 32 * half, s);
      ptx::tmem_ld_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(s_free + 8 * (g & 1u));
      const int sees = r < rows ? cur.len - behind - cur.tile * kKeys - key0 : 0;
      if (sees < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i >= sees) s[i] = 0xFF800000u;
      }
      const float top = max_of(s) * p.scale_log2;
      ctl->part[who][r] = top;
      // The reference maximum moves only when some row's maximum grew by 2^8:
      // until then weights of up to 2^8 are as exact as weights of up to 1.
      if (bar_any(1, kSoftmaxThreads, first || dead || top - m > kGrow + Elem<T>::kLift)) {
        if (bar_any(2, kSoftmaxThreads, dead)) break;
        const float tops = fmaxf(fmaxf(ctl->part[0][r], ctl->part[1][r]), fmaxf(ctl->part[2][r], ctl->part[3][r]));
        const float mn = fmaxf(m, tops - Elem<T>::kLift);
        const float a = mn == m ? 1.0f : exp2_approx(m - mn);
        m = mn;
        l *= a;
        bar_sync(2, kSoftmaxThreads);         // all have read the maxima
        if (!first) {
          wait(bar(ctl->pv_done), (g - 1) & 1u);
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t o[32];
            ptx::tmem_ld_32x32b_x32(tmem + lanes + 128 * half + c, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
            ptx::tmem_st_32x32b_x32(tmem + lanes + 128 * half + c, o);
          }
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
        }
      }
      // the weights, rounded to 16 bits for the second product; their sum stays float32
      const float neg = m == -INFINITY ? 0.0f : -m;
      uint32_t w[16];
      float l1 = 0.0f;
      weights<T>(s, w, p.scale_log2, neg, l, l1);
      l += l1;
      if (g) wait(bar(ctl->pv_done), (g - 1) & 1u);  // P is free
      const uint32_t at = base + kPOff + upper * kPBytes + r * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        ptx::sts128(at + (((4 * half + i) ^ (r & 7)) << 4), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      // Rows of the tile past the last key may hold anything, and 0 * NaN is
      // NaN: they are zeroed, once the tile's values have landed, before the
      // second product reads them.
      wait(bar(ctl->v_full), g & 1u);
      if (keys < kKeys) {
        const int from = max(keys, 0);
        const uint32_t v = base + kVOff;
#pragma unroll 1
        for (int i = threadIdx.x; i < (kKeys - from) * 32; i += kSoftmaxThreads) {
          const int k = from + (i >> 5);      // 32 pieces of 16 bytes a key: eight in each of four atoms
          ptx::sts128(v + (k >> 3) * kVGroup + ((i >> 3) & 3) * 1024 + (k & 7) * 128 + (i & 7) * 16, 0, 0, 0, 0);
        }
      }
      // What the arrival announces lies in this CTA, and the even CTA's issuer
      // has both CTAs' tensor cores use it: weights and zeros in shared memory,
      // ordered for the tensor core by the proxy fence and across the pair by
      // the arrival's release, which is restricted to shared memory (a full
      // cluster-scope release waits for global memory too, some 2000 cycles:
      // 128 sequences x 128 heads 202 us, even with one warp alone releasing;
      // like this 154); a rescaled O in tensor memory, by the tcgen05 fence.
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_release_smem(p_full);
      if (last) {
        const bool whole = cur.first == 0 && cur.tile + 1 == cur.tiles;
        const int64_t part = 2 * blockIdx.x + (cur.pos - cur.tile + cur.first == share * range ? 0 : 1);
        const int64_t row0 = whole ? int64_t(cur.b) * p.rows + (2 * cur.block + int(rank)) * kRows : part * kRows;
        ctl->part[who][r] = l;                // the maxima have been read
        bar_sync(2, kSoftmaxThreads);
        const float sum = (ctl->part[0][r] + ctl->part[1][r]) + (ctl->part[2][r] + ctl->part[3][r]);
        bar_sync(2, kSoftmaxThreads);         // all have read the sums: the next tile's maxima take their place
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (who == 0 && r < rows) {
          const float e = sum == 0.0f ? -INFINITY : m + log2f(sum);
          (whole ? p.lse : p.part_lse)[row0 + r] = whole ? e * kLn2 : e;
        }
        const bool empty = __any_sync(kFull, sum == 0.0f);  // some row saw no key
        wait(bar(ctl->pv_done), g & 1u);
        ptx::tc_fence_after();
        // Columns 32 c .. of half `half` are values 256 half + 128 upper + 32 c ...
        // Not unrolled here and where else code runs once an item: its
        // instructions come from L2 each time (unrolled, 5 us an item).
        const uint32_t stage = base + kPOff + warp * 2048;  // P is free until the next tile's vote
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          ptx::tmem_ld_32x32b_x32(tmem + lanes + 128 * half + 32 * c, o);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
          if (empty) {                        // zeros, also where masked values were not finite
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (sum == 0.0f) o[i] = 0u;
          }
          if (whole) {
            // a row's 64 bytes through shared memory, so that a store covers 8 rows' whole sectors
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = Elem<T>::pack(__uint_as_float(o[8 * i + 2 * e]), __uint_as_float(o[8 * i + 2 * e + 1]));
              ptx::sts128(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
            T* out = reinterpret_cast<T*>(p.out) + row0 * kLatent + 256 * half + 128 * upper + 32 * c + 8 * (lane & 3);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int q = 8 * k + (lane >> 2), row = 32 * (quarter & 1) + q;
              const uint4 w = ptx::lds128(stage + q * 64 + (((lane & 3) ^ ((q >> 1) & 3)) << 4));
              if (row < rows) *reinterpret_cast<uint4*>(out + int64_t(row) * kLatent) = w;
            }
            __syncwarp();
          } else {
            // partial rows stay in the order of tensor memory (part_offset), 512 bytes a store
            float* out = p.part_o + part * kRows * kLatent;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(out + part_offset(r, half, upper, 8 * c + i)) =
                  make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(o_free);
      }
      cur.next(p);
      ++g;
    }
  }

  // No CTA of the pair leaves, or frees its tensor memory, while the other's
  // MMAs or copies may still use it.
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  if (warp == kIssuer) ptx::tmem_dealloc_pair(tmem, kTmemCols);
  ptx::cluster_sync();
}

// Joins the pair kernel's partial results (see join_kernel).  A warp takes
// eight rows and 128 values: lane l row l % 8 and every fourth piece of four
// values, so that loads cover 128 contiguous bytes and stores whole sectors.
// BY_ITEM: block (item, .), eight warps share the pieces of the ranges.
constexpr int kPairJoinThreads = 128;
template <typename T, bool BY_ITEM>
__global__ void __launch_bounds__((BY_ITEM ? 2 : 1) * kPairJoinThreads) join_pair_kernel(const DecodeParams p) {
  constexpr int kShare = BY_ITEM ? 8 : 1;
  __shared__ float4 s_sum[kShare][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int start, tiles, share, b, block;
  if (BY_ITEM) find_item<pair::kKeys>(p, blockIdx.x, b, block, start, tiles, share);  // as in join_kernel
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  if (!BY_ITEM) {
    const Head h = p.heads[blockIdx.x + 1];
    start = h.start, tiles = h.tiles, share = h.share, b = h.b, block = h.block;
    if (!border_joins(int(blockIdx.x), start, tiles, share)) return;
  }
  const int first = start / share, last = (start + tiles - 1) / share;
  if (first == last) return;                  // whole: written by its pair
  const int pieces = last - first + 1, lead = start != first * share ? 1 : 0;
  // 16 groups of eight rows x four blocks of 128 values: blockIdx.y, and the warp where it has no pieces of its own
  const int task = BY_ITEM ? blockIdx.y : blockIdx.y * 4 + warp;
  const int row = (task >> 2) * 8 + (lane & 7), half = (task >> 1) & 1, upper = task & 1, q0 = lane >> 3;
  const int rows = p.rows - block * 2 * kRows;  // of the item
  if ((task >> 2) * 8 >= rows) return;        // the same for all warps that share a row
  const int cta = row >> 6, r = row & 63;
  auto slot = [&](int i) { return int64_t(2 * (2 * (first + i) + cta) + (i == 0 ? lead : 0)); };
  float top = -INFINITY, sum = 0.0f;
  const bool live = row < rows;
  // the four lanes of a row share its log-sums
  if (live) {
#pragma unroll 4
    for (int i = q0; i < pieces; i += 4) top = fmaxf(top, p.part_lse[slot(i) * kRows + r]);
  }
  top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
  top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
  const float ref = top == -INFINITY ? 0.0f : top;
  if (live) {
#pragma unroll 4
    for (int i = q0; i < pieces; i += 4) sum += exp2_approx(p.part_lse[slot(i) * kRows + r] - ref);
  }
  sum += __shfl_xor_sync(kFull, sum, 8);
  sum += __shfl_xor_sync(kFull, sum, 16);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  float4 acc[8] = {};
  if (live) {
    constexpr int kAhead = BY_ITEM ? 3 : 2;   // pieces whose loads are in flight together
#pragma unroll 1
    for (int i = BY_ITEM ? warp : 0; i < pieces; i += kAhead * kShare) {
      float4 o[kAhead][8];
      float a[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const bool more = i + j * kShare < pieces;
        const int64_t from = slot(more ? i + j * kShare : i);
        const float* at = p.part_o + from * kRows * kLatent;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          o[j][k] = more ? *reinterpret_cast<const float4*>(at + part_offset(r, half, upper, 4 * k + q0)) : float4{};
        a[j] = more ? p.part_lse[from * kRows + r] : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const float w = exp2_approx(a[j] - ref) * inv;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          acc[k].x += w * o[j][k].x, acc[k].y += w * o[j][k].y, acc[k].z += w * o[j][k].z, acc[k].w += w * o[j][k].w;
      }
    }
  }
  const int64_t at = int64_t(b) * p.rows + block * 2 * kRows + row;
  auto store = [&](int k, float4 v) {
    *reinterpret_cast<uint2*>(p.out + 2 * (at * kLatent + 256 * half + 128 * upper + 4 * (4 * k + q0))) =
        make_uint2(Elem<T>::pack(v.x, v.y), Elem<T>::pack(v.z, v.w));
  };
  if (live && (task & 3) == 0 && q0 == 0 && (!BY_ITEM || warp == 0))
    p.lse[at] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * kLn2;
  if (BY_ITEM) {                              // warp k adds up the k-th part of the values
#pragma unroll
    for (int k = 0; k < 8; ++k) s_sum[warp][k][lane] = acc[k];
    __syncthreads();
    float4 v = s_sum[0][warp][lane];
#pragma unroll
    for (int i = 1; i < kShare; ++i) {
      const float4 o = s_sum[i][warp][lane];
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    if (live) store(warp, v);
  } else if (live) {
#pragma unroll
    for (int k = 0; k < 8; ++k) store(k, acc[k]);
  }
}

}  // namespace
}  // namespace nvfp4moe
