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
// partial results (unnormalised rows and their log-sums) in the workspace,
// which a second kernel joins.
//
// Warp roles: warps 0-3 softmax and epilogue, warp 4 TMA producer, warp 5
// tensor-memory owner and MMA issuer.  Every wait is bounded.
#include <algorithm>
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

__device__ unsigned g_decode_flags = 0;

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kRows = 64;                     // rows of a block
constexpr int kKeys = 64;                     // keys of a tile
constexpr int kChunk = 64 * 128;              // 64 rows x 64 values, 128-byte rows
constexpr int kTile = 9 * kChunk;
constexpr int kGroup = 8 * 2 * kRow;          // 8 keys: nine atoms of 8 rows x 128 bytes
constexpr int kPieces = 4;                    // of a tile: 16 keys each, freed one by one
constexpr int kStages = 2;
constexpr int kThreads = 192;
constexpr int kSoftmaxThreads = 128;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;               // S buffers after the 4 x 64 columns of O^T
constexpr float kGrow = 8.0f;                 // rescale O only when a maximum grew by 2^8

// Shared memory after the 1024-byte control block.
constexpr int kCtrl = 1024;
constexpr int kQOff = kCtrl;
constexpr int kKvOff = kQOff + kTile;
constexpr int kPOff = kKvOff + kStages * kTile;
constexpr int kSmem = kPOff + kChunk;

struct Control {
  uint64_t full[kStages], empty[kStages][kPieces];
  uint64_t q_full, q_empty, s_full[2], p_full, pv_done, o_free, drain;
  uint32_t tmem, pad;
  WaitCtl wait;
  float col[kRows];                           // per-row factors for the transposed accumulator
};
static_assert(sizeof(Control) <= kCtrl, "control block");
static_assert(kSmem <= 232448, "shared memory");

// What CTA c's range begins with, for the kernel that joins partial results.
struct Head {
  int64_t tile, tiles;                        // first tile within the item, and the item's tiles
  int32_t b, block;
};

struct DecodeParams {
  const int32_t* tables;
  int64_t table_stride;
  const int32_t* lens;
  int B, Sq, H, rows, blocks;                 // rows = Sq * H of a sequence, in `blocks` row blocks
  int num_pages, page, log_page, max_pages;
  float scale_log2, scale;
  uint8_t* out;                               // [B, rows, 512]
  float* lse;                                 // [B, rows]
  int64_t min_share;
  Head* heads;                                // [grid]
  float* part_o;                              // [grid][2][64][512]
  float* part_lse;                            // [grid][2][64], log2 domain
  uint32_t wait_us;
};

__device__ __forceinline__ int seq_len(const DecodeParams& p, int b) {
  const int n = __ldg(p.lens + b);
  return n < 0 ? 0 : int(min(int64_t(n), int64_t(p.max_pages) * p.page));
}
// Tiles of an item; an empty sequence has one, whose keys are all masked.
__device__ __forceinline__ int64_t item_tiles(int len) { return len > 0 ? (len + kKeys - 1) / kKeys : 1; }

// Walks the tiles [pos, end) of the flattened (sequence, row block, tile) list.
struct Cursor {
  int64_t pos, end;                           // in the tile list
  int64_t tile, tiles, first;                 // within the item; where this CTA entered it
  int b, block, len;

  // Executed by a whole warp: the CTA's range and its first item.  Returns the share.
  __device__ __forceinline__ int64_t init(const DecodeParams& p) {
    const int lane = threadIdx.x & 31;
    int64_t total = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) total += b0 + lane < p.B ? item_tiles(seq_len(p, b0 + lane)) : 0;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) total += __shfl_xor_sync(kFull, total, d);
    total *= p.blocks;
    int64_t share = (total + gridDim.x - 1) / gridDim.x;
    share = share > p.min_share ? share : p.min_share;
    pos = share * blockIdx.x;
    end = min(total, pos + share);
    if (pos >= end) return share;
    int64_t before = 0;                       // tiles of the sequences before b0
    for (int b0 = 0;; b0 += 32) {
      const int n = b0 + lane < p.B ? seq_len(p, b0 + lane) : 0;
      const int64_t mine = b0 + lane < p.B ? item_tiles(n) * p.blocks : 0;
      int64_t upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t v = __shfl_up_sync(kFull, upto, d);
        if (lane >= d) upto += v;
      }
      const unsigned hit = __ballot_sync(kFull, before + upto > pos);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b = b0 + src;
        len = __shfl_sync(kFull, n, src);
        const int64_t in = pos - before - __shfl_sync(kFull, upto - mine, src);
        tiles = item_tiles(len);
        block = int(in / tiles);
        tile = first = in - int64_t(block) * tiles;
        return share;
      }
      before += __shfl_sync(kFull, upto, 31);
    }
  }
  __device__ __forceinline__ bool valid() const { return pos < end; }
  __device__ __forceinline__ bool is_first() const { return tile == first; }
  __device__ __forceinline__ bool is_last() const { return tile + 1 == tiles || pos + 1 == end; }
  __device__ __forceinline__ void next(const DecodeParams& p) {
    ++pos;
    if (++tile == tiles) {
      tile = first = 0;
      if (++block == p.blocks) {
        block = 0;
        if (++b < p.B) {
          len = seq_len(p, b);
          tiles = item_tiles(len);
        }
      }
    }
  }
  __device__ __forceinline__ int keys() const { return min(kKeys, len - int(tile) * kKeys); }  // <= 0: none
  __device__ __forceinline__ int rows(const DecodeParams& p) const { return min(kRows, p.rows - block * kRows); }
};

// 16-bit rows [rows, 576] in boxes of `box_rows` rows x `chunks` chunks of 64
// values, which land chunk by chunk, each as box_rows x 128 bytes.
template <typename T>
bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int box_rows, int chunks) {
  const int64_t dims[3] = {64, rows, kRow / 64}, strides[2] = {2 * kRow, 128};
  const int box[3] = {64, box_rows, chunks};
  return encode_map(m, Elem<T>::kMap, 3, base, dims, strides, box);
}

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
      ptx::mbar_init(bar(ctl->full[s]), 1);
      for (int i = 0; i < kPieces; ++i) ptx::mbar_init(bar(ctl->empty[s][i]), 1);
    }
    ptx::mbar_init(bar(ctl->q_full), 1);
    ptx::mbar_init(bar(ctl->q_empty), 1);
    ptx::mbar_init(bar(ctl->s_full[0]), 1);
    ptx::mbar_init(bar(ctl->s_full[1]), 1);
    ptx::mbar_init(bar(ctl->p_full), kSoftmaxThreads);
    ptx::mbar_init(bar(ctl->pv_done), 1);
    ptx::mbar_init(bar(ctl->o_free), kSoftmaxThreads);
    ptx::mbar_init(bar(ctl->drain), 1);
    ptx::fence_barrier_init();
    ctl->wait.abort = 0;
    ctl->wait.limit_us = p.wait_us;
    ctl->wait.flags = &g_decode_flags;
  }
  if (warp == 4 && lane == 0) {
    ptx::prefetch_tmap(&q_map);
    ptx::prefetch_tmap(&kv_map);
  }
  if (warp == 5) {
    ptx::tmem_alloc(base + uint32_t(offsetof(Control, tmem)), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, ctl->tmem, 0);
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();

  Cursor cur;
  const int64_t share = cur.init(p);

  if (warp == 4) {
    // ---- producer ----
    if (blockIdx.x == 0)                      // lengths that are not served as they are
      for (int b = lane; b < p.B; b += 32)
        if (__ldg(p.lens + b) != seq_len(p, b)) atomicOr(&g_decode_flags, kFlagBadData);
    const uint32_t el = elect_one();
    const int oob = p.num_pages * p.page;
    const int per = p.page < kKeys ? kKeys / p.page : 1;  // pages of a tile
    uint32_t g = 0, seg = 0;
    // First cache rows of the tile's four pieces of 16 keys, one a lane.
    auto look_up = [&](const Cursor& c) {
      const int row = int(c.tile) * kKeys, i = lane & (kPieces - 1);
      if (i * 16 >= c.keys()) return oob;
      const int id = __ldg(p.tables + c.b * p.table_stride + (row >> p.log_page) + ((i * per) >> 2));
      if (id >= 0 && id < p.num_pages) return id * p.page + ((row + 16 * i) & (p.page - 1));
      atomicOr(&g_decode_flags, kFlagBadData);  // zero rows instead of a page that does not exist
      return oob;
    };
    int mine = cur.valid() ? look_up(cur) : 0;
    bool ok = true;
    while (ok && cur.valid()) {
      if (cur.is_first()) {
        if (!wait_warp(bar(ctl->q_empty), (seg & 1u) ^ 1u, wctl)) break;
        arrive_expect_tx(el, bar(ctl->q_full), kTile);
#pragma unroll
        for (int c = 0; c < 9; c += 3)
          tma_load_3d(el, base + kQOff + c * kChunk, &q_map, bar(ctl->q_full), 0, cur.b * p.rows + cur.block * kRows, c);
        ++seg;
      }
      const uint32_t s = g & 1u, ph = (g >> 1) & 1u, fb = bar(ctl->full[s]);
      const int groups = (max(cur.keys(), 0) + 7) / 8;
      Cursor nxt = cur;
      nxt.next(p);
      const int next = nxt.valid() ? look_up(nxt) : 0;
      const uint32_t dst = base + kKvOff + s * kTile;
      ok = wait_warp(bar(ctl->empty[s][0]), ph ^ 1u, wctl);
      if (!ok) break;
      arrive_expect_tx(el, fb, uint32_t(groups * kGroup));
      ++g;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        // After an abort the rest of the tile still comes: the copies that
        // the barrier was told to expect have to end before the CTA does.
        if (i && ok) ok = wait_warp(bar(ctl->empty[s][i]), ph ^ 1u, wctl);
        const int from = __shfl_sync(kFull, mine, i);
        if (2 * i < groups) tma_load_3d(el, dst + 2 * i * kGroup, &kv_map, fb, 0, from, 0);
        if (2 * i + 1 < groups)
          tma_load_3d(el, dst + (2 * i + 1) * kGroup, &kv_map, fb, 0, min(from, oob - 8) + 8, 0);
      }
      mine = next;
      cur = nxt;
    }
    // every copy that was issued has landed before the CTA leaves
    if (seg) drain_phase(bar(ctl->q_full), (seg - 1) & 1u);
    for (uint32_t s = 0; s < kStages; ++s) {
      const uint32_t n = (g + 1 - s) / 2;     // uses of the stage
      if (n) drain_phase(bar(ctl->full[s]), (n - 1) & 1u);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ---- MMA issuer ----
    const uint32_t el = elect_one();
    const uint32_t idesc_s = idesc_f16(Elem<T>::kFormat, 64, kKeys, false, false);
    uint32_t gs = 0, gp = 0, seg_s = 0, seg_p = 0;  // tiles and segments begun by S and by P V
    Cursor cs = cur;
    uint64_t idle_since = 0;
    uint32_t idle = 0;
    // S of the next tile and P V of the oldest go out as their operands
    // arrive: S first would leave a tile's buffer occupied while the next
    // tile is still on its way.
    while (cur.valid()) {
      if (cs.valid() && gs <= gp + 1 && test_warp(bar(ctl->full[gs & 1u]), (gs >> 1) & 1u) &&
          (!cs.is_first() || test_warp(bar(ctl->q_full), seg_s & 1u))) {
        ptx::tc_fence_after();
        const uint32_t d = tmem + kSCol + (gs & 1u) * kKeys;
        const uint64_t a = desc_sw128(base + kQOff, 16, 1024);
        const uint64_t b = desc_sw128(base + kKvOff + (gs & 1u) * kTile, 16, kGroup);
#pragma unroll
        for (int c = 0; c < 9; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16(el, d, a + c * (kChunk >> 4) + 2 * k, b + c * (1024 >> 4) + 2 * k, idesc_s, c + k > 0);
        tc_commit(el, bar(ctl->s_full[gs & 1u]));
        if (cs.is_last()) tc_commit(el, bar(ctl->q_empty));
        if (cs.is_first()) ++seg_s;
        cs.next(p);
        ++gs;
        idle = 0;
      } else if (gp < gs && test_warp(bar(ctl->p_full), gp & 1u) &&
                 // the previous segment's accumulator has been read
                 (!cur.is_first() || seg_p == 0 || test_warp(bar(ctl->o_free), (seg_p - 1) & 1u))) {
        ptx::tc_fence_after();
        const uint32_t idesc_o = idesc_f16(Elem<T>::kFormat, 128, (cur.rows(p) + 15) / 16 * 16, true, false);
        const uint32_t more = cur.is_first() ? 0u : 1u;
        const uint64_t a = desc_sw128(base + kKvOff + (gp & 1u) * kTile, 1024, kGroup);
        const uint64_t b = desc_sw128(base + kPOff, 16, 1024);
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {   // 16 keys: two groups of C, 32 bytes of P
#pragma unroll
          for (int m = 0; m < 4; ++m)         // 128 values: two chunks
            mma_f16(el, tmem + m * kRows, a + k * (2 * kGroup >> 4) + m * (2 * 1024 >> 4), b + 2 * k, idesc_o,
                    k ? 1u : more);
          tc_commit(el, bar(ctl->empty[gp & 1u][k]));
        }
        tc_commit(el, bar(ctl->pv_done));
        if (cur.is_first()) ++seg_p;
        cur.next(p);
        ++gp;
        idle = 0;
      } else if ((++idle & 255u) == 0u) {
        const uint64_t now = ptx::globaltimer_ns();
        if (idle == 256u) idle_since = now;
        bool quit = wctl->abort != 0;
        if (now - idle_since > uint64_t(wctl->limit_us) * 1000u) {
          wctl->abort = 1;
          atomicOr(&g_decode_flags, kFlagTimeout);
          quit = true;
        }
        if (__any_sync(kFull, quit)) break;
      }
    }
    tc_commit(el, bar(ctl->drain));
    drain_phase(bar(ctl->drain), 0);
    __syncwarp();
  } else {
    // ---- softmax and epilogue ----
    if (threadIdx.x == 0) {
      Head h;
      h.tile = cur.valid() ? cur.tile : 0;
      h.tiles = cur.valid() ? cur.tiles : 0;
      h.b = cur.valid() ? cur.b : 0;
      h.block = cur.valid() ? cur.block : 0;
      p.heads[blockIdx.x] = h;
    }
    const uint32_t quarter = uint32_t(warp) << 21;  // lane 32 * warp
    const int r0 = 16 * warp + (lane >> 2);         // this thread's rows: r0 and r0 + 8
    float m[2], l[2];                               // running maximum (log2 domain) and sum
    uint32_t g = 0;
    // A failed wait is remembered and ends the loop for all four warps at the
    // next tile's vote, so that no thread leaves others at a barrier.
    bool dead = false;
    auto wait = [&](uint32_t b, uint32_t parity) {
      dead |= !wait_phase<false>(b, parity, wctl);
      __syncwarp();
    };
    while (cur.valid()) {
      const bool first = cur.is_first(), last = cur.is_last();
      const int keys = cur.keys(), rows = cur.rows(p);
      wait(bar(ctl->s_full[g & 1u]), (g >> 1) & 1u);
      ptx::tc_fence_after();
      uint32_t sr[32];
      tmem_ld_16x256b_x8(tmem + quarter + kSCol + (g & 1u) * kKeys, sr);
      ptx::tmem_ld_wait();
      ptx::tc_fence_before();
      // keys that row r0 + 8 i sees in this tile: query token s of Sq sees len - Sq + s + 1
      int sees[2];
      bool masked = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + 8 * i;
        const int tok = (cur.block * kRows + r) / p.H;
        sees[i] = r < rows ? cur.len - (p.Sq - 1 - tok) - int(cur.tile) * kKeys : 0;
        masked |= sees[i] < kKeys;
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (8 * (i >> 2) + 2 * (lane & 3) + (i & 1) >= sees[(i >> 1) & 1]) sr[i] = 0xFF800000u;
      }
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 32; ++i) top[(i >> 1) & 1] = fmaxf(top[(i >> 1) & 1], __uint_as_float(sr[i]));
      bool grew = false;
      float mn[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(kFull, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(kFull, top[i], 2));
        top[i] *= p.scale_log2;
        if (first) m[i] = top[i], l[i] = 0.0f;  // a first tile grows nothing
        mn[i] = fmaxf(m[i], top[i]);
        grew |= mn[i] - m[i] > kGrow;         // also from -inf
      }
      if (bar_any(1, kSoftmaxThreads, grew || dead)) {
        if (bar_any(2, kSoftmaxThreads, dead)) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = mn[i] == m[i] ? 1.0f : exp2_approx(m[i] - mn[i]);
          m[i] = mn[i];
          l[i] *= a;
          if ((lane & 3) == 0) ctl->col[r0 + 8 * i] = a;
        }
        bar_sync(2, kSoftmaxThreads);
        wait(bar(ctl->pv_done), (g - 1) & 1u);
        ptx::tc_fence_after();
        for (int c = 0; c < 4 * kRows; c += 32) {
          if ((c & (kRows - 1)) >= rows) continue;
          uint32_t o[32];
          ptx::tmem_ld_32x32b_x32(tmem + quarter + c, o);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * ctl->col[(c & (kRows - 1)) + i]);
          ptx::tmem_st_32x32b_x32(tmem + quarter + c, o);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
      }
      // the weights, rounded to 16 bits for the second product; their sum stays float32
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int k = (i >> 1) & 1;
        const float e = exp2_approx(fmaf(__uint_as_float(sr[i]), p.scale_log2, m[k] == -INFINITY ? 0.0f : -m[k]));
        l[k] += e;
        sr[i] = __float_as_uint(e);
      }
      if (g) wait(bar(ctl->pv_done), (g - 1) & 1u);  // P is free
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const int r = r0 + 8 * ((i >> 1) & 1);
        sts32(base + kPOff + r * 128 + (((i >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4,
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
        const int64_t part = 2 * int64_t(blockIdx.x) + (cur.pos - cur.tile + cur.first == share * blockIdx.x ? 0 : 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[i] += __shfl_xor_sync(kFull, l[i], 1);
          l[i] += __shfl_xor_sync(kFull, l[i], 2);
          const int r = r0 + 8 * i;
          const float e = l[i] == 0.0f ? -INFINITY : m[i] + log2f(l[i]);
          if ((lane & 3) == 0) {
            ctl->col[r] = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
            if (r < rows) {
              if (whole) p.lse[int64_t(cur.b) * p.rows + cur.block * kRows + r] = e * kLn2;
              else p.part_lse[part * kRows + r] = e;
            }
          }
        }
        bar_sync(2, kSoftmaxThreads);
        wait(bar(ctl->pv_done), g & 1u);
        ptx::tc_fence_after();
        for (int c = 0; c < 4 * kRows; c += 32) {
          const int c0 = c & (kRows - 1);     // first row of the piece
          if (c0 >= rows) continue;
          uint32_t o[32];
          ptx::tmem_ld_32x32b_x32(tmem + quarter + c, o);
          ptx::tmem_ld_wait();
          const int dim = (c / kRows) * 128 + 32 * warp + lane;
          if (whole) {
            T* out = reinterpret_cast<T*>(p.out) +
                     (int64_t(cur.b) * p.rows + cur.block * kRows + c0) * kLatent + dim;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float v = ctl->col[c0 + i] == 0.0f ? 0.0f : __uint_as_float(o[i]) * ctl->col[c0 + i];
              if (c0 + i < rows) out[i * kLatent] = Elem<T>::from(v);
            }
          } else {
            float* out = p.part_o + (part * kRows + c0) * kLatent + dim;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float v = ctl->col[c0 + i] == 0.0f ? 0.0f : __uint_as_float(o[i]) * ctl->col[c0 + i];
              if (c0 + i < rows) out[i * kLatent] = v;
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
  if (warp == 5) ptx::tmem_dealloc(tmem, kTmemCols);
}

// Joins the partial results of the items that a range border cut.  Block
// (c, .) serves the item that CTA c + 1's range begins inside of, if no
// earlier range does.  With e_i the log2-sum of piece i and o_i its
// normalised rows, out = sum 2^(e_i - e) o_i, e = log2 sum 2^e_i.
// A block takes `4 / groups` rows; `groups` sets of 128 threads (four values
// each) share a row's pieces.
template <typename T>
__global__ void __launch_bounds__(512) join_kernel(const DecodeParams p, int grid, int groups) {
  __shared__ float4 s_sum[3][128];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int c = int(blockIdx.x) + 1;
  const Head h = p.heads[c];
  if (h.tile == 0 || h.tiles == 0) return;
  // the share is the same for every CTA: recovered from this one's predecessor
  const Head before = p.heads[c - 1];
  const bool same = before.b == h.b && before.block == h.block && before.tiles == h.tiles && before.tile != 0;
  if (same) return;                           // an earlier border inside the item serves it
  // pieces: the end of range c - 1, then ranges c, c + 1, ... while they begin inside the item
  int last = c;
  while (last + 1 < grid) {
    const Head n = p.heads[last + 1];
    if (n.b != h.b || n.block != h.block || n.tile == 0 || n.tiles == 0) break;
    ++last;
  }
  const int pieces = last - c + 2;
  const int set = threadIdx.x >> 7, t = threadIdx.x & 127;
  const int row = blockIdx.y * (4 / groups) + set / groups, grp = set % groups;
  const int rows = min(kRows, p.rows - h.block * kRows);
  const bool live = row < rows;
  // piece 0 is the first segment of range c - 1 if that range begins with the item, else its last
  const bool at_start = before.b == h.b && before.block == h.block && before.tiles != 0 && before.tile == 0;
  auto piece_row = [&](int i) -> int64_t {
    return (i == 0 ? 2 * int64_t(c - 1) + (at_start ? 0 : 1) : 2 * int64_t(c - 1 + i)) * kRows + row;
  };
  float e_top = -INFINITY, sum = 0.0f;
  float4 acc = make_float4(0, 0, 0, 0);
  if (live) {
    for (int i = 0; i < pieces; ++i) e_top = fmaxf(e_top, p.part_lse[piece_row(i)]);
    const float ref = e_top == -INFINITY ? 0.0f : e_top;
    for (int i = 0; i < pieces; ++i) sum += exp2_approx(p.part_lse[piece_row(i)] - ref);
    const float e = sum == 0.0f ? -INFINITY : ref + log2f(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll 4
    for (int i = grp; i < pieces; i += groups) {
      const int64_t at = piece_row(i);
      const float w = exp2_approx(p.part_lse[at] - ref) * inv;
      const float4 o = *reinterpret_cast<const float4*>(p.part_o + at * kLatent + 4 * t);
      acc.x += w * o.x, acc.y += w * o.y, acc.z += w * o.z, acc.w += w * o.w;
    }
    if (grp == 0 && t == 0) p.lse[int64_t(h.b) * p.rows + h.block * kRows + row] = e * kLn2;
  }
  if (groups > 1) {
    if (grp) s_sum[set - 1][t] = acc;
    __syncthreads();
    if (grp) return;
    for (int i = 1; i < groups; ++i) {
      const float4 o = s_sum[set + i - 1][t];
      acc.x += o.x, acc.y += o.y, acc.z += o.z, acc.w += o.w;
    }
  }
  if (live)
    *reinterpret_cast<uint2*>(p.out + 2 * ((int64_t(h.b) * p.rows + h.block * kRows + row) * kLatent + 4 * t)) =
        make_uint2(Elem<T>::pack(acc.x, acc.y), Elem<T>::pack(acc.z, acc.w));
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles a CTA takes at least: below this, splitting a sequence costs more in partial results than it gains.
constexpr int64_t kMinShare = 4;

// Most tiles the call can have, and the grid that covers them.
int64_t most_tiles(const MlaDecodeArgs& a) {
  const int64_t longest = std::max<int64_t>(1, ceil_div(int64_t(a.max_pages) * a.page, kKeys));
  return int64_t(a.B) * ceil_div(int64_t(a.Sq) * a.H, kRows) * longest;
}

template <typename T>
int launch(const MlaDecodeArgs& a, int num_sms, cudaStream_t st) {
  CUtensorMap q_map, kv_map;
  const int rows = a.Sq * a.H;
  if (!encode_rows<T>(&q_map, a.q, int64_t(a.B) * rows, kRows, 3) ||
      !encode_rows<T>(&kv_map, a.cache, int64_t(a.num_pages) * a.page, 8, 9)) {
    set_error_detail("cuTensorMapEncodeTiled failed or is unavailable");
    return NVFP4MOE_ERR_CUDA;
  }
  const int grid = int(std::min<int64_t>(std::min(num_sms, kMlaDecodeMaxGrid), ceil_div(most_tiles(a), kMinShare)));
  DecodeParams p;
  p.tables = a.tables;
  p.table_stride = a.table_stride;
  p.lens = a.lens;
  p.B = a.B, p.Sq = a.Sq, p.H = a.H;
  p.rows = rows;
  p.blocks = int(ceil_div(rows, kRows));
  p.num_pages = a.num_pages;
  p.page = a.page;
  p.log_page = 0;
  while ((1 << p.log_page) < a.page) ++p.log_page;
  p.max_pages = a.max_pages;
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  p.out = static_cast<uint8_t*>(a.out);
  p.lse = a.lse;
  p.min_share = kMinShare;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.heads = reinterpret_cast<Head*>(ws);
  p.part_lse = reinterpret_cast<float*>(ws + kMlaDecodeHeadBytes);
  p.part_o = p.part_lse + int64_t(kMlaDecodeMaxGrid) * 2 * kRows;
  p.wait_us = wait_limit_us();
  static_assert(sizeof(Head) * (kMlaDecodeMaxGrid + 1) <= kMlaDecodeHeadBytes, "workspace header");
  auto kernel = decode_kernel<T>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (err == cudaSuccess) err = launch_kernel(kernel, dim3(grid), dim3(kThreads), kSmem, st, false, q_map, kv_map, p);
  if (err == cudaSuccess && grid > 1) {
    const int groups = int64_t(a.B) * p.blocks * 8 <= grid ? 4 : 1;
    err = launch_kernel(join_kernel<T>, dim3(grid - 1, kRows * groups / 4), dim3(512), 0, st, false, p, grid, groups);
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

cudaError_t mla_decode_read_and_clear_flags(unsigned* flags) {
  unsigned zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(flags, g_decode_flags, sizeof(unsigned));
  if (err != cudaSuccess) return err;
  return cudaMemcpyToSymbol(g_decode_flags, &zero, sizeof(unsigned));
}

}  // namespace nvfp4moe
