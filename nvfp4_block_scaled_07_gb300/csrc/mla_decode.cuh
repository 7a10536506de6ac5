// Shared by the two absorbed-attention kernels (one CTA, CTA pair): the tile
// list and its ranges, and the workspace that joins their partial results.
#pragma once

#include <cstddef>
#include <cstdint>

#include "mla_common.cuh"
#include "mla_join.h"

namespace nvfp4moe {
namespace {

using namespace mla;

__device__ unsigned g_decode_flags = 0;

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kRows = 64;                     // rows of a CTA
constexpr int kGroup = 8 * 2 * kRow;          // 8 keys: nine atoms of 8 rows x 128 bytes
constexpr float kGrow = 8.0f;                 // rescale O only when a maximum grew by 2^8

// What a CTA's range begins with, for the kernel that joins partial results.
struct Head {
  int32_t start, tiles, share;                // the item's place in the tile list, its tiles; tiles of a range
  int32_t b, block;
};

struct DecodeParams {
  const uint8_t* cache;
  const int32_t* tables;
  int64_t table_stride;
  const int32_t* lens;
  int B, Sq, H, rows, blocks;                 // rows = Sq * H of a sequence, in `blocks` row blocks
  int ctas;                                   // CTAs of a range: one with 64 rows, or a pair with 128
  int num_pages, page, log_page, max_pages;
  float scale_log2;
  uint8_t* out;                               // [B, rows, 512]
  float* lse;                                 // [B, rows]
  int ranges, min_share;
  Head* heads;                                // [ranges]
  float* part_o;                              // [grid][2][64][512]
  float* part_lse;                            // [grid][2][64], log2 domain
  uint32_t wait_us;
};

__device__ __forceinline__ int seq_len(const DecodeParams& p, int b) {
  const int n = __ldg(p.lens + b);
  return n < 0 ? 0 : int(min(int64_t(n), int64_t(p.max_pages) * p.page));
}
// Tiles of an item; an empty sequence has one, whose keys are all masked.
template <int KEYS>
__device__ __forceinline__ int item_tiles(int len) {
  return len > 0 ? (len + KEYS - 1) / KEYS : 1;
}

// Tiles of a range, of `total` in the list.
__device__ __forceinline__ int range_tiles(const DecodeParams& p, int total, int ranges) {
  return max(int((unsigned(total) + ranges - 1) / ranges), p.min_share);
}

// Walks the tiles [pos, end) of range `index` of `ranges` of the flattened (sequence, row block, tile) list.
template <int KEYS>
struct Cursor {
  int pos, end;                               // in the tile list
  int tile, tiles, first;                     // within the item; where this CTA entered it
  int b, block, len;

  // Executed by a whole warp: the range and its first item.  Returns the share.
  __device__ __forceinline__ int init(const DecodeParams& p, int index, int ranges) {
    // A lane takes `per` consecutive sequences: independent loads and one scan.
    const int lane = threadIdx.x & 31, per = (p.B + 31) / 32, from_b = lane * per;
    int mine = 0;
#pragma unroll 4
    for (int i = 0; i < per; ++i)
      if (from_b + i < p.B) mine += item_tiles<KEYS>(seq_len(p, from_b + i));
    mine *= p.blocks;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(kFull, upto, d);
      if (lane >= d) upto += v;
    }
    const int total = __shfl_sync(kFull, upto, 31);
    const int share = range_tiles(p, total, ranges);
    const int64_t from = int64_t(share) * index;
    pos = int(min(from, int64_t(total)));
    end = int(min(from + share, int64_t(total)));
    if (pos >= end) return share;
    const int src = __ffs(__ballot_sync(kFull, upto > pos)) - 1;
    int in = pos - (upto - mine);             // tiles into the lane's sequences, where lane == src
    b = from_b;
    len = tiles = 0;
    if (lane == src) {
      for (;; ++b) {
        len = seq_len(p, b);
        tiles = item_tiles<KEYS>(len);
        if (in < tiles * p.blocks) break;
        in -= tiles * p.blocks;
      }
    }
    b = __shfl_sync(kFull, b, src);
    len = __shfl_sync(kFull, len, src);
    in = __shfl_sync(kFull, in, src);
    tiles = item_tiles<KEYS>(len);
    block = in / tiles;
    tile = first = in - block * tiles;
    return share;
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
          tiles = item_tiles<KEYS>(len);
        }
      }
    }
  }
  __device__ __forceinline__ int keys() const { return min(KEYS, len - tile * KEYS); }  // <= 0: none
  // Rows of the item's 64-row part `part` (0, or 0 and 1 for a pair); <= 0: none.
  __device__ __forceinline__ int rows(const DecodeParams& p, int part = 0) const {
    return min(kRows, p.rows - (block * p.ctas + part) * kRows);
  }
};

// Place of an item in the tile list and the tiles of a range, from the lengths
// alone: a whole warp of a joining kernel finds them while the ranges still run.
template <int KEYS>
__device__ __forceinline__ void find_item(const DecodeParams& p, int item, int& b, int& block, int& start, int& tiles,
                                          int& share) {
  b = item / p.blocks;
  block = item - b * p.blocks;
  int before = 0, total = 0;
  for (int i = threadIdx.x & 31; i < p.B; i += 32) {
    const int t = item_tiles<KEYS>(seq_len(p, i));
    total += t;
    if (i < b) before += t;
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    before += __shfl_xor_sync(kFull, before, d);
    total += __shfl_xor_sync(kFull, total, d);
  }
  tiles = item_tiles<KEYS>(seq_len(p, b));
  start = before * p.blocks + tiles * block;
  share = range_tiles(p, total * p.blocks, p.ranges);
}

__device__ __forceinline__ void prefetch_l2(uint32_t elected, const void* at, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q cp.async.bulk.prefetch.L2.global [%0], %1;\n\t}" ::"l"(at),
      "r"(bytes), "r"(elected)
      : "memory");
}

// 16-bit rows [rows, 576] in boxes of `box_rows` rows x `chunks` chunks of 64
// values, which land chunk by chunk, each as box_rows x 128 bytes.
template <typename T>
bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int box_rows, int chunks) {
  const int64_t dims[3] = {64, rows, kRow / 64}, strides[2] = {2 * kRow, 128};
  const int box[3] = {64, box_rows, chunks};
  return encode_map(m, Elem<T>::kMap, 3, base, dims, strides, box);
}

}  // namespace
}  // namespace nvfp4moe
