// Which block of the joining kernels takes a cut item (absorbed attention).
// Plain C++, so that it is tested without a GPU.
#pragma once

#ifdef __CUDACC__
#define NVFP4MLA_HD __host__ __device__ __forceinline__
#else
#define NVFP4MLA_HD inline
#endif

namespace nvfp4moe {

// Ranges take `share` tiles each, border c lies between ranges c and c + 1.
// The item (places start .. start + tiles - 1 of the tile list) is the one
// that range c + 1 begins with, tiles = 0 if there is none.  Block c joins it
// if border c is the first to cut it: an item that begins at the border is not
// cut there, and one that an earlier border cuts has its own block already.
NVFP4MLA_HD bool border_joins(int c, int start, int tiles, int share) {
  return tiles != 0 && start >= c * share && start < (c + 1) * share;
}

}  // namespace nvfp4moe
