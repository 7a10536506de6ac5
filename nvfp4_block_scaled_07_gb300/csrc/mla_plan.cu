// Block tables and slot maps of a step's new tokens (mla_plan).
//
// Request b has past[b] tokens in the cache and brings new[b].  It holds
// ceil(past / page) pages and needs ceil((past + new) / page); the missing ones
// are popped from the end of the free pages, requests in their order.  With
// the running sum of what the requests miss, the i-th missing page of request
// b is free[count - 1 - (sum before b + i)], so nothing waits for another
// request.
//
// One block scans the requests (tokens, then pages) in pieces of its threads,
// and writes the new table entries and, up to kOneBlock tokens, the tokens.
// More tokens are written by a second kernel over all SMs, which reads the
// tables.  Bound by latency: a decode step is one launch and two scans.
#include <climits>
#include <cstdint>

#include "../../include/nvfp4mla.h"
#include "internal.h"
#include "launch.cuh"
#include "sm103_ptx.cuh"

namespace nvfp4moe {
namespace {

__device__ unsigned g_plan_flags = 0;

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMaxThreads = 1024;
constexpr int kOneBlock = 8192;   // tokens

// Running sums over a block of x and, through the result of y_of(sum of x before), of y.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* shared, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t a = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(kFull, a, d);
    if (lane >= d) a += u;
  }
  if (lane == 31) shared[warp] = a;
  __syncthreads();
  int64_t w = lane < warps ? shared[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(kFull, w, d);
    if (lane >= d) w += u;
  }
  *total = __shfl_sync(kFull, w, 31);
  const int64_t before = warp ? __shfl_sync(kFull, w, warp - 1) : 0;
  __syncthreads();
  return before + a;                          // inclusive
}

// The first of n ascending values that is above x.
template <typename V>
__device__ __forceinline__ int first_above(const V* v, int n, V x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ void put_token(const MlaPlanArgs& p, int64_t t, int64_t position, int page_id) {
  p.positions[t] = int(position < INT_MAX ? position : INT_MAX);
  p.slots[t] = page_id < 0 ? -1 : (int64_t(page_id) << p.shift) + (position & ((int64_t(1) << p.shift) - 1));
}

__global__ void __launch_bounds__(kMaxThreads) plan_kernel(const MlaPlanArgs p, bool tokens_too) {
  __shared__ int64_t s_scan[32];
  __shared__ int64_t s_tokens[kMaxThreads], s_pages[kMaxThreads];  // running sums of this piece
  __shared__ int s_past[kMaxThreads], s_held[kMaxThreads];
  __shared__ bool s_ok[kMaxThreads];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int tid = threadIdx.x;
  int64_t count = *p.free_count;
  bool bad = count < 0 || count > p.num_free;
  count = count < 0 ? 0 : (count > p.num_free ? p.num_free : count);
  const int64_t page = int64_t(1) << p.shift;
  int64_t tokens = 0, pages = 0;              // of the pieces before; pages: asked for
  int64_t given = 0;
  if (tid == 0) p.cu_seqlens[0] = 0;
  for (int64_t b0 = 0; b0 < p.B; b0 += blockDim.x) {
    const int64_t b = b0 + tid;
    int64_t past = 0, fresh = 0;
    if (b < p.B) {
      past = p.past[b], fresh = p.fresh[b];
      bad |= past < 0 || fresh < 0;
      past = past < 0 ? 0 : past;
      fresh = fresh < 0 ? 0 : fresh;
    }
    int64_t piece_tokens, piece_pages;
    const int64_t upto = tokens + block_scan(fresh, s_scan, &piece_tokens);
    const int64_t held = (past + page - 1) >> p.shift, after = (past + fresh + page - 1) >> p.shift;
    const bool rows = upto <= p.T, fits = rows && after <= p.max_pages;
    bad |= !rows;
    const int64_t need = fits ? after - held : 0;
    const int64_t asked = block_scan(need, s_scan, &piece_pages);
    const bool ok = fits && (need == 0 || pages + asked <= count);
    s_tokens[tid] = upto, s_pages[tid] = asked;
    s_past[tid] = int(past), s_held[tid] = int(held);
    s_ok[tid] = ok && b < p.B;
    if (b < p.B) {
      p.cu_seqlens[b + 1] = int(upto < p.T ? upto : p.T);
      p.seq_lens[b] = int(ok ? past + fresh : past);
      p.granted[b] = int(ok ? fresh : 0);
    }
    // pages that this piece is given: those asked for while they last, whole requests only
    const int64_t left = count - pages;
    __syncthreads();
    const int n = int(p.B - b0 < blockDim.x ? p.B - b0 : blockDim.x);
    const int whole = first_above<int64_t>(s_pages, n, left);    // requests whose sum is within
    const int64_t here = whole > 0 ? s_pages[whole - 1] : 0;
    for (int64_t i = tid; i < here; i += blockDim.x) {
      const int r = first_above<int64_t>(s_pages, n, i);
      const int64_t before = r > 0 ? s_pages[r - 1] : 0;
      p.tables[(b0 + r) * p.table_stride + s_held[r] + (i - before)] = p.free_pages[count - 1 - (pages + i)];
    }
    if (tokens_too) {
      const int64_t end = tokens + piece_tokens < p.T ? tokens + piece_tokens : p.T;
      for (int64_t t = tokens + tid; t < end; t += blockDim.x) {
        const int r = first_above<int64_t>(s_tokens, n, t);
        const int64_t position = s_past[r] + t - (r > 0 ? s_tokens[r - 1] : tokens);
        int id = -1;
        if (s_ok[r]) {
          const int64_t at = position >> p.shift;
          id = at < s_held[r] ? p.tables[(b0 + r) * p.table_stride + at]
                              : p.free_pages[count - 1 - (pages + (r > 0 ? s_pages[r - 1] : 0) + at - s_held[r])];
        }
        put_token(p, t, position, id);
      }
    }
    given += here;
    tokens += piece_tokens;
    pages += piece_pages;
    __syncthreads();
  }
  if (tokens_too)
    for (int64_t t = (tokens < p.T ? tokens : p.T) + tid; t < p.T; t += blockDim.x) {
      p.positions[t] = 0;
      p.slots[t] = -1;
    }
  if (__syncthreads_or(bad) && tid == 0) atomicOr(&g_plan_flags, kFlagBadData);
  if (tid == 0) *p.free_count_out = int(count - given);
}

__global__ void __launch_bounds__(256) plan_tokens_kernel(const MlaPlanArgs p) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (t >= p.T) return;
  const int b = first_above<int32_t>(p.cu_seqlens + 1, p.B, int32_t(t));
  if (b == p.B) {
    p.positions[t] = 0;
    p.slots[t] = -1;
    return;
  }
  const int past = max(p.past[b], 0);
  const int64_t position = int64_t(past) + t - p.cu_seqlens[b];
  put_token(p, t, position, p.granted[b] > 0 ? p.tables[b * p.table_stride + (position >> p.shift)] : -1);
}

}  // namespace

cudaError_t launch_mla_plan(const MlaPlanArgs& a, cudaStream_t st) {
  const bool one = a.T <= kOneBlock;
  const int64_t most = one && a.T > a.B ? a.T : a.B;
  const int threads = most >= kMaxThreads ? kMaxThreads : int(most + 31) / 32 * 32;
  cudaError_t err = launch_kernel(plan_kernel, dim3(1), dim3(threads < 32 ? 32 : threads), 0, st, false, a, one);
  if (err != cudaSuccess || one) return err;
  return launch_kernel(plan_tokens_kernel, dim3(unsigned((a.T + 255) / 256)), dim3(256), 0, st, false, a);
}

cudaError_t mla_plan_flags_address(unsigned** at) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_plan_flags);
}

}  // namespace nvfp4moe
