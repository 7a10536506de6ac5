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
// and writes the new table entries and a few tokens.  More tokens are written by a second kernel over all SMs, which reads the
// tables.  Bound by latency: a decode step is one launch and two scans.  One
// request of one token takes 2.5 us, 700 of three 4.8 us, 37 of 7000 8.6 us.
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
// The one block writes up to kOneBlock tokens, and up to kFew a request on average, which the scanning threads write as
// they go.  Measured (us with one kernel, with two): 8 requests of 1024 tokens together 6.4, 6.3, of 8192 9.8, 6.4, of
// 65536 41, 6.8; 300 requests of 4096 9.8, 8.7; 700 requests of three each 4.8, 11.1; 10000 of one 24, 59.
constexpr int kOneBlock = 1024;
constexpr int kFew = 8;           // new tokens of a request: at most two pages
constexpr int kSmall = 1 << 20;   // up to so many rows and free pages, a piece's two sums fit one 64-bit scan
constexpr int kTokensPerBlock = 1024;

// Inclusive sums over a block, and their total.
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
  return before + a;
}

// Of N values x: how many of n ascending values are not above each (the first
// that is above).  Side by side, so that their loads are in flight together.
template <int N, typename V>
__device__ __forceinline__ void first_above(const V* v, int n, const V (&x)[N], int (&at)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) at[i] = 0;
  for (int step = n > 0 ? 1 << (31 - __clz(n)) : 0; step; step >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at[i] + step <= n && v[at[i] + step - 1] <= x[i]) at[i] += step;
}

// Stores row t: a token's position and slot (page id < 0: none).
__device__ __forceinline__ void put_token(const MlaPlanArgs& p, int64_t t, int64_t position, int page_id) {
  p.positions[t] = int(position < INT_MAX ? position : INT_MAX);
  p.slots[t] = page_id < 0 ? -1 : (int64_t(page_id) << p.shift) + (position & ((int64_t(1) << p.shift) - 1));
}

__global__ void __launch_bounds__(kMaxThreads) plan_kernel(const MlaPlanArgs p, bool tokens_too) {
  __shared__ int64_t s_scan[32];
  __shared__ int64_t s_tokens[kMaxThreads], s_pages[kMaxThreads];  // running sums of this piece
  __shared__ int s_past[kMaxThreads], s_held[kMaxThreads];
  __shared__ bool s_ok[kMaxThreads];
  __shared__ int s_given;
  constexpr int kAtOnce = 4;                  // tokens or pages of a thread
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int tid = threadIdx.x, threads = blockDim.x;
  int64_t count = *p.free_count;
  bool bad = count < 0 || count > p.num_free;
  count = count < 0 ? 0 : (count > p.num_free ? p.num_free : count);
  const int64_t page = int64_t(1) << p.shift;
  int64_t tokens = 0, pages = 0;              // of the pieces before; pages: asked for
  int64_t given = 0;
  if (tid == 0) p.cu_seqlens[0] = 0, s_given = 0;
  for (int64_t b0 = 0; b0 < p.B; b0 += threads) {
    const int64_t b = b0 + tid;
    int64_t past = 0, fresh = 0;
    if (b < p.B) {
      past = p.past[b], fresh = p.fresh[b];
      bad |= past < 0 || fresh < 0;
      past = past < 0 ? 0 : past;
      fresh = fresh < 0 ? 0 : fresh;
    }
    const int64_t held = (past + page - 1) >> p.shift, after = (past + fresh + page - 1) >> p.shift;
    const bool short_table = after > p.max_pages || past + fresh > INT_MAX;    // a length has 31 bits
    int64_t need = short_table ? 0 : after - held;
    int64_t piece_tokens, piece_pages, upto, asked;
    bool rows = true;                         // the request's tokens have rows
    bool again = true;
    if (p.T <= kSmall && p.num_free <= kSmall) {
      // what is more than all rows or pages is more than all of them
      const int64_t f = min(fresh, int64_t(p.T) + 1), n = min(need, int64_t(p.num_free) + 1);
      int64_t total;
      const int64_t both = block_scan(n << 32 | f, s_scan, &total);
      piece_tokens = total & 0xFFFFFFFF, piece_pages = total >> 32;
      upto = tokens + (both & 0xFFFFFFFF), asked = both >> 32;
      again = tokens + piece_tokens > p.T;
    }
    if (again) {                              // tokens first: those without rows ask for no page
      upto = tokens + block_scan(fresh, s_scan, &piece_tokens);
      rows = upto <= p.T;
      bad |= !rows;
      if (!rows) need = 0;
      asked = block_scan(need, s_scan, &piece_pages);
    }
    const bool ok = rows && !short_table && (need == 0 || pages + asked <= count);
    if (b < p.B) {
      p.cu_seqlens[b + 1] = int(upto < p.T ? upto : p.T);
      p.seq_lens[b] = int(ok ? past + fresh : past);
      p.granted[b] = int(ok ? fresh : 0);
    }
    if (tokens_too && !__syncthreads_or(fresh > kFew)) {
      // a few tokens each: every request's thread writes its own
      const int64_t popped = pages + asked - need;                       // before its first new page
      if (ok)
        for (int i = 0; i < int(need); ++i)
          p.tables[b * p.table_stride + held + i] = p.free_pages[count - 1 - (popped + i)];
      for (int i = 0; i < int(fresh); ++i) {
        const int64_t t = upto - fresh + i, at = (past + i) >> p.shift;
        if (t >= p.T) break;
        put_token(p, t, past + i,
                  !ok ? -1 : at < held ? p.tables[b * p.table_stride + at] : p.free_pages[count - 1 - (popped + at - held)]);
      }
      const int mine = __reduce_add_sync(kFull, ok ? int(need) : 0);
      if ((tid & 31) == 0 && mine) atomicAdd(&s_given, mine);
      tokens += piece_tokens;
      pages += piece_pages;
      continue;
    }
    s_tokens[tid] = upto, s_pages[tid] = asked;
    s_past[tid] = int(past), s_held[tid] = int(held);
    s_ok[tid] = ok && b < p.B;
    __syncthreads();
    // pages that this piece is given: those asked for while they last, whole requests only
    const int n = int(p.B - b0 < threads ? p.B - b0 : threads);
    const int64_t left[1] = {count - pages};
    int whole[1];
    first_above(s_pages, n, left, whole);
    const int64_t here = whole[0] > 0 ? s_pages[whole[0] - 1] : 0;
    for (int64_t i0 = tid; i0 < here; i0 += kAtOnce * threads) {
      int64_t i[kAtOnce];
      int r[kAtOnce], id[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        i[j] = i0 + j * threads;
        id[j] = i[j] < here ? p.free_pages[count - 1 - (pages + i[j])] : 0;
      }
      first_above(s_pages, n, i, r);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (i[j] < here)
          p.tables[(b0 + r[j]) * p.table_stride + s_held[r[j]] + (i[j] - (r[j] > 0 ? s_pages[r[j] - 1] : 0))] = id[j];
    }
    if (tokens_too) {
      const int64_t end = tokens + piece_tokens < p.T ? tokens + piece_tokens : p.T;
      for (int64_t t0 = tokens + tid; t0 < end; t0 += kAtOnce * threads) {
        int64_t t[kAtOnce], position[kAtOnce];
        int r[kAtOnce], id[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) t[j] = min(t0 + j * threads, end - 1);
        first_above(s_tokens, n, t, r);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int before = r[j] - 1;
          position[j] = s_past[r[j]] + t[j] - (r[j] > 0 ? s_tokens[before] : tokens);
          id[j] = -1;
          if (s_ok[r[j]]) {                   // an old page by the table, a new one as it is popped
            const int64_t at = position[j] >> p.shift;
            id[j] = at < s_held[r[j]]
                        ? p.tables[(b0 + r[j]) * p.table_stride + at]
                        : p.free_pages[count - 1 - (pages + (r[j] > 0 ? s_pages[before] : 0) + at - s_held[r[j]])];
          }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
          if (t0 + j * threads < end) put_token(p, t[j], position[j], id[j]);
      }
    }
    given += here;
    tokens += piece_tokens;
    pages += piece_pages;
    __syncthreads();
  }
  if (tokens_too)
    for (int64_t t = (tokens < p.T ? tokens : p.T) + tid; t < p.T; t += threads) {
      p.positions[t] = 0;
      p.slots[t] = -1;
    }
  if (__syncthreads_or(bad) && tid == 0) atomicOr(&g_plan_flags, kFlagBadData);
  if (tid == 0) *p.free_count_out = int(count - given - s_given);
}

// Rows of kTokensPerBlock tokens: the first one's request by counting the
// offsets that are not above it, the others among the next requests.
__global__ void __launch_bounds__(256) plan_tokens_kernel(const MlaPlanArgs p) {
  constexpr int kAtOnce = kTokensPerBlock / 256;
  __shared__ int s_cu[257];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int tid = threadIdx.x;
  const int64_t t0 = int64_t(blockIdx.x) * kTokensPerBlock;
  int first = 0;                              // requests that end at or before t0
  for (int64_t b = 0; b < p.B; b += 256) {
    const int here = __syncthreads_count(b + tid < p.B && p.cu_seqlens[b + tid + 1] <= t0);
    first += here;
    if (here < 256) break;                    // ascending: the next end later
  }
  const int n = min(256, p.B - first);        // and the requests that follow
  if (tid < n) s_cu[tid] = p.cu_seqlens[first + tid + 1];
  __syncthreads();
  int t[kAtOnce], r[kAtOnce], id[kAtOnce];
  int64_t position[kAtOnce];
#pragma unroll
  for (int j = 0; j < kAtOnce; ++j) t[j] = int(min(t0 + j * 256 + tid, int64_t(p.T) - 1));
  first_above(s_cu, n, t, r);
#pragma unroll
  for (int j = 0; j < kAtOnce; ++j) {
    int b = first + r[j];
    if (r[j] == n && b < p.B) {               // more than 256 requests in these rows
      const int x[1] = {t[j]};
      int at[1];
      first_above(p.cu_seqlens + 1, p.B, x, at);
      b = at[0];
    }
    position[j] = 0, id[j] = -1;
    if (b < p.B) {
      const int granted = p.granted[b];       // seq_lens - granted: the tokens before; past_lens may be seq_lens itself
      position[j] = int64_t(p.seq_lens[b]) - granted + t[j] - p.cu_seqlens[b];
      if (granted > 0) id[j] = p.tables[b * p.table_stride + (position[j] >> p.shift)];
    }
  }
#pragma unroll
  for (int j = 0; j < kAtOnce; ++j)
    if (t0 + j * 256 + tid < p.T) put_token(p, t[j], position[j], id[j]);
}

}  // namespace

cudaError_t launch_mla_plan(const MlaPlanArgs& a, cudaStream_t st) {
  const bool one = a.T <= kOneBlock || a.T <= int64_t(kFew) * a.B;
  const int64_t most = one && a.T < kMaxThreads ? (a.T > a.B ? a.T : a.B) : kMaxThreads;   // pages of many tokens as well
  const int threads = most >= kMaxThreads ? kMaxThreads : most < 32 ? 32 : int(most + 31) / 32 * 32;
  const cudaError_t err = launch_kernel(plan_kernel, dim3(1), dim3(threads), 0, st, false, a, one);
  if (err != cudaSuccess || one) return err;
  return launch_kernel(plan_tokens_kernel, dim3(unsigned((int64_t(a.T) + kTokensPerBlock - 1) / kTokensPerBlock)), dim3(256), 0,
                       st, false, a);
}

cudaError_t mla_plan_flags_address(unsigned** at) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_plan_flags);
}

}  // namespace nvfp4moe
