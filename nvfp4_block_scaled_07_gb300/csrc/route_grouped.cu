// Routing to experts with a bias that only selects, groups of experts and a
// factor on the weights (moe_route_grouped).
//
//   s_e = sigma(v_e) or softmax(v)_e          c_e = s_e + b_e
//   value of a group = its largest c, or the sum of its two largest
//   the topk_group best groups; in them the k best c, the lower index first
//   w_j = factor * s_j, divided by the sum of the k chosen s on request
//
// The choice is that of exact scores: float32 scores of near experts round to
// one value, or change places.  A warp takes a token: it chooses by float32
// scores and their error bound d, and where two candidates that the choice
// depends on differ by no more than 2 d it chooses again in float64 (one token
// in a thousand for random logits).  Without a bias c orders like v, which
// needs no bound (unless groups are valued by sums).
//
// A lane holds consecutive experts, so that a group is whole lanes in the
// usual shapes and its value takes two shuffles.  The k rounds are warp maxima
// of integer keys that order like the floats; the lowest lane with the maximum
// has the lowest index.
#include <cfloat>
#include <climits>
#include <cstdint>

#include "../../include/nvfp4few.h"
#include "internal.h"
#include "launch.cuh"
#include "sm103_ptx.cuh"

namespace nvfp4moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kWarps = 8;

struct RouteParams {
  const float* logits;
  const float* bias;
  int T, E, k, groups, keep, best, softmax, renorm;
  float factor;
  int32_t* idx;
  float* w;
};

// Unsigned keys that order like floats; 0 stands for "not a candidate", below -inf's.
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (uint32_t(int(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// NaN counts as -inf (score 0), +inf as the largest number.
__device__ __forceinline__ float clean(float v) { return v != v ? -INFINITY : fminf(v, FLT_MAX); }

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

// ---- the choice in float64 ------------------------------------------------------
template <int VPL>
__device__ __noinline__ int choose_exactly(const RouteParams& p, int t, int lane) {
  const float* row = p.logits + int64_t(t) * p.E;
  const int per = p.E / p.groups;
  double c[VPL];
  float top = -INFINITY;
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    if (e < p.E) top = fmaxf(top, clean(row[e]));
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
  double sum = 0.0;
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    c[i] = -INFINITY;
    if (e >= p.E) continue;
    const double v = clean(row[e]);
    c[i] = p.softmax ? (v == -INFINITY ? 0.0 : exp(v - double(top))) : 1.0 / (1.0 + exp(-v));
    sum += c[i];
  }
  if (p.softmax) {
    sum = warp_sum(sum);
    if (sum == 0.0) sum = 1.0;
  }
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    if (e >= p.E) continue;
    if (p.softmax) c[i] /= sum;
    if (p.bias) c[i] += double(clean(p.bias[e]));
  }
  // the groups' values (lane g holds group g's) and ranks
  double mine = -INFINITY;
  for (int g = 0; g < p.groups && p.groups > 1; ++g) {
    double a = -INFINITY, b = -INFINITY;
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (e < p.E && e / per == g) {
        if (c[i] > a) b = a, a = c[i];
        else if (c[i] > b) b = c[i];
      }
    }
    for (int d = 16; d; d >>= 1) {
      const double oa = __shfl_xor_sync(kFull, a, d), ob = __shfl_xor_sync(kFull, b, d);
      b = fmax(fmin(a, oa), fmax(b, ob));
      a = fmax(a, oa);
    }
    if (lane == g) mine = p.best == 2 ? a + b : a;
  }
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const double other = __shfl_sync(kFull, mine, g);
    rank += other > mine || (other == mine && g < lane);
  }
  const uint32_t kept = __ballot_sync(kFull, lane < p.groups && rank < p.keep);
  uint32_t open = 0;                          // bit i: expert i of the lane can be chosen
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    if (e < p.E && ((kept >> (e / per)) & 1)) open |= 1u << i;
  }
  int my_e = 0;
  for (int j = 0; j < p.k; ++j) {
    double v = -INFINITY;
    int e = INT_MAX;
    for (int i = 0; i < VPL; ++i)
      if (((open >> i) & 1) && (e == INT_MAX || c[i] > v)) v = c[i], e = lane * VPL + i;
    for (int d = 16; d; d >>= 1) {
      const double ov = __shfl_xor_sync(kFull, v, d);
      const int oe = __shfl_xor_sync(kFull, e, d);
      if (oe != INT_MAX && (e == INT_MAX || ov > v || (ov == v && oe < e))) v = ov, e = oe;
    }
    if (e / VPL == lane) open &= ~(1u << (e % VPL));
    if (lane == j) my_e = e;
  }
  return my_e;
}

// ---- the choice in float32 --------------------------------------------------------
// A lane's experts are VPL consecutive ones.  WHOLE: a lane's are all of one
// group, and a group is a power of two of lanes.
template <int VPL, bool WHOLE>
__global__ void __launch_bounds__(32 * kWarps) route_grouped_kernel(const RouteParams p) {
  __shared__ float s_group[WHOLE ? 1 : kWarps][WHOLE ? 1 : 32 * VPL];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= p.T) return;
  const float* row = p.logits + int64_t(t) * p.E;
  const int e0 = lane * VPL, per = p.E / p.groups;
  float v[VPL], c[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) v[i] = e0 + i < p.E ? clean(row[e0 + i]) : -INFINITY;

  // scores
  float top = 0.0f, sum = 0.0f;               // softmax
  float error = 0.0f;                         // |c - exact c| of any expert
  const bool plain = !p.bias && (p.groups == 1 || p.best == 1);   // c orders like v
  if (p.softmax && !(plain && p.renorm)) {
    top = v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = fmaxf(top, v[i]);
    top = value_of(__reduce_max_sync(kFull, key_of(top)));
    if (top == -INFINITY) top = 0.0f;         // all masked: scores of 0
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      c[i] = expf(v[i] - top);
      sum += c[i];
    }
    sum = warp_sum(sum);
  }
  if (plain) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = v[i];
  } else {
    float most = 0.0f;                        // largest |c|, for its rounding
    if (p.softmax) {
      const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] *= inv;
      // exp(x), x = v - top rounded: (2 + |x| / 2) ulp, at most 2 ulp of 1 times exp(x); the
      // sum's and the quotient's 40 ulp; all times the largest score, inv
      error = inv * 0x1p-17f;
    } else {
      // __expf is within 2 + 1.2 |v| ulp, which moves s by at most 0.7 of an ulp of 1 as
      // s (1 - s) falls faster; the sum and the reciprocal take 2 ulp
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = ptx::rcp_approx(1.0f + __expf(-v[i]));
      error = 0x1p-21f;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (p.bias) c[i] += e0 + i < p.E ? clean(__ldg(p.bias + e0 + i)) : -INFINITY;
      if (c[i] > -INFINITY) most = fmaxf(most, fabsf(c[i]));
    }
    error += __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(most))) * 0x1p-23f;
  }
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = e0 + i < p.E ? key_of(c[i]) : 0u;

  bool sure = true;
  if (p.groups > 1) {
    float value;                              // of group g, in lane g (not WHOLE) or the group's lanes
    const int lanes = WHOLE ? per / VPL : 1;
    if (WHOLE) {
      float a = c[0], b = -INFINITY;
#pragma unroll
      for (int i = 1; i < VPL; ++i) {
        b = fmaxf(b, fminf(a, c[i]));
        a = fmaxf(a, c[i]);
      }
      for (int d = 1; d < lanes; d <<= 1) {
        const float oa = __shfl_xor_sync(kFull, a, d), ob = __shfl_xor_sync(kFull, b, d);
        b = fmaxf(fminf(a, oa), fmaxf(b, ob));
        a = fmaxf(a, oa);
      }
      value = p.best == 2 ? a + b : a;
    } else {
      float* sh = s_group[warp];
#pragma unroll
      for (int i = 0; i < VPL; ++i) sh[e0 + i] = c[i];
      __syncwarp();
      float a = -INFINITY, b = -INFINITY;
      for (int i = 0; i < per && lane < p.groups; ++i) {
        const float x = sh[lane * per + i];
        b = fmaxf(b, fminf(a, x));
        a = fmaxf(a, x);
      }
      value = p.best == 2 ? a + b : a;
    }
    // lane g: group g's value and rank
    const float mine = __shfl_sync(kFull, value, (lane * lanes) & 31);
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const float other = __shfl_sync(kFull, mine, g);
      rank += other > mine || (other == mine && g < lane);
    }
    const bool is_kept = lane < p.groups && rank < p.keep;
    const uint32_t kept = __ballot_sync(kFull, is_kept);
    if (!plain && p.keep < p.groups) {
      const float low = value_of(__reduce_min_sync(kFull, is_kept ? key_of(mine) : kFull));
      const float high = value_of(__reduce_max_sync(kFull, lane < p.groups && !is_kept ? key_of(mine) : 0u));
      // a sum of two rounds once more
      sure = low - high > 2.0f * (p.best * error + 0x1p-23f * fmaxf(fabsf(low), fabsf(high)));
    }
    if (WHOLE) {
      const bool in = (kept >> (lane / lanes)) & 1;
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = in ? key[i] : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (!((kept >> min((e0 + i) / per, 31)) & 1)) key[i] = 0u;
    }
  }

  // k rounds; the margin of the last is that to the best candidate left
  uint32_t local = key[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) local = max(local, key[i]);
  int my_e = 0;
  float before = INFINITY;
  auto margin = [&](uint32_t m) {             // to the candidate before
    const float now = value_of(m);
    sure = sure && (m == 0u || before - now > 2.0f * error);
    before = now;
  };
  for (int j = 0; j < p.k; ++j) {
    const uint32_t m = __reduce_max_sync(kFull, local);
    if (!plain) margin(m);
    const int from = __ffs(__ballot_sync(kFull, local == m)) - 1;
    int e = 0;
    if (lane == from) {
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i)
        if (key[i] == m) e = i;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == e) key[i] = 0u;
      local = key[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) local = max(local, key[i]);
      e += e0;
    }
    e = __shfl_sync(kFull, e, from);
    if (lane == j) my_e = e;
  }
  if (!plain) margin(__reduce_max_sync(kFull, local));
  if (!sure) my_e = choose_exactly<VPL>(p, t, lane);

  // weights of the chosen
  const bool mine = lane < p.k;
  float s = 0.0f;
  if (p.softmax) {
    const float x = mine ? clean(row[my_e]) : -INFINITY;
    if (p.renorm) {                           // the whole softmax's sum cancels
      top = value_of(__reduce_max_sync(kFull, key_of(x)));
      if (top == -INFINITY) top = 0.0f;
    }
    // x - top exactly, as its rounding and what that lost
    const float d = x - top, back = d - x, lost = (x - (d - back)) + (-top - back);
    s = mine && d > -200.0f ? expf(d) * (1.0f + lost) : 0.0f;
    if (!p.renorm) s = sum > 0.0f ? s / sum : 0.0f;
  } else if (mine) {
    s = 1.0f / (1.0f + expf(-clean(row[my_e])));
  }
  if (p.renorm) {
    const float all = warp_sum(s);
    s = all > 0.0f ? s / all : 0.0f;
  }
  if (mine) {
    p.idx[int64_t(t) * p.k + lane] = my_e;
    p.w[int64_t(t) * p.k + lane] = s * p.factor;
  }
}

template <int VPL>
cudaError_t launch_vpl(const RouteParams& p, cudaStream_t st) {
  const int per = p.E / p.groups, lanes = per / VPL;
  const bool whole = p.E == 32 * VPL && per % VPL == 0 && (lanes & (lanes - 1)) == 0;
  return launch_kernel(whole ? route_grouped_kernel<VPL, true> : route_grouped_kernel<VPL, false>,
                       dim3(unsigned((p.T + kWarps - 1) / kWarps)), dim3(32 * kWarps), 0, st, false, p);
}

}  // namespace

cudaError_t launch_route_grouped(const float* logits, const float* bias, int T, int E, int k, int groups, int keep, int best,
                                 int softmax, int renorm, float factor, int32_t* idx, float* w, cudaStream_t st) {
  const RouteParams p = {logits, bias, T, E, k, groups, keep, best, softmax, renorm, factor, idx, w};
  if (E <= 32) return launch_vpl<1>(p, st);
  if (E <= 64) return launch_vpl<2>(p, st);
  if (E <= 128) return launch_vpl<4>(p, st);
  if (E <= 256) return launch_vpl<8>(p, st);
  if (E <= 512) return launch_vpl<16>(p, st);
  return launch_vpl<32>(p, st);
}

}  // namespace nvfp4moe
