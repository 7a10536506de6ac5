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
// in a thousand for random logits), of the candidates at the border only.  Without a bias c orders like v, which
// needs no bound (unless groups are valued by sums).
//
// A lane holds consecutive experts, so that a group is whole lanes in the
// usual shapes and its value takes two shuffles.  The k rounds are warp maxima
// of integer keys that order like the floats; the lowest lane with the maximum
// has the lowest index.
//
// Bound by the instructions that it spends on a token (issue slots 74 % busy, DRAM
// 10 %): 16384 tokens of 256 experts take 21 us in 8 groups of which 4 are kept, 16.6
// us without groups, 24 us with one group masked by its biases, one token 3.3 us.
// Choosing all groups again in float64 where two were close took 31 us for the
// 16384, and one bound for all groups, the widest, 299 us beside a masked one.
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
  int wide;                                   // rows of logits, and the bias, start on 16-byte boundaries
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

// NaN counts as -inf (score 0), +inf as the largest number; the sum makes +0 of -0,
// which are equal as values but not as keys.
__device__ __forceinline__ float clean(float v) { return v != v ? -INFINITY : fminf(v, FLT_MAX) + 0.0f; }

// VPL values from e0 on, -inf past the E-th.
template <int VPL>
__device__ __forceinline__ void load(float (&v)[VPL], const float* from, int e0, int E, bool wide) {
  if (VPL >= 4 && wide && e0 + VPL <= E) {
#pragma unroll
    for (int i = 0; i + 3 < VPL; i += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(from + e0 + i));
      v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = e0 + i < E ? __ldg(from + e0 + i) : -INFINITY;
  }
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

// Whether all of a token's logits are equal, and the biases too (a padded token's, often): then the order is that of indexes.
__device__ __noinline__ bool all_alike(const RouteParams& p, const float* row, int lane) {
  bool same = true;
  for (int e = lane; e < p.E; e += 32)
    same = same && clean(row[e]) == clean(row[0]) && (!p.bias || clean(p.bias[e]) == clean(p.bias[0]));
  return __all_sync(kFull, same);
}

// ---- the choice in float64 ------------------------------------------------------
// Keys that order like doubles, compared as integers.
__device__ __forceinline__ uint64_t key_of(double d) {
  const uint64_t u = uint64_t(__double_as_longlong(d));
  return u ^ (uint64_t(int64_t(u) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double value_of(uint64_t key) {
  return __longlong_as_double(int64_t(key & 0x8000000000000000ull ? key ^ 0x8000000000000000ull : ~key));
}
// The sum of a token's softmax relative to its largest logit `top` (a warp).
template <int VPL>
__device__ __noinline__ double softmax_sum(const float* row, int E, float top, int lane) {
  double sum = 0.0;
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    const float v = e < E ? clean(row[e]) : -INFINITY;
    if (v > -INFINITY) sum += exp(double(v) - double(top));
  }
  return warp_sum(sum);
}
__device__ __noinline__ double exact_score(const RouteParams& p, const float* row, int e, float top, double sum) {
  const double v = clean(row[e]);
  double c;
  if (p.softmax) c = v == -INFINITY ? 0.0 : exp(v - double(top)) / sum;
  else c = 1.0 / (1.0 + exp(-v));
  return p.bias ? c + double(clean(p.bias[e])) : c;
}

// All of it: the groups' values, the groups, the experts.  Lane j < k returns the j-th.
template <int VPL>
__device__ __noinline__ int choose_exactly(const RouteParams& p, int t, float top, int lane) {
  const float* row = p.logits + int64_t(t) * p.E;
  const int per = p.E / p.groups;
  const double sum = p.softmax ? softmax_sum<VPL>(row, p.E, top, lane) : 0.0;
  uint64_t key[VPL];                          // 0: no candidate
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    key[i] = e < p.E ? key_of(exact_score(p, row, e, top, sum)) : 0;
  }
  auto better = [](uint64_t& x, int& e, uint64_t y, int f) {  // of two candidates, the lower index first
    if (y > x || (y == x && f < e)) x = y, e = f;
  };
  if (p.groups > 1) {
    int of[VPL];
    for (int i = 0; i < VPL; ++i) of[i] = (lane * VPL + i) / per;
    double mine = -INFINITY;                  // lane g: group g's value
    for (int g = 0; g < p.groups; ++g) {
      uint64_t best = 0, second = 0;
      int e1 = INT_MAX, e2 = INT_MAX;
      for (int i = 0; i < VPL; ++i)
        if (key[i] && of[i] == g) better(best, e1, key[i], lane * VPL + i);
      for (int d = 16; d; d >>= 1) better(best, e1, __shfl_xor_sync(kFull, best, d), __shfl_xor_sync(kFull, e1, d));
      if (p.best == 2) {
        for (int i = 0; i < VPL; ++i)
          if (key[i] && of[i] == g && lane * VPL + i != e1) better(second, e2, key[i], lane * VPL + i);
        for (int d = 16; d; d >>= 1) better(second, e2, __shfl_xor_sync(kFull, second, d), __shfl_xor_sync(kFull, e2, d));
      }
      if (lane == g) mine = p.best == 2 ? value_of(best) + value_of(second) : value_of(best);
    }
    const uint64_t value = lane < p.groups ? key_of(mine) : 0;
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const uint64_t other = __shfl_sync(kFull, value, g);
      rank += other > value || (other == value && g < lane);
    }
    const uint32_t kept = __ballot_sync(kFull, lane < p.groups && rank < p.keep);
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (e < p.E && !((kept >> of[i]) & 1)) key[i] = 0;
    }
  }
  int my_e = 0;
  for (int j = 0; j < p.k; ++j) {
    uint64_t best = 0;
    int e = INT_MAX;
    for (int i = 0; i < VPL; ++i)
      if (key[i]) better(best, e, key[i], lane * VPL + i);
    for (int d = 16; d; d >>= 1) better(best, e, __shfl_xor_sync(kFull, best, d), __shfl_xor_sync(kFull, e, d));
    for (int i = 0; i < VPL; ++i)
      if (lane * VPL + i == e) key[i] = 0;
    if (lane == j) my_e = e;
  }
  return my_e;
}

// Of `count` groups, the j-th's value that of experts e of lanes 2 j and 2 j + 1: bit 2 j, whether it is among the `places` best.
template <int VPL>
__device__ __noinline__ uint32_t among_near(const RouteParams& p, int t, float top, int lane, int e, int count, int places) {
  const float* row = p.logits + int64_t(t) * p.E;
  const double sum = p.softmax ? softmax_sum<VPL>(row, p.E, top, lane) : 0.0;
  double v = exact_score(p, row, e, top, sum);
  if (p.best == 2) v += __shfl_xor_sync(kFull, v, 1);
  const uint64_t value = key_of(v);
  int rank = 0;
  for (int j = 0; j < count; ++j) {
    const uint64_t other = __shfl_sync(kFull, value, 2 * j);
    rank += other > value || (other == value && 2 * j < lane);
  }
  return __ballot_sync(kFull, rank < places);
}

// Among at most 32 candidates, in ascending order in `from`: the k best.
template <int VPL>
__device__ __noinline__ int choose_among(const RouteParams& p, int t, float top, int lane, int n, int* from) {
  const float* row = p.logits + int64_t(t) * p.E;
  const double sum = p.softmax ? softmax_sum<VPL>(row, p.E, top, lane) : 0.0;
  const int e = lane < n ? from[lane] : 0;
  const uint64_t key = lane < n ? key_of(exact_score(p, row, e, top, sum)) : 0;
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const uint64_t other = __shfl_sync(kFull, key, i);
    rank += other > key || (other == key && i < lane);
  }
  __syncwarp();
  if (lane < n && rank < p.k) from[rank] = e;
  __syncwarp();
  return lane < p.k ? from[lane] : 0;
}

// ---- the weights ------------------------------------------------------------------
// x - top exactly, as its rounding and what that lost.
struct Shifted {
  float v, lost;
};
__device__ __forceinline__ Shifted shifted(float x, float top) {
  const float d = x - top, back = d - x;
  return {d, d > -INFINITY ? (x - (d - back)) + (-top - back) : 0.0f};
}

constexpr float kFar = -80.0f;                // below, exp(x) nears the end of float32's normal numbers
// The factor is below e^70: e^-200 of anything is no float32 with it.
constexpr float kFarthest = 200.0f;
constexpr float kNoSigmoid = -709.78f;        // below, exp(-x) is no float64: a score of 0

// A token's weights where scores leave float32's normal numbers, of a warp whose lane j holds the j-th chosen logit x
// (-inf: none).  Scores are taken relative to e^ref, and one below e^-80 of that as a number with the factor e^-72, so
// that neither the sum nor what a large factor brings back is lost.
__device__ __noinline__ float far_weight(const RouteParams& p, float x, float top, float sum) {
  float ref = top;
  if (!p.softmax) {
    if (x < kNoSigmoid) x = -INFINITY;
    ref = 0.0f;
    if (p.renorm) {                           // e^x / (1 + e^x): e^ref cancels
      ref = fminf(value_of(__reduce_max_sync(kFull, key_of(x))), 0.0f);
      if (ref == -INFINITY) ref = 0.0f;
    }
  }
  const Shifted d = shifted(x, ref);
  const float v = fminf(d.v, 0.0f);
  const bool small = v < kFar;
  float s = v > -kFarthest ? expf(small ? v + 72.0f : v) * (1.0f + d.lost) : 0.0f;   // v + 72 is exact
  const float unit = small ? 5.3801861e-32f : 1.0f;                                  // e^-72
  if (!p.softmax) s /= 1.0f + expf(-fabsf(x));
  float f = p.factor;
  if (p.renorm) {
    const float all = warp_sum(s * unit);     // at least 1/2 if there is any
    f = all > 0.0f ? f / all : 0.0f;
  } else if (p.softmax) {
    f = sum > 0.0f ? f / sum : 0.0f;          // the sum is at least 1
  }
  return f * s * unit;
}

// ---- the choice in float32 --------------------------------------------------------
// A lane's experts are VPL consecutive ones.  WHOLE: a lane's are all of one
// group, and a group is a power of two of lanes.
template <int VPL, bool WHOLE>
__global__ void __launch_bounds__(32 * kWarps, VPL <= 8 ? 5 : 1) route_grouped_kernel(const RouteParams p) {
  __shared__ float s_group[WHOLE ? 1 : kWarps][WHOLE ? 1 : 32 * VPL];
  __shared__ __align__(16) uint32_t s_key[kWarps][32];
  __shared__ uint32_t s_sorted[kWarps][36];
  __shared__ int s_expert[kWarps][32];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned row_of = blockIdx.x * kWarps + warp;   // up to 2^31 + 6
  if (row_of >= unsigned(p.T)) return;
  const int t = int(row_of);
  const float* row = p.logits + int64_t(t) * p.E;
  const int e0 = lane * VPL, per = p.E / p.groups;
  float v[VPL], c[VPL];
  load<VPL>(v, row, e0, p.E, p.wide);

  // scores
  float top = 0.0f, sum = 0.0f;               // softmax
  // |c - exact c| is at most error + 2^-24 |c|, the rounding of a sum with the bias
  float error = 0.0f;
  const bool plain = !p.bias && (p.groups == 1 || p.best == 1);   // c orders like v
  if (plain || p.softmax) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = clean(v[i]);
  }
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
      for (int i = 0; i < VPL; ++i) c[i] = fmaxf(ptx::rcp_approx(1.0f + __expf(-v[i])), 0.0f);  // NaN: 0
      error = 0x1p-21f;
    }
    if (p.bias) {
      float b[VPL];
      load<VPL>(b, p.bias, e0, p.E, p.wide);
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = fminf(fmaxf(c[i] + b[i], -INFINITY), FLT_MAX);   // as of a clean bias
    }
  }
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = e0 + i < p.E ? key_of(c[i]) : 0u;
  uint32_t local = key[0];                    // the lane's largest
#pragma unroll
  for (int i = 1; i < VPL; ++i) local = max(local, key[i]);

  // Whether two keys in descending order (0: none) are those of experts in that order.  -inf is exact (a masked expert).
  auto clear = [&](uint32_t before, uint32_t after) {
    const float x = value_of(before), y = value_of(after);
    return after == 0u || y == -INFINITY || x - y > 2.0f * error + 0x1p-22f * fmaxf(fabsf(x), fabsf(y));
  };

  bool alike = false, sure = true, open = true;              // open (WHOLE): the lane's group is kept
  if (p.groups > 1) {
    // of group g, in lane g (not WHOLE) or the group's lanes; and what it is off by: its parts' errors, their
    // rounding, its own and that of its bounds.  Sums of two as halves: biases of the type's lowest and largest value do not leave float32's range.
    float value, off;
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
      value = p.best == 2 ? 0.5f * a + 0.5f * b : a;
      off = error + 0x1.8p-23f * (p.best == 2 ? 0.5f * fabsf(a) + 0.5f * fabsf(b) : fabsf(a));
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
      value = p.best == 2 ? 0.5f * a + 0.5f * b : a;
      off = error + 0x1.8p-23f * (p.best == 2 ? 0.5f * fabsf(a) + 0.5f * fabsf(b) : fabsf(a));
    }
    // lane g: group g's value and rank
    const float mine = __shfl_sync(kFull, value, (lane * lanes) & 31);
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const float other = __shfl_sync(kFull, mine, g);
      rank += other > mine || (other == mine && g < lane);
    }
    bool is_kept = lane < p.groups && rank < p.keep;
    if (!plain && p.keep < p.groups) {
      // -inf is exact (a masked expert), and a tie of two goes by their indexes, as the ranks do
      off = __shfl_sync(kFull, off, (lane * lanes) & 31);
      const bool masked = mine == -INFINITY;
      const float least = masked ? mine : mine - off, most = masked ? mine : mine + off;
      const float low = value_of(__reduce_min_sync(kFull, is_kept ? key_of(least) : kFull));
      const float high = value_of(__reduce_max_sync(kFull, lane < p.groups && !is_kept ? key_of(most) : 0u));
      if (low <= high && high > -INFINITY && !(alike = all_alike(p, row, lane))) {
        // Exact values of those that the order of float32 values leaves open, for the places
        // that the others do not take: lanes 2 j and 2 j + 1 take the j-th one's two experts.
        const uint32_t near = __ballot_sync(kFull, lane < p.groups && (is_kept ? least <= high : !masked && most >= low));
        const int places = __popc(__ballot_sync(kFull, is_kept) & near), count = __popc(near);
        sure = count <= 16;
        int e = 0;
        if (sure) {
          int j = 0;
#pragma unroll 1
          for (uint32_t rest = near; rest; rest &= rest - 1, ++j) {
            const int g = __ffs(rest) - 1;
            uint32_t used = 0, last = 0, m = 0;
#pragma unroll 1
            for (int n = 0; n <= p.best; ++n) {
              uint32_t largest = 0;
              int at = 0;
#pragma unroll
              for (int i = VPL - 1; i >= 0; --i)
                if (key[i] >= max(largest, 1u) && !((used >> i) & 1) && (WHOLE ? lane / lanes : (e0 + i) / per) == g)
                  largest = key[i], at = i;
              last = m;
              m = __reduce_max_sync(kFull, largest);
              const int from = __ffs(__ballot_sync(kFull, largest == m)) - 1;
              const int expert = __shfl_sync(kFull, e0 + at, from);
              if (lane == from) used |= 1u << at;
              if (n < p.best && lane == 2 * j + n) e = expert;
            }
            // and whether float32 tells which experts they are
            sure = sure && clear(last, m);
          }
        }
        if (sure) {
          const uint32_t in = among_near<VPL>(p, t, top, lane, e, count, places);
          const int j = __popc(near & ((1u << lane) - 1));
          if ((near >> lane) & 1) is_kept = (in >> (2 * j)) & 1;
        }
      }
    }
    const uint32_t kept = __ballot_sync(kFull, is_kept);
    if (WHOLE) {
      open = (kept >> (lane / lanes)) & 1;
      if (!open) local = 0u;
    } else {
      local = 0u;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (!((kept >> min((e0 + i) / per, 31)) & 1)) key[i] = 0u;
        local = max(local, key[i]);
      }
    }
  }

  const bool groups_sure = sure;

  // Candidates: keys not below the (k + 1)-th largest of the lanes' largest, the
  // k + 1 best among them, a dozen or so.  Each goes to a lane of its own, in the order
  // of experts, and counts those before it.
  uint32_t bound = 0;
  for (uint32_t j = 0, rest = local; j <= uint32_t(p.k); ++j) {
    bound = __reduce_max_sync(kFull, rest);
    if (rest == bound) rest = 0u;             // of equal lanes all: only lowers the bound
  }
  bound = max(bound, 1u);
  uint32_t in = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) in |= uint32_t(key[i] >= bound) << i;
  if (!open) in = 0;
  int n = __popc(in), at = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(kFull, at, d);
    if (lane >= d) at += u;
  }
  const int candidates = __shfl_sync(kFull, at, 31);
  int my_e = 0;
  float last = 0.0f;                          // the k-th best
  if (candidates > 32 && !alike) alike = all_alike(p, row, lane);
  if (alike) {
    my_e = lane;
  } else if (candidates <= 32) {
    s_key[warp][lane] = 0u;
    if (lane < 4) s_sorted[warp][32 + lane] = 0u;
    s_sorted[warp][lane] = 0u;
    __syncwarp();
    at -= n;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if ((in >> i) & 1) {
        s_key[warp][at] = key[i];
        s_expert[warp][at++] = e0 + i;
      }
    __syncwarp();
    const uint32_t mine = s_key[warp][lane];
    const int e = s_expert[warp][lane];
    int rank = 0;                             // equal ones: the lower index, which is the lower lane
    for (int i = 0; i < candidates; i += 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(&s_key[warp][i]);
      rank += (q.x + (i < lane) > mine) + (q.y + (i + 1 < lane) > mine) + (q.z + (i + 2 < lane) > mine) +
              (q.w + (i + 3 < lane) > mine);
    }
    __syncwarp();
    if (lane < candidates) {
      s_sorted[warp][rank] = mine;
      s_expert[warp][rank] = e;
    }
    __syncwarp();
    my_e = s_expert[warp][lane];
    const uint32_t here = s_sorted[warp][lane], next = s_sorted[warp][lane + 1];
    last = value_of(__shfl_sync(kFull, here, p.k - 1));
    if (!plain) sure = sure && __all_sync(kFull, lane >= p.k || clear(here, next));
  } else {
    // many equal or hardly any lanes: k rounds of the warp's maximum
    uint32_t left[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) left[i] = open ? key[i] : 0u;
    uint32_t before = 0u;
    for (int j = 0; j < p.k; ++j) {
      const uint32_t m = __reduce_max_sync(kFull, local);
      if (!plain && j > 0) sure = sure && clear(before, m);
      before = m;
      const int from = __ffs(__ballot_sync(kFull, local == m)) - 1;
      int e = 0;
      if (lane == from) {
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
          if (left[i] == m) e = i;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (i == e) left[i] = 0u;
        local = left[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) local = max(local, left[i]);
        e += e0;
      }
      e = __shfl_sync(kFull, e, from);
      if (lane == j) my_e = e;
    }
    last = value_of(before);
    if (!plain) sure = sure && clear(before, __reduce_max_sync(kFull, local));
  }
  if (!sure) {
    // the exact k best are within 2 d of the k-th here
    const float least = last - 2.0f * error - 0x1p-21f * fabsf(last);
    in = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) in |= uint32_t(open && key[i] != 0u && c[i] >= least) << i;
    n = at = __popc(in);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(kFull, at, d);
      if (lane >= d) at += u;
    }
    const int near = __shfl_sync(kFull, at, 31);
    if (groups_sure && near <= 32) {
      at -= n;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if ((in >> i) & 1) s_expert[warp][at++] = e0 + i;
      __syncwarp();
      my_e = choose_among<VPL>(p, t, top, lane, near, s_expert[warp]);
    } else {
      my_e = choose_exactly<VPL>(p, t, top, lane);
    }
  }

  // weights of the chosen
  const bool mine = lane < p.k;
  const float x = mine ? clean(row[my_e]) : -INFINITY;
  float s = 0.0f;
  bool far;
  if (p.softmax) {
    if (p.renorm) {                           // the whole softmax's sum cancels
      top = value_of(__reduce_max_sync(kFull, key_of(x)));
      if (top == -INFINITY) top = 0.0f;
    }
    const Shifted d = shifted(x, top);
    far = d.v < kFar && d.v > -kFarthest;
    s = mine ? expf(d.v) * (1.0f + d.lost) : 0.0f;
    if (!p.renorm) s = sum > 0.0f ? s / sum : 0.0f;
  } else {
    far = x < kFar && x >= kNoSigmoid;
    if (mine) s = 1.0f / (1.0f + expf(-x));
  }
  if (p.renorm) {
    const float all = warp_sum(s);
    s = all > 0.0f ? s / all : 0.0f;
  }
  s *= p.factor;
  if (__any_sync(kFull, far)) s = far_weight(p, x, top, sum);
  if (mine) {
    p.idx[int64_t(t) * p.k + lane] = my_e;
    p.w[int64_t(t) * p.k + lane] = s;
  }
}

template <int VPL>
cudaError_t launch_vpl(const RouteParams& p, cudaStream_t st) {
  const int per = p.E / p.groups, lanes = per / VPL;
  const bool whole = p.E == 32 * VPL && per % VPL == 0 && (lanes & (lanes - 1)) == 0;
  return launch_kernel(whole ? route_grouped_kernel<VPL, true> : route_grouped_kernel<VPL, false>,
                       dim3((unsigned(p.T) + kWarps - 1) / kWarps), dim3(32 * kWarps), 0, st, false, p);
}

}  // namespace

cudaError_t launch_route_grouped(const float* logits, const float* bias, int T, int E, int k, int groups, int keep, int best,
                                 int softmax, int renorm, float factor, int32_t* idx, float* w, cudaStream_t st) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(bias);
  const RouteParams p = {logits, bias, T, E, k, groups, keep, best, softmax, renorm, factor, E % 4 == 0 && at % 16 == 0, idx, w};
  if (E <= 32) return launch_vpl<1>(p, st);
  if (E <= 64) return launch_vpl<2>(p, st);
  if (E <= 128) return launch_vpl<4>(p, st);
  if (E <= 256) return launch_vpl<8>(p, st);
  if (E <= 512) return launch_vpl<16>(p, st);
  return launch_vpl<32>(p, st);
}

}  // namespace nvfp4moe
