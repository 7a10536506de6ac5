// Appending tokens to the paged latent cache: RMS norm of the latent part,
// rotation of the key's and the queries' rotary parts, and the scattered
// store of the row, in one pass.
//
// With x the 512 latent values of a token, w the norm's weight and (c_i, s_i)
// the angles' cosines and sines at the token's position:
//   n_j = x_j * rsqrt(sum x^2 / 512 + eps) * w_j
//   (a_i, b_i) -> (a_i c_i - b_i s_i, b_i c_i + a_i s_i)       32 pairs a head
// Everything is float32 between the loads and the single rounding at the
// stores.
//
// Bound by memory: every value is read once and written once (the row twice:
// cache and copy).  A warp takes one unit, either a token's row (each lane 16
// latent values as two 16-byte loads; lanes 0-3 the rotary part) or sixteen
// heads of its queries (four lanes a head and its eighth neighbour, eight
// pairs a lane, so that both pair layouts are two 16-byte loads), so all loads
// of a unit are in flight at once and no unit waits for another.
// 16384 tokens with 16 heads (128 MB): 23.2 us, 5.5 TB/s, four fifths of a
// plain copy's rate; with units of eight heads 25.1 us, without the bound of
// 48 registers (58, four blocks an SM instead of five) 23.9 us.
// One token takes 2.1 us, the launch.
#include <cstdint>

#include "../../include/nvfp4mla.h"
#include "internal.h"
#include "launch.cuh"
#include "mla_common.cuh"
#include "sm103_ptx.cuh"

namespace nvfp4moe {
namespace {

__device__ unsigned g_append_flags = 0;

constexpr int kWarps = 8;         // warps a block
constexpr int kHeadsPerWarp = 16; // query heads of one unit

struct AppendParams {
  const uint8_t* latent;   // byte strides below
  int64_t latent_stride;
  const uint8_t* k_rope;
  int64_t k_rope_stride;
  const uint4* norm_weight;
  float eps;
  const int32_t* positions;
  const int64_t* slots;
  int T;
  const float* table;
  int64_t max_positions;
  uint8_t* cache;
  int64_t num_slots;
  uint8_t* rows_out;
  const uint8_t* q;
  int64_t q_token_stride, q_head_stride;
  int H;
  uint8_t* q_out;
  int64_t qo_token_stride, qo_head_stride;
  int units;               // units a token: its row and ceil(H / 16) groups of heads
};

// Rotates the eight pairs 8j .. 8j+7 of one head (j = 0..3).  In the
// interleaved layout they are values 16j .. 16j+15, otherwise values 8j ..
// 8j+7 and 32+8j .. 32+8j+7; `lo` and `hi` are those two 16-byte pieces.
template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void rotate(uint4& lo, uint4& hi, const float (&c)[8], const float (&s)[8]) {
  uint32_t* l = reinterpret_cast<uint32_t*>(&lo);
  uint32_t* h = reinterpret_cast<uint32_t*>(&hi);
  if (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = i < 4 ? l[i] : h[i - 4];
      const float2 v = mla::Elem<T>::unpack(w);
      w = mla::Elem<T>::pack(v.x * c[i] - v.y * s[i], v.y * c[i] + v.x * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = mla::Elem<T>::unpack(l[i]), b = mla::Elem<T>::unpack(h[i]);
      l[i] = mla::Elem<T>::pack(a.x * c[2 * i] - b.x * s[2 * i], a.y * c[2 * i + 1] - b.y * s[2 * i + 1]);
      h[i] = mla::Elem<T>::pack(b.x * c[2 * i] + a.x * s[2 * i], b.y * c[2 * i + 1] + a.y * s[2 * i + 1]);
    }
  }
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps, 5) append_kernel(const AppendParams p) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int lane = threadIdx.x & 31;
  // unit kWarps * blockIdx.x + warp of T * units, without a 64-bit division
  const unsigned units = unsigned(p.units), group = blockIdx.x / units;
  const unsigned in = kWarps * (blockIdx.x - group * units) + (threadIdx.x >> 5);
  const int t = int(kWarps * group + in / units), u = int(in % units);
  if (t >= p.T) return;
  // byte offsets of the two pieces that the lane rotates within a head
  const int j = lane & 3;
  const int off_lo = INTERLEAVED ? 32 * j : 16 * j, off_hi = INTERLEAVED ? 32 * j + 16 : 64 + 16 * j;
  const int pos = __ldg(p.positions + t);
  const bool pos_ok = pos >= 0 && pos < p.max_positions;
  float c[8], s[8];                           // cosines and sines of the lane's eight pairs
  auto angles = [&] {
    const float* cs = p.table + int64_t(pos_ok ? pos : 0) * mla::kRope + 8 * j;
    *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(cs));
    *reinterpret_cast<float4*>(c + 4) = __ldg(reinterpret_cast<const float4*>(cs + 4));
    *reinterpret_cast<float4*>(s) = __ldg(reinterpret_cast<const float4*>(cs + 32));
    *reinterpret_cast<float4*>(s + 4) = __ldg(reinterpret_cast<const float4*>(cs + 36));
  };

  if (u == 0) {
    const uint8_t* x = p.latent + t * p.latent_stride;
    uint4 a = *reinterpret_cast<const uint4*>(x + 16 * lane);          // values 8 lane ..
    uint4 b = *reinterpret_cast<const uint4*>(x + 512 + 16 * lane);    // values 256 + 8 lane ..
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (lane < 4) {
      const uint8_t* r = p.k_rope + t * p.k_rope_stride;
      lo = *reinterpret_cast<const uint4*>(r + off_lo);
      hi = *reinterpret_cast<const uint4*>(r + off_hi);
    }
    const int64_t slot = __ldg(p.slots + t);
    if (!pos_ok || slot >= p.num_slots) {
      if (lane == 0) atomicOr(&g_append_flags, kFlagBadData);
      if (!pos_ok) return;
    }
    if (p.norm_weight) {
      uint32_t* av = reinterpret_cast<uint32_t*>(&a);
      uint32_t* bv = reinterpret_cast<uint32_t*>(&b);
      const uint4 wa = __ldg(p.norm_weight + lane), wb = __ldg(p.norm_weight + 32 + lane);
      const uint32_t* wav = reinterpret_cast<const uint32_t*>(&wa);
      const uint32_t* wbv = reinterpret_cast<const uint32_t*>(&wb);
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = mla::Elem<T>::unpack(av[i]), w = mla::Elem<T>::unpack(bv[i]);
        ss += v.x * v.x + v.y * v.y + w.x * w.x + w.y * w.y;
      }
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
      const float inv = 1.0f / sqrtf(ss * (1.0f / mla::kLatent) + p.eps);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = mla::Elem<T>::unpack(av[i]), w = mla::Elem<T>::unpack(wav[i]);
        av[i] = mla::Elem<T>::pack(v.x * inv * w.x, v.y * inv * w.y);
        const float2 v2 = mla::Elem<T>::unpack(bv[i]), w2 = mla::Elem<T>::unpack(wbv[i]);
        bv[i] = mla::Elem<T>::pack(v2.x * inv * w2.x, v2.y * inv * w2.y);
      }
    }
    if (lane < 4) {
      angles();
      rotate<T, INTERLEAVED>(lo, hi, c, s);
    }
    auto store = [&](uint8_t* dst) {
      *reinterpret_cast<uint4*>(dst + 16 * lane) = a;
      *reinterpret_cast<uint4*>(dst + 512 + 16 * lane) = b;
      if (lane < 4) {
        *reinterpret_cast<uint4*>(dst + 1024 + off_lo) = lo;
        *reinterpret_cast<uint4*>(dst + 1024 + off_hi) = hi;
      }
    };
    if (slot >= 0 && slot < p.num_slots) store(p.cache + slot * (2 * mla::kRow));
    if (p.rows_out) store(p.rows_out + int64_t(t) * (2 * mla::kRow));
  } else if (pos_ok) {  // the row's unit raises the flag of a bad position
    const int h = (u - 1) * kHeadsPerWarp + (lane >> 2);
    if (h >= p.H) return;
    const bool both = h + 8 < p.H;            // and head h + 8, with the same angles
    const uint8_t* x = p.q + t * p.q_token_stride + h * p.q_head_stride;
    const uint8_t* x2 = both ? x + 8 * p.q_head_stride : x;
    uint4 lo = *reinterpret_cast<const uint4*>(x + off_lo), hi = *reinterpret_cast<const uint4*>(x + off_hi);
    uint4 lo2 = *reinterpret_cast<const uint4*>(x2 + off_lo), hi2 = *reinterpret_cast<const uint4*>(x2 + off_hi);
    angles();
    rotate<T, INTERLEAVED>(lo, hi, c, s);
    rotate<T, INTERLEAVED>(lo2, hi2, c, s);
    uint8_t* y = p.q_out + t * p.qo_token_stride + h * p.qo_head_stride;
    *reinterpret_cast<uint4*>(y + off_lo) = lo;
    *reinterpret_cast<uint4*>(y + off_hi) = hi;
    if (both) {
      y += 8 * p.qo_head_stride;
      *reinterpret_cast<uint4*>(y + off_lo) = lo2;
      *reinterpret_cast<uint4*>(y + off_hi) = hi2;
    }
  }
}

int units_of(int H) { return 1 + (H + kHeadsPerWarp - 1) / kHeadsPerWarp; }

}  // namespace

int64_t mla_append_blocks(int T, int H) { return (int64_t(T) * units_of(H) + kWarps - 1) / kWarps; }

cudaError_t launch_mla_append(const MlaAppendArgs& a, cudaStream_t st) {
  AppendParams p;
  p.latent = static_cast<const uint8_t*>(a.latent);
  p.latent_stride = 2 * a.latent_stride;
  p.k_rope = static_cast<const uint8_t*>(a.k_rope);
  p.k_rope_stride = 2 * a.k_rope_stride;
  p.norm_weight = static_cast<const uint4*>(a.norm_weight);
  p.eps = a.eps;
  p.positions = a.positions;
  p.slots = a.slots;
  p.T = a.T;
  p.table = a.table;
  p.max_positions = a.max_positions;
  p.cache = static_cast<uint8_t*>(a.cache);
  p.num_slots = a.num_slots;
  p.rows_out = static_cast<uint8_t*>(a.rows_out);
  p.q = static_cast<const uint8_t*>(a.q);
  p.q_token_stride = 2 * a.q_token_stride;
  p.q_head_stride = 2 * a.q_head_stride;
  p.H = a.H;
  p.q_out = static_cast<uint8_t*>(a.q_out);
  p.qo_token_stride = 2 * a.qo_token_stride;
  p.qo_head_stride = 2 * a.qo_head_stride;
  p.units = units_of(a.H);
  auto kernel = a.fp16 ? (a.interleaved ? append_kernel<__half, true> : append_kernel<__half, false>)
                       : (a.interleaved ? append_kernel<__nv_bfloat16, true> : append_kernel<__nv_bfloat16, false>);
  return launch_kernel(kernel, dim3(unsigned(mla_append_blocks(a.T, a.H))), dim3(32 * kWarps), 0, st, false, p);
}

cudaError_t mla_append_flags_address(unsigned** at) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_append_flags);
}

}  // namespace nvfp4moe
