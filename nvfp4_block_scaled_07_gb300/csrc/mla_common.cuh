// Shared pieces of the latent-attention kernels: 16-bit element types,
// bounded waits, 16-bit tcgen05 MMAs and their descriptors, tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <mutex>

#include "internal.h"
#include "sm103_ptx.cuh"

namespace nvfp4moe {
namespace mla {

constexpr int kLatent = 512;
constexpr int kRope = 64;
constexpr int kRow = kLatent + kRope;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Two 16-bit values in one register, the first in the low half.
// kLift: log2 of a softmax weight at its row's maximum.  float16 ends at 2^-24,
// and many small weights beside a large one would vanish in the product with
// the values but not in their sum: its weights begin at 2^7, so that with a
// maximum that grew by 2^8 (kGrow) they stay below 2^16.  bfloat16 has the
// exponents of float32.
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1;  // tcgen05 kind::f16 operand format
  static constexpr float kLift = 0.0f;
  static constexpr CUtensorMapDataType kMap = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Elem<__half> {
  static constexpr uint32_t kFormat = 0;
  static constexpr float kLift = 7.0f;
  static constexpr CUtensorMapDataType kMap = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
};

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two float32 values in one instruction.
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float c) {  // (x, y) = (x, y) * a + b, c
  asm("{\n\t.reg .b64 v, f, g;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 f, {%2, %2};\n\tmov.b64 g, {%3, %4};\n\t"
      "fma.rn.f32x2 v, v, f, g;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {           // (x, y) += (a, b)
  asm("{\n\t.reg .b64 v, w;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\t"
      "add.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

__device__ __forceinline__ float max_of(const uint32_t (&s)[32]) {
  float a = __uint_as_float(s[0]), b = __uint_as_float(s[1]);  // two chains of three-way maxima
#pragma unroll
  for (int k = 2; k < 30; k += 4) {
    a = fmaxf(fmaxf(a, __uint_as_float(s[k])), __uint_as_float(s[k + 1]));
    b = fmaxf(fmaxf(b, __uint_as_float(s[k + 2])), __uint_as_float(s[k + 3]));
  }
  return fmaxf(fmaxf(a, b), fmaxf(__uint_as_float(s[30]), __uint_as_float(s[31])));
}
// w = exp2(s * scale + neg) of 32 scores, rounded to 16 bits for the second
// product; their float32 sum is added to sum0 + sum1.
template <typename T>
__device__ __forceinline__ void weights(const uint32_t (&s)[32], uint32_t (&w)[16], float scale, float neg, float& sum0,
                                        float& sum1) {
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    float e0 = __uint_as_float(s[k]), e1 = __uint_as_float(s[k + 1]);
    fma2(e0, e1, scale, neg, neg);
    e0 = exp2_approx(e0), e1 = exp2_approx(e1);
    add2(sum0, sum1, e0, e1);
    w[k / 2] = Elem<T>::pack(e0, e1);
  }
}

// ---- bounded waits ---------------------------------------------------------------
// Shared state of one CTA's waits: a wait that exceeds the limit raises the
// sticky flag and makes every role leave its loop.
struct WaitCtl {
  int abort;
  uint32_t limit_us;
  unsigned* flags;
};

// The timer is read only after 256 polls: reading it takes longer than most
// waits last.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile WaitCtl* ctl) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0u) {
      if (ctl->abort) return false;
      const uint64_t now = ptx::globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > uint64_t(ctl->limit_us) * 1000u) {
        ctl->abort = 1;
        atomicOr(ctl->flags, kFlagTimeout);
        return false;
      }
    }
  }
}

// The same for a whole converged warp (producers and MMA issuers), polled
// without suspending the threads; its lanes all get one answer.  The
// loop itself is uniform: code behind a divergent one would issue its MMAs
// and copies through per-lane registers, several times slower.
__device__ __forceinline__ bool test_warp(uint32_t bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, ptx::mbar_test_wait(bar, parity) != 0);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile WaitCtl* ctl) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (test_warp(bar, parity)) return true;
    if ((i & 255u) == 0u) {
      const uint64_t now = ptx::globaltimer_ns();
      if (t0 == 0) t0 = now;
      const bool late = now - t0 > uint64_t(ctl->limit_us) * 1000u;
      if (__any_sync(0xFFFFFFFFu, late)) {
        ctl->abort = 1;
        atomicOr(ctl->flags, kFlagTimeout);
      }
      if (__any_sync(0xFFFFFFFFu, late || ctl->abort)) return false;
    }
  }
}
// A value that is the same in all lanes, said so to the compiler.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Wait for a CTA's own copies or MMAs before it leaves, also after an abort.
__device__ __forceinline__ void drain_phase(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity))
    if (ptx::globaltimer_ns() - t0 > 2000000000ull) return;
}

// ---- tcgen05 kind::f16 -------------------------------------------------------------
// Instruction descriptor: both operands of one 16-bit format, float32
// accumulator, dense; *_mn: the operand is stored with M (N) contiguous
// instead of K.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t format, int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4)                               // D format: float32
         | (format << 7) | (format << 10)        // A and B format
         | (uint32_t(a_mn ? 1u : 0u) << 15) | (uint32_t(b_mn ? 1u : 0u) << 16)
         | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}
// One lane of a converged warp, chosen by the hardware (the same one each
// time).  The MMA and TMA issuers run their loops with the whole warp and
// predicate the issue on this: with warp-uniform operands an MMA issues in
// about 30 cycles, from a single-lane branch (whose operands are moved to
// uniform registers one by one) in about 50 and more.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      :
      : "memory");
  return r;
}
// Shared-memory operand descriptors, 128-byte swizzle.  An operand is made of
// atoms of 8 rows x 128 bytes (1024 bytes, aligned to as much).
//   K-major: rows are M (N), their 64 values along K; `stride` from one 8-row
//     group to the next; 16 values of K are 32 bytes.
//   MN-major: rows are K, their 64 values along M (N); `stride` from one
//     8-row group of K to the next, `lead` to the next 64 values of M (N).
// The address and lead are the low word, which the MMAs of a tile step by
// constants; the stride is the high word, a constant of the MMA.
__device__ __forceinline__ uint32_t desc_sw128(uint32_t saddr, uint32_t lead) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t stride) { return (stride >> 4) | (1u << 14) | (2u << 29); }

// D[tmem] (+)= A[smem] B[smem]^T, K = 16, issued where `elected`.
template <uint32_t A_STRIDE, uint32_t B_STRIDE>
__device__ __forceinline__ void mma_f16(uint32_t elected, uint32_t d_tmem, uint32_t a_desc, uint32_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %7};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_desc), "r"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected), "n"(desc_hi(A_STRIDE)), "n"(desc_hi(B_STRIDE))
      : "memory");
}
// The same with A in tensor memory: lane = row of A, 16-bit pairs along K.
template <uint32_t B_STRIDE>
__device__ __forceinline__ void mma_f16_ts(uint32_t elected, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %6};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected), "n"(desc_hi(B_STRIDE))
      : "memory");
}
// The first on a CTA pair, issued by the even CTA: M rows, half of them in
// each CTA's shared memory at one offset; N rows of B likewise.  With M = 128
// a CTA's tensor memory holds its 64 rows in lanes 0-63 for the first half of
// the columns and in lanes 64-127 for the second.
template <uint32_t A_STRIDE, uint32_t B_STRIDE>
__device__ __forceinline__ void mma_f16_pair(uint32_t elected, uint32_t d_tmem, uint32_t a_desc, uint32_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %7};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_desc), "r"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected), "n"(desc_hi(A_STRIDE)), "n"(desc_hi(B_STRIDE))
      : "memory");
}
// Arrive on the mbarrier at offset `bar` in both CTAs of the pair.
__device__ __forceinline__ void tc_commit_pair(uint32_t elected, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"((unsigned short)3), "r"(elected)
      : "memory");
}
// Pair form of the load: the data lands in this CTA, the completion counts
// on `bar`, a cluster address.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t elected, uint32_t dst, const void* tmap, uint32_t bar,
                                                 int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t elected, uint32_t dst, const void* tmap, uint32_t bar, int32_t c0,
                                            int32_t c1, int32_t c2, int32_t c3) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %7, 0;\n\t"
      "@q cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(elected)
      : "memory");
}

// Arrive on `bar` once every MMA issued so far by the elected lane has completed.
__device__ __forceinline__ void tc_commit(uint32_t elected, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t elected, uint32_t dst, const void* tmap, uint32_t bar, int32_t c0,
                                            int32_t c1, int32_t c2) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void arrive_expect_tx(uint32_t elected, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(elected)
      : "memory");
}

// Arrive on an mbarrier of the other CTA of a pair; it announces nothing but itself.
__device__ __forceinline__ void arrive_peer(uint32_t elected, uint32_t cluster_addr) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_addr),
      "r"(elected)
      : "memory");
}

// 16 lanes x 32 columns of a warp's lane quarter: thread l holds, in r[4i ..
// 4i+3], columns 8i + 2 (l % 4) + {0, 1} of lane l / 4 and then of lane l / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 16 consecutive columns of each lane.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void sts32(uint32_t saddr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(saddr), "r"(v) : "memory");
}
// Barrier among `n` threads of the CTA (ids 1..15; 0 is __syncthreads).
__device__ __forceinline__ void bar_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// The same, returning whether any of the threads passed a true predicate.
__device__ __forceinline__ bool bar_any(int id, int n, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(uint32_t(pred))
      : "memory");
  return r != 0;
}

// ---- tensor maps ------------------------------------------------------------------
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}
// 16-bit tensor of `rank` dimensions (innermost first, strides in bytes of
// dimensions 1..) with a 128-byte swizzled box; out-of-range rows read zero.
inline bool encode_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const int64_t* dims,
                       const int64_t* strides, const int* box) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t d[5], s[4];
  cuuint32_t b[5], e[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = cuuint64_t(dims[i]);
    b[i] = cuuint32_t(box[i]);
    e[i] = 1;
    if (i) s[i - 1] = cuuint64_t(strides[i - 1]);
  }
  return enc(m, type, cuuint32_t(rank), const_cast<void*>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mla
}  // namespace nvfp4moe
