// C entry points of libnvfp4moe: argument validation, the per-device
// attribute cache and status plumbing.  The compute lives in
// kernels_prep.cu and grouped_gemm.cu; nothing here allocates device memory.
#include <atomic>
#include <cstdint>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "../../include/nvfp4few.h"
#include "../../include/nvfp4mla.h"
#include "../../include/nvfp4moe.h"
#include "internal.h"

namespace nvfp4moe {

namespace {

thread_local char t_detail[512] = "";

struct DeviceInfo {
  bool checked = false;
  int status = NVFP4MOE_OK;
  int num_sms = 0;
  int smem_optin = 0;
};

constexpr int kMaxDevices = 64;
DeviceInfo g_devices[kMaxDevices];
std::mutex g_dev_mutex;

int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_detail, sizeof(t_detail), fmt, ap);
  va_end(ap);
  return status;
}

int check_device(int dev, DeviceInfo* out) {
  if (dev < 0 || dev >= kMaxDevices) return fail(NVFP4MOE_ERR_INVALID_ARG, "device %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  DeviceInfo& d = g_devices[dev];
  if (!d.checked) {
    cudaDeviceProp prop;
    cudaError_t err = cudaGetDeviceProperties(&prop, dev);
    if (err != cudaSuccess) return fail(NVFP4MOE_ERR_CUDA, "cudaGetDeviceProperties: %s", cudaGetErrorString(err));
    int optin = 0;
    err = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (err != cudaSuccess) return fail(NVFP4MOE_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(err));
    d.num_sms = prop.multiProcessorCount;
    d.smem_optin = optin;
    d.status = (prop.major == 10 && prop.minor == 3) ? NVFP4MOE_OK : NVFP4MOE_ERR_UNSUPPORTED;
    d.checked = true;
    if (d.status != NVFP4MOE_OK)
      snprintf(t_detail, sizeof(t_detail), "device %d is compute capability %d.%d; libnvfp4moe is built for 10.3",
               dev, prop.major, prop.minor);
  }
  if (d.status != NVFP4MOE_OK) return fail(d.status, "device %d is not compute capability 10.3", dev);
  *out = d;
  return NVFP4MOE_OK;
}

int current_device(DeviceInfo* out) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return fail(NVFP4MOE_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(err));
  return check_device(dev, out);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int cuda_status(cudaError_t err, const char* what) {
  if (err == cudaSuccess) return NVFP4MOE_OK;
  return fail(NVFP4MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(err));
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

void set_error_detail(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_detail, sizeof(t_detail), fmt, ap);
  va_end(ap);
}

}  // namespace nvfp4moe

namespace nvfp4moe {
namespace {
std::atomic<uint32_t> g_wait_limit_us{kDefaultWaitUs};
}  // namespace
uint32_t wait_limit_us() { return g_wait_limit_us.load(std::memory_order_relaxed); }
}  // namespace nvfp4moe

namespace nvfp4moe {
namespace {
// The sticky flags of the kernel files that raise any, on the current device.
constexpr int kFlagWords = 8;
struct FlagWords {
  unsigned* at[kFlagWords];
};
std::mutex g_status_mutex;              // of g_collected between kernel and copy
__device__ unsigned g_collected;

// Reads and clears all flags at once, each atomically.
__global__ void collect_flags(const FlagWords w) {
  unsigned f = 0;
  if (threadIdx.x < kFlagWords) f = atomicExch(w.at[threadIdx.x], 0u);
  f = __reduce_or_sync(0xFFFFFFFFu, f);
  if (threadIdx.x == 0) g_collected = f;
}

// One kernel and one copy, whatever the number of files (a copy to read and
// one to clear each took 75 us for five files; this 23).
cudaError_t read_and_clear_flags(unsigned* flags, cudaStream_t st) {
  FlagWords w;
  cudaError_t err;
  if ((err = prep_flags_address(&w.at[0])) != cudaSuccess || (err = gemm_flags_address(&w.at[1])) != cudaSuccess ||
      (err = mla_append_flags_address(&w.at[2])) != cudaSuccess || (err = mla_decode_flags_address(&w.at[3])) != cudaSuccess ||
      (err = mla_prefill_flags_address(&w.at[4])) != cudaSuccess || (err = few_flags_address(&w.at[5])) != cudaSuccess ||
      (err = mla_plan_flags_address(&w.at[6])) != cudaSuccess || (err = stream_flags_address(&w.at[7])) != cudaSuccess)
    return err;
  std::lock_guard<std::mutex> lock(g_status_mutex);
  collect_flags<<<1, 32, 0, st>>>(w);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  err = cudaMemcpyFromSymbolAsync(flags, g_collected, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, st);
  if (err != cudaSuccess) return err;
  return cudaStreamSynchronize(st);
}
}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

#define NVFP4MOE_REQUIRE(cond, status, ...) \
  do {                                      \
    if (!(cond)) return fail(status, __VA_ARGS__); \
  } while (0)

extern "C" {

int nvfp4moe_version(void) { return 1 * 10000 + 0 * 100 + 0; }

const char* nvfp4moe_status_string(int status) {
  switch (status) {
    case NVFP4MOE_OK: return "ok";
    case NVFP4MOE_ERR_INVALID_ARG: return "invalid argument";
    case NVFP4MOE_ERR_UNSUPPORTED: return "unsupported shape or device";
    case NVFP4MOE_ERR_SMEM: return "tile pipeline exceeds the opt-in shared memory";
    case NVFP4MOE_ERR_WORKSPACE: return "workspace too small";
    case NVFP4MOE_ERR_CUDA: return "CUDA runtime error";
    case NVFP4MOE_ERR_TIMEOUT: return "device pipeline wait timed out";
    case NVFP4MOE_ERR_DEVICE_DATA: return "device data out of range";
    default: return "unknown status";
  }
}

const char* nvfp4moe_last_error_detail(void) { return t_detail; }

int nvfp4moe_device_check(int device) {
  DeviceInfo d;
  t_detail[0] = 0;
  return check_device(device, &d);
}

int nvfp4moe_set_wait_limit_us(uint32_t us) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(us <= kMaxWaitUs, NVFP4MOE_ERR_INVALID_ARG, "wait limit %u us above the maximum %u us", us,
                   kMaxWaitUs);
  g_wait_limit_us.store(us == 0 ? kDefaultWaitUs : us, std::memory_order_relaxed);
  return NVFP4MOE_OK;
}

uint32_t nvfp4moe_wait_limit_us(void) { return wait_limit_us(); }

int nvfp4moe_wait_selftest(uint32_t expected_arrivals, uint32_t arrivals, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(expected_arrivals >= 1 && expected_arrivals <= 64 && arrivals <= 32, NVFP4MOE_ERR_INVALID_ARG,
                   "expected_arrivals %u (1..64), arrivals %u (0..32)", expected_arrivals, arrivals);
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_wait_selftest(expected_arrivals, arrivals, stream), "wait self-test launch");
}

int nvfp4moe_sync_status(cudaStream_t stream) {
  // first of all: a stream that is being captured refuses this, before anything is launched on it
  int st = cuda_status(cudaStreamSynchronize(stream), "cudaStreamSynchronize");
  if (st) return st;
  unsigned f = 0;
  st = cuda_status(read_and_clear_flags(&f, stream), "reading device flags");
  if (st) return st;
  if (f & kFlagTimeout) return fail(NVFP4MOE_ERR_TIMEOUT, "a device wait (grouped GEMM, attention or few-token pipeline, or prepare grid barrier) exceeded its time limit");
  if (f & kFlagBadData) return fail(NVFP4MOE_ERR_DEVICE_DATA, "an expert id, row index, cache slot, page, position, sequence length or page count was out of range");
  return NVFP4MOE_OK;
}

size_t nvfp4moe_blocked_scales_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0 || cols % 64) return 0;
  return size_t(ceil_div(rows, 128) * 128 * (cols / 16));
}

size_t nvfp4moe_mxfp4_blocked_scales_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0 || cols % 128) return 0;
  return size_t(ceil_div(rows, 128) * 128 * (cols / 32));
}

size_t nvfp4moe_tiled_weights_bytes(int64_t rows, int K) {
  if (rows <= 0 || rows % 128 || K <= 0 || K % 64) return 0;
  return size_t((rows / 128) * ceil_div(int64_t(K), 256) * kWeightBoxBytes);
}

int nvfp4moe_tile_weights(const uint8_t* w_packed, int64_t rows, int K, uint8_t* w_tiled, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(rows > 0 && rows % 128 == 0 && K > 0 && K % 64 == 0, NVFP4MOE_ERR_UNSUPPORTED,
                   "rows = %lld must be a positive multiple of 128 and K = %d of 64", (long long)rows, K);
  NVFP4MOE_REQUIRE(w_packed && w_tiled && aligned16(w_packed) && aligned16(w_tiled), NVFP4MOE_ERR_INVALID_ARG,
                   "null or misaligned pointer");
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_tile_weights(w_packed, rows, K, w_tiled, d.num_sms, stream), "tile weights launch");
}

// ---- a1 ---------------------------------------------------------------------
int moe_route_topk(const float* logits, const float* bias, int T, int E, int k, int score_fn, int renormalize,
                   int32_t* topk_idx, float* topk_w, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(T >= 0, NVFP4MOE_ERR_INVALID_ARG, "T = %d must be >= 0", T);
  NVFP4MOE_REQUIRE(E >= 1 && E <= 1024, NVFP4MOE_ERR_UNSUPPORTED, "E = %d outside [1, 1024]", E);
  NVFP4MOE_REQUIRE(k >= 1 && k <= E && k <= 32, NVFP4MOE_ERR_UNSUPPORTED, "k = %d outside [1, min(E, 32)]", k);
  NVFP4MOE_REQUIRE(score_fn == NVFP4MOE_SCORE_SOFTMAX || score_fn == NVFP4MOE_SCORE_SIGMOID,
                   NVFP4MOE_ERR_INVALID_ARG, "score_fn %d", score_fn);
  if (T == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(logits && topk_idx && topk_w, NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_route_topk(logits, bias, T, E, k, score_fn, renormalize ? 1 : 0, topk_idx, topk_w, stream),
                     "route launch");
}

size_t moe_route_batch_aware_workspace_size(int E) {
  if (E < 1) return 0;
  return size_t(ceil_div(E, 32)) * sizeof(uint32_t);
}

int moe_route_batch_aware(const float* logits, const float* bias, int T, int E, int k, int k_primary, int score_fn,
                          int renormalize, int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes,
                          cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(T >= 0, NVFP4MOE_ERR_INVALID_ARG, "T = %d must be >= 0", T);
  NVFP4MOE_REQUIRE(E >= 1 && E <= 1024, NVFP4MOE_ERR_UNSUPPORTED, "E = %d outside [1, 1024]", E);
  NVFP4MOE_REQUIRE(k >= 1 && k <= E && k <= 32, NVFP4MOE_ERR_UNSUPPORTED, "k = %d outside [1, min(E, 32)]", k);
  NVFP4MOE_REQUIRE(k_primary >= 1 && k_primary <= k, NVFP4MOE_ERR_INVALID_ARG, "k_primary = %d outside [1, k = %d]",
                   k_primary, k);
  NVFP4MOE_REQUIRE(score_fn == NVFP4MOE_SCORE_SOFTMAX || score_fn == NVFP4MOE_SCORE_SIGMOID,
                   NVFP4MOE_ERR_INVALID_ARG, "score_fn %d", score_fn);
  if (T == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(logits && topk_idx && topk_w, NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  const size_t need = moe_route_batch_aware_workspace_size(E);
  NVFP4MOE_REQUIRE(ws && ws_bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 3) == 0, NVFP4MOE_ERR_WORKSPACE,
                   "workspace %zu < %zu or misaligned", ws_bytes, need);
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_route_batch_aware(logits, bias, T, E, k, k_primary, score_fn, renormalize ? 1 : 0,
                                              topk_idx, topk_w, static_cast<uint32_t*>(ws), stream),
                     "batch-aware route launch");
}

// ---- a2 ---------------------------------------------------------------------
size_t moe_quantize_nvfp4_workspace_size(int64_t rows, int64_t cols, int flags) {
  (void)rows;
  (void)cols;
  return (flags & NVFP4MOE_QUANT_COMPUTE_GLOBAL) ? 16 : 0;
}

int moe_quantize_nvfp4(const void* x_bf16, int64_t rows, int64_t cols, float* global_scale, int flags,
                       uint8_t* packed, uint8_t* scales, void* ws, size_t ws_bytes, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(rows >= 0 && cols > 0, NVFP4MOE_ERR_INVALID_ARG, "rows %lld cols %lld", (long long)rows,
                   (long long)cols);
  NVFP4MOE_REQUIRE((flags & ~3) == 0, NVFP4MOE_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
  const bool blocked = flags & NVFP4MOE_QUANT_SCALES_BLOCKED;
  const bool compute = flags & NVFP4MOE_QUANT_COMPUTE_GLOBAL;
  NVFP4MOE_REQUIRE(cols % 16 == 0, NVFP4MOE_ERR_UNSUPPORTED, "cols %lld is not a multiple of 16", (long long)cols);
  NVFP4MOE_REQUIRE(!blocked || cols % 64 == 0, NVFP4MOE_ERR_UNSUPPORTED,
                   "blocked scales need cols %% 64 == 0 (cols %lld)", (long long)cols);
  if (rows == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(x_bf16 && global_scale && packed && scales, NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(aligned16(x_bf16) && aligned16(packed), NVFP4MOE_ERR_INVALID_ARG,
                   "x and packed must be 16-byte aligned");
  const size_t need = moe_quantize_nvfp4_workspace_size(rows, cols, flags);
  NVFP4MOE_REQUIRE(ws_bytes >= need && (need == 0 || ws), NVFP4MOE_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes,
                   need);
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_quantize(x_bf16, rows, cols, global_scale, compute, blocked, packed, scales,
                                     static_cast<unsigned*>(ws), d.num_sms, stream),
                     "quantize launch");
}

int moe_quantize_mxfp4(const void* x_bf16, int64_t rows, int64_t cols, int flags, uint8_t* packed, uint8_t* scales,
                       cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(rows >= 0 && cols > 0, NVFP4MOE_ERR_INVALID_ARG, "rows %lld cols %lld", (long long)rows,
                   (long long)cols);
  NVFP4MOE_REQUIRE((flags & ~NVFP4MOE_QUANT_SCALES_BLOCKED) == 0, NVFP4MOE_ERR_INVALID_ARG, "unknown flags 0x%x",
                   flags);
  const bool blocked = flags & NVFP4MOE_QUANT_SCALES_BLOCKED;
  NVFP4MOE_REQUIRE(cols % 32 == 0, NVFP4MOE_ERR_UNSUPPORTED, "cols %lld is not a multiple of 32", (long long)cols);
  NVFP4MOE_REQUIRE(!blocked || cols % 128 == 0, NVFP4MOE_ERR_UNSUPPORTED,
                   "blocked scales need cols %% 128 == 0 (cols %lld)", (long long)cols);
  if (rows == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(x_bf16 && packed && scales, NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(aligned16(x_bf16) && aligned16(packed), NVFP4MOE_ERR_INVALID_ARG,
                   "x and packed must be 16-byte aligned");
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_quantize_mx(x_bf16, rows, cols, blocked, packed, scales, d.num_sms, stream),
                     "MXFP4 quantize launch");
}

int moe_scales_to_blocked(const uint8_t* scales_row_major, int64_t rows, int64_t cols, uint8_t* scales_blocked,
                          cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(rows >= 0 && cols > 0, NVFP4MOE_ERR_INVALID_ARG, "bad shape");
  NVFP4MOE_REQUIRE(cols % 64 == 0, NVFP4MOE_ERR_UNSUPPORTED, "cols must be a multiple of 64");
  if (rows == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(scales_row_major && scales_blocked, NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE((reinterpret_cast<uintptr_t>(scales_row_major) & 3) == 0 && aligned16(scales_blocked),
                   NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_scales_to_blocked(scales_row_major, rows, cols, scales_blocked, d.num_sms, stream),
                     "scale re-layout launch");
}

// ---- a3 ---------------------------------------------------------------------
int64_t moe_permute_rows_capacity(int T, int E, int k) {
  if (T < 0 || E < 1 || k < 1) return 0;
  return ceil_div(int64_t(T) * k + int64_t(E) * 127, 128) * 128;
}

size_t moe_permute_workspace_size(int T, int E, int k) {
  if (T < 0 || E < 1 || k < 1) return 0;
  const int64_t R = int64_t(T) * k;
  const int64_t nseg = ceil_div(R, kPermuteSegment);
  const size_t rank = size_t(ceil_div(R, 64) * 64) * 4;
  const size_t seg = size_t(ceil_div(nseg * E, 64) * 64) * 4;
  return rank + 2 * seg + 256;
}

static int permute_common(const int32_t* topk_idx, int T, int E, int k, const uint8_t* xq, const uint8_t* xs, int H, int scale_block,
                int32_t* expert_counts, int32_t* expert_offsets, int32_t* row_offsets, int32_t* perm_to_flat,
                int32_t* flat_to_perm, uint8_t* a_packed, uint8_t* a_scales, void* ws, size_t ws_bytes,
                cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(T >= 0, NVFP4MOE_ERR_INVALID_ARG, "T = %d", T);
  NVFP4MOE_REQUIRE(E >= 1 && E <= 1024, NVFP4MOE_ERR_UNSUPPORTED, "E = %d outside [1, 1024]", E);
  NVFP4MOE_REQUIRE(k >= 1 && k <= E, NVFP4MOE_ERR_UNSUPPORTED, "k = %d outside [1, E]", k);
  NVFP4MOE_REQUIRE(H > 0 && H % (4 * scale_block) == 0, NVFP4MOE_ERR_UNSUPPORTED,
                   "H = %d must be a positive multiple of %d", H, 4 * scale_block);
  NVFP4MOE_REQUIRE(int64_t(T) * k <= (int64_t(1) << 30), NVFP4MOE_ERR_UNSUPPORTED, "T*k too large");
  NVFP4MOE_REQUIRE(expert_counts && expert_offsets && row_offsets && perm_to_flat, NVFP4MOE_ERR_INVALID_ARG,
                   "null pointer");
  NVFP4MOE_REQUIRE(T == 0 || (topk_idx && xq && xs && flat_to_perm && a_packed && a_scales),
                   NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(T == 0 || (aligned16(xq) && aligned16(a_packed) && aligned16(a_scales) &&
                              (reinterpret_cast<uintptr_t>(xs) & 3) == 0),
                   NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = moe_permute_workspace_size(T, E, k);
  NVFP4MOE_REQUIRE(ws && ws_bytes >= need, NVFP4MOE_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, need);
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  const int64_t R = int64_t(T) * k;
  const int64_t nseg = ceil_div(R, kPermuteSegment);
  int32_t* rank = static_cast<int32_t*>(ws);
  int32_t* seg_count = rank + ceil_div(R, 64) * 64;
  int32_t* seg_base = seg_count + ceil_div(nseg * E, 64) * 64;
  return cuda_status(launch_permute(topk_idx, T, E, k, xq, xs, H, H / (4 * scale_block), expert_counts, expert_offsets, row_offsets,
                                    perm_to_flat, flat_to_perm, a_packed, a_scales,
                                    moe_permute_rows_capacity(T, E, k), rank, seg_count, seg_base, d.num_sms,
                                    stream),
                     "permute launch");
}

int moe_permute(const int32_t* topk_idx, int T, int E, int k, const uint8_t* xq, const uint8_t* xs, int H,
                int32_t* expert_counts, int32_t* expert_offsets, int32_t* row_offsets, int32_t* perm_to_flat,
                int32_t* flat_to_perm, uint8_t* a_packed, uint8_t* a_scales, void* ws, size_t ws_bytes,
                cudaStream_t stream) {
  return permute_common(topk_idx, T, E, k, xq, xs, H, 16, expert_counts, expert_offsets, row_offsets, perm_to_flat,
                        flat_to_perm, a_packed, a_scales, ws, ws_bytes, stream);
}

int moe_permute_mxfp4(const int32_t* topk_idx, int T, int E, int k, const uint8_t* xq, const uint8_t* xs, int H,
                      int32_t* expert_counts, int32_t* expert_offsets, int32_t* row_offsets, int32_t* perm_to_flat,
                      int32_t* flat_to_perm, uint8_t* a_packed, uint8_t* a_scales, void* ws, size_t ws_bytes,
                      cudaStream_t stream) {
  return permute_common(topk_idx, T, E, k, xq, xs, H, 32, expert_counts, expert_offsets, row_offsets, perm_to_flat,
                        flat_to_perm, a_packed, a_scales, ws, ws_bytes, stream);
}

int moe_permute_no_alloc(const int32_t* topk_idx, int T, int E, int k, const uint8_t* xq, const uint8_t* xs, int H,
                         int32_t* expert_counts, int32_t* expert_offsets, int32_t* row_offsets,
                         int32_t* perm_to_flat, int32_t* flat_to_perm, uint8_t* a_packed, uint8_t* a_scales,
                         cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(T >= 0, NVFP4MOE_ERR_INVALID_ARG, "T = %d", T);
  NVFP4MOE_REQUIRE(E >= 1 && E <= 1024, NVFP4MOE_ERR_UNSUPPORTED, "E = %d outside [1, 1024]", E);
  NVFP4MOE_REQUIRE(k >= 1 && k <= E, NVFP4MOE_ERR_UNSUPPORTED, "k = %d outside [1, E]", k);
  NVFP4MOE_REQUIRE(H > 0 && H % 64 == 0, NVFP4MOE_ERR_UNSUPPORTED, "H = %d must be a positive multiple of 64", H);
  const int64_t R = int64_t(T) * k;
  const int64_t seg_experts = ceil_div(R, kPermuteSegment) * E;
  NVFP4MOE_REQUIRE(R <= kNoAllocMaxRoutedRows && seg_experts <= kNoAllocMaxSegmentExperts, NVFP4MOE_ERR_UNSUPPORTED,
                   "T*k = %lld routed rows and %lld segment-expert counters exceed the library's static scratch "
                   "(at most %lld routed rows and %lld counters); use moe_permute with a workspace",
                   (long long)R, (long long)seg_experts, (long long)kNoAllocMaxRoutedRows,
                   (long long)kNoAllocMaxSegmentExperts);
  NVFP4MOE_REQUIRE(expert_counts && expert_offsets && row_offsets && perm_to_flat, NVFP4MOE_ERR_INVALID_ARG,
                   "null pointer");
  NVFP4MOE_REQUIRE(T == 0 || (topk_idx && xq && xs && flat_to_perm && a_packed && a_scales),
                   NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(T == 0 || (aligned16(xq) && aligned16(a_packed) && aligned16(a_scales) &&
                              (reinterpret_cast<uintptr_t>(xs) & 3) == 0),
                   NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  int32_t* scratch = nullptr;
  if (int st = permute_scratch_address(stream, &scratch)) return st;
  return cuda_status(launch_permute_static_scratch(scratch, topk_idx, T, E, k, xq, xs, H, expert_counts,
                                                   expert_offsets, row_offsets, perm_to_flat, flat_to_perm, a_packed,
                                                   a_scales, moe_permute_rows_capacity(T, E, k), d.num_sms, stream),
                     "permute (static scratch) launch");
}

// ---- a1 + a2 + a3 -----------------------------------------------------------
size_t moe_prepare_workspace_size(int T, int E, int k) {
  if (T < 0 || E < 1 || k < 1) return 0;
  return size_t(prepare_layout(T, E, k).bytes);
}

static int prepare_common(bool mx, const float* logits, const float* bias, const void* x_bf16, int T, int E, int k,
                          int k_primary, int H, int score_fn, int renormalize, int32_t* topk_idx, float* topk_w,
                          float* x_gscale, uint8_t* xq, uint8_t* xs, int32_t* expert_counts, int32_t* expert_offsets,
                          int32_t* row_offsets, int32_t* perm_to_flat, int32_t* flat_to_perm, uint8_t* a_packed,
                          uint8_t* a_scales, void* ws, size_t ws_bytes, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(T >= 0, NVFP4MOE_ERR_INVALID_ARG, "T = %d must be >= 0", T);
  NVFP4MOE_REQUIRE(E >= 1 && E <= 1024, NVFP4MOE_ERR_UNSUPPORTED, "E = %d outside [1, 1024]", E);
  NVFP4MOE_REQUIRE(k >= 1 && k <= E && k <= 32, NVFP4MOE_ERR_UNSUPPORTED, "k = %d outside [1, min(E, 32)]", k);
  NVFP4MOE_REQUIRE(k_primary >= 1 && k_primary <= k, NVFP4MOE_ERR_INVALID_ARG, "k_primary = %d outside [1, k = %d]",
                   k_primary, k);
  const int hq = mx ? 128 : 64;
  NVFP4MOE_REQUIRE(H > 0 && H % hq == 0, NVFP4MOE_ERR_UNSUPPORTED, "H = %d must be a positive multiple of %d", H, hq);
  NVFP4MOE_REQUIRE(int64_t(T) * k <= (int64_t(1) << 30), NVFP4MOE_ERR_UNSUPPORTED, "T*k too large");
  NVFP4MOE_REQUIRE(score_fn == NVFP4MOE_SCORE_SOFTMAX || score_fn == NVFP4MOE_SCORE_SIGMOID,
                   NVFP4MOE_ERR_INVALID_ARG, "score_fn %d", score_fn);
  NVFP4MOE_REQUIRE((mx || x_gscale) && expert_counts && expert_offsets && row_offsets && perm_to_flat,
                   NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(T == 0 || (logits && x_bf16 && topk_idx && topk_w && xq && xs && flat_to_perm && a_packed &&
                              a_scales),
                   NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(T == 0 || (aligned16(x_bf16) && aligned16(xq) && aligned16(a_packed) && aligned16(a_scales) &&
                              (reinterpret_cast<uintptr_t>(xs) & 3) == 0),
                   NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = moe_prepare_workspace_size(T, E, k);
  NVFP4MOE_REQUIRE(ws && ws_bytes >= need, NVFP4MOE_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, need);
  NVFP4MOE_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255) == 0, NVFP4MOE_ERR_INVALID_ARG,
                   "workspace must be 256-byte aligned");
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_prepare(logits, bias, x_bf16, T, E, k, k_primary, H, score_fn, renormalize ? 1 : 0,
                                    topk_idx, topk_w, x_gscale, xq, xs, expert_counts, expert_offsets, row_offsets,
                                    perm_to_flat, flat_to_perm, a_packed, a_scales,
                                    moe_permute_rows_capacity(T, E, k), ws, mx, d.num_sms, stream),
                     "prepare launch");
}

int moe_prepare(const float* logits, const float* bias, const void* x_bf16, int T, int E, int k, int k_primary,
                int H, int score_fn, int renormalize, int32_t* topk_idx, float* topk_w, float* x_gscale, uint8_t* xq,
                uint8_t* xs, int32_t* expert_counts, int32_t* expert_offsets, int32_t* row_offsets,
                int32_t* perm_to_flat, int32_t* flat_to_perm, uint8_t* a_packed, uint8_t* a_scales, void* ws,
                size_t ws_bytes, cudaStream_t stream) {
  return prepare_common(false, logits, bias, x_bf16, T, E, k, k_primary, H, score_fn, renormalize, topk_idx, topk_w,
                        x_gscale, xq, xs, expert_counts, expert_offsets, row_offsets, perm_to_flat, flat_to_perm,
                        a_packed, a_scales, ws, ws_bytes, stream);
}

int moe_prepare_mxfp4(const float* logits, const float* bias, const void* x_bf16, int T, int E, int k,
                      int k_primary, int H, int score_fn, int renormalize, int32_t* topk_idx, float* topk_w,
                      uint8_t* xq, uint8_t* xs, int32_t* expert_counts, int32_t* expert_offsets,
                      int32_t* row_offsets, int32_t* perm_to_flat, int32_t* flat_to_perm, uint8_t* a_packed,
                      uint8_t* a_scales, void* ws, size_t ws_bytes, cudaStream_t stream) {
  return prepare_common(true, logits, bias, x_bf16, T, E, k, k_primary, H, score_fn, renormalize, topk_idx, topk_w,
                        nullptr, xq, xs, expert_counts, expert_offsets, row_offsets, perm_to_flat, flat_to_perm,
                        a_packed, a_scales, ws, ws_bytes, stream);
}

// ---- a4/a5 ------------------------------------------------------------------
size_t moe_grouped_gemm_nvfp4_workspace_size(int E, int N, int K, int epilogue) {
  (void)E;
  (void)N;
  (void)K;
  (void)epilogue;
  return kGemmWorkspaceBytes;
}

int nvfp4moe_gemm_tile_choice(int E, int N, int64_t m_total, int tile_n) {
  // tile_n = 0: token-major tiles once experts average kTokenMajorMinRows
  // rows, on CTA pairs from kPairMinRows
  if (tile_n != 0 || N % 256 != 0 || E < 1) return tile_n;
  if (m_total >= kPairMinRows * E) return NVFP4MOE_TILE_TOKEN_MAJOR_PAIR;
  if (m_total >= kTokenMajorMinRows * E) return NVFP4MOE_TILE_TOKEN_MAJOR;
  return 0;
}

static int grouped_gemm_common(bool mx, const uint8_t* a_packed, const uint8_t* a_scales, const float* a_gscale,
                               const int32_t* expert_counts, const int32_t* row_offsets, int E, int64_t rows_capacity,
                               int64_t m_total, const uint8_t* w_packed, const uint8_t* w_scales,
                               const float* w_gscale, int N, int K, int epilogue, const float* c_gscale, void* c_out,
                               uint8_t* c_scales, int tile_n, int w_layout, int32_t min_rows,
                               int32_t max_rows, void* ws, size_t ws_bytes, cudaStream_t stream,
                               const int32_t* perm_to_flat = nullptr, const float* topk_w = nullptr, int T = 0,
                               int k = 0) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(min_rows >= 1 && min_rows <= max_rows, NVFP4MOE_ERR_INVALID_ARG,
                   "expert row range [%d, %d) must have 1 <= min_rows <= max_rows", min_rows, max_rows);
  NVFP4MOE_REQUIRE(w_layout == NVFP4MOE_W_ROWMAJOR || w_layout == NVFP4MOE_W_TILED, NVFP4MOE_ERR_INVALID_ARG,
                   "w_layout %d", w_layout);
  NVFP4MOE_REQUIRE(!ws || (ws_bytes >= kGemmWorkspaceBytes && (reinterpret_cast<uintptr_t>(ws) & 255) == 0),
                   NVFP4MOE_ERR_WORKSPACE, "workspace must be NULL or %zu bytes, 256-byte aligned (got %zu)",
                   kGemmWorkspaceBytes, ws_bytes);
  const int requant = mx ? NVFP4MOE_EPI_SWIGLU_MXFP4 : NVFP4MOE_EPI_SWIGLU_NVFP4;
  const bool fin = epilogue == NVFP4MOE_EPI_FINALIZE_F32;
  NVFP4MOE_REQUIRE(epilogue == NVFP4MOE_EPI_BF16 || epilogue == requant || epilogue == NVFP4MOE_EPI_SWIGLU_F32 ||
                       (fin && !mx && perm_to_flat),
                   NVFP4MOE_ERR_INVALID_ARG, "epilogue %d", epilogue);
  NVFP4MOE_REQUIRE(!fin || (topk_w && T >= 0 && k >= 1 && int64_t(T) * k <= rows_capacity), NVFP4MOE_ERR_INVALID_ARG,
                   "fused finalize needs perm_to_flat, topk_w, T >= 0 and 1 <= k with T*k <= rows_capacity");
  NVFP4MOE_REQUIRE(E >= 1 && E <= 1024, NVFP4MOE_ERR_UNSUPPORTED, "E = %d outside [1, 1024]", E);
  const int kq = mx ? 128 : 64;
  NVFP4MOE_REQUIRE(K >= kq && K % kq == 0, NVFP4MOE_ERR_UNSUPPORTED, "K = %d must be a positive multiple of %d", K,
                   kq);
  const bool swiglu = epilogue != NVFP4MOE_EPI_BF16 && !fin;
  NVFP4MOE_REQUIRE(N > 0 && N % (swiglu ? 256 : 128) == 0, NVFP4MOE_ERR_UNSUPPORTED,
                   "N = %d must be a multiple of %d for this epilogue", N, swiglu ? 256 : 128);
  NVFP4MOE_REQUIRE(int64_t(E) * N < (int64_t(1) << 31), NVFP4MOE_ERR_UNSUPPORTED, "E*N too large");
  NVFP4MOE_REQUIRE(rows_capacity >= 128 && rows_capacity % 128 == 0 && rows_capacity < (int64_t(1) << 31),
                   NVFP4MOE_ERR_INVALID_ARG, "rows_capacity %lld must be a positive multiple of 128",
                   (long long)rows_capacity);
  NVFP4MOE_REQUIRE(m_total >= 0, NVFP4MOE_ERR_INVALID_ARG, "m_total < 0");
  NVFP4MOE_REQUIRE(tile_n == 0 || tile_n == 128 || (!swiglu && tile_n == 256) ||
                       ((tile_n == NVFP4MOE_TILE_TOKEN_MAJOR || tile_n == NVFP4MOE_TILE_TOKEN_MAJOR_PAIR) &&
                        N % 256 == 0),
                   NVFP4MOE_ERR_UNSUPPORTED,
                   "tile_n %d (expected 0, 128, 256 for the bf16 epilogue, or NVFP4MOE_TILE_TOKEN_MAJOR[_PAIR] with "
                   "N %% 256 == 0)",
                   tile_n);
  NVFP4MOE_REQUIRE(a_packed && a_scales && expert_counts && row_offsets && w_packed && w_scales && c_out,
                   NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(mx || (a_gscale && w_gscale), NVFP4MOE_ERR_INVALID_ARG, "null per-tensor scale pointer");
  NVFP4MOE_REQUIRE(epilogue != NVFP4MOE_EPI_SWIGLU_NVFP4 || (c_gscale && c_scales), NVFP4MOE_ERR_INVALID_ARG,
                   "SWIGLU_NVFP4 needs c_gscale and c_scales");
  NVFP4MOE_REQUIRE(epilogue != NVFP4MOE_EPI_SWIGLU_MXFP4 || c_scales, NVFP4MOE_ERR_INVALID_ARG,
                   "SWIGLU_MXFP4 needs c_scales");
  NVFP4MOE_REQUIRE(aligned16(a_packed) && aligned16(a_scales) && aligned16(w_packed) && aligned16(w_scales) &&
                       aligned16(c_out),
                   NVFP4MOE_ERR_INVALID_ARG, "operands must be 16-byte aligned");
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  GemmArgs a;
  a.a_packed = a_packed;
  a.a_scales = a_scales;
  a.a_gscale = a_gscale;
  a.counts = expert_counts;
  a.row_offsets = row_offsets;
  a.E = E;
  a.rows_capacity = rows_capacity;
  a.m_total = m_total;
  a.w_packed = w_packed;
  a.w_scales = w_scales;
  a.w_gscale = w_gscale;
  a.N = N;
  a.K = K;
  a.epilogue = epilogue;
  a.c_gscale = c_gscale;
  a.c_out = c_out;
  a.c_scales = c_scales;
  a.tile_n = nvfp4moe_gemm_tile_choice(E, N, m_total, tile_n);
  a.mx = mx;
  a.w_tiled = w_layout == NVFP4MOE_W_TILED;
  a.sched = ws;
  a.min_rows = min_rows;
  a.max_rows = max_rows;
  a.perm_to_flat = perm_to_flat;
  a.topk_w = topk_w;
  a.k = k;
  return launch_grouped_gemm(a, d.num_sms, d.smem_optin, stream);  // detail already set on failure
}

int moe_grouped_gemm_nvfp4(const uint8_t* a_packed, const uint8_t* a_scales, const float* a_gscale,
                           const int32_t* expert_counts, const int32_t* row_offsets, int E, int64_t rows_capacity,
                           int64_t m_total, const uint8_t* w_packed, const uint8_t* w_scales,
                           const float* w_gscale, int N, int K, int epilogue, const float* c_gscale, void* c_out,
                           uint8_t* c_scales, int tile_n, int w_layout, void* ws, size_t ws_bytes,
                           cudaStream_t stream) {
  return grouped_gemm_common(false, a_packed, a_scales, a_gscale, expert_counts, row_offsets, E, rows_capacity,
                             m_total, w_packed, w_scales, w_gscale, N, K, epilogue, c_gscale, c_out, c_scales, tile_n,
                             w_layout, 1, INT32_MAX, ws, ws_bytes, stream);
}

int moe_grouped_gemm_nvfp4_range(const uint8_t* a_packed, const uint8_t* a_scales, const float* a_gscale,
                                 const int32_t* expert_counts, const int32_t* row_offsets, int E,
                                 int64_t rows_capacity, int64_t m_total, const uint8_t* w_packed,
                                 const uint8_t* w_scales, const float* w_gscale, int N, int K, int epilogue,
                                 const float* c_gscale, void* c_out, uint8_t* c_scales, int tile_n, int w_layout,
                                 int32_t min_rows, int32_t max_rows, void* ws, size_t ws_bytes,
                                 cudaStream_t stream) {
  return grouped_gemm_common(false, a_packed, a_scales, a_gscale, expert_counts, row_offsets, E, rows_capacity,
                             m_total, w_packed, w_scales, w_gscale, N, K, epilogue, c_gscale, c_out, c_scales, tile_n,
                             w_layout, min_rows, max_rows, ws, ws_bytes, stream);
}

int moe_grouped_gemm_mxfp4(const uint8_t* a_packed, const uint8_t* a_scales, const int32_t* expert_counts,
                           const int32_t* row_offsets, int E, int64_t rows_capacity, int64_t m_total,
                           const uint8_t* w_packed, const uint8_t* w_scales, int N, int K, int epilogue, void* c_out,
                           uint8_t* c_scales, int tile_n, int w_layout, void* ws, size_t ws_bytes,
                           cudaStream_t stream) {
  return grouped_gemm_common(true, a_packed, a_scales, nullptr, expert_counts, row_offsets, E, rows_capacity, m_total,
                             w_packed, w_scales, nullptr, N, K, epilogue, nullptr, c_out, c_scales, tile_n, w_layout,
                             1, INT32_MAX, ws, ws_bytes, stream);
}

int moe_grouped_gemm_nvfp4_finalize(const uint8_t* a_packed, const uint8_t* a_scales, const float* a_gscale,
                                    const int32_t* expert_counts, const int32_t* row_offsets, int E,
                                    int64_t rows_capacity, int64_t m_total, const uint8_t* w_packed,
                                    const uint8_t* w_scales, const float* w_gscale, int N, int K,
                                    const int32_t* perm_to_flat, const float* topk_w, int T, int k, float* out_f32,
                                    int tile_n, int w_layout, int32_t min_rows, int32_t max_rows, void* ws,
                                    size_t ws_bytes, cudaStream_t stream) {
  return grouped_gemm_common(false, a_packed, a_scales, a_gscale, expert_counts, row_offsets, E, rows_capacity,
                             m_total, w_packed, w_scales, w_gscale, N, K, NVFP4MOE_EPI_FINALIZE_F32, nullptr, out_f32,
                             nullptr, tile_n, w_layout, min_rows, max_rows, ws, ws_bytes, stream, perm_to_flat, topk_w,
                             T, k);
}

int moe_finalize_f32(float* acc_f32, int T, int H, void* out_bf16, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(T >= 0 && H > 0 && H % 8 == 0, NVFP4MOE_ERR_INVALID_ARG, "T %d H %d (H %% 8 == 0)", T, H);
  NVFP4MOE_REQUIRE(T == 0 || (acc_f32 && out_bf16 && aligned16(acc_f32) && aligned16(out_bf16)),
                   NVFP4MOE_ERR_INVALID_ARG, "null or misaligned pointer");
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_finalize_f32(acc_f32, int64_t(T) * H, out_bf16, d.num_sms, stream),
                     "finalize_f32 launch");
}

int moe_grouped_gemm_mxfp4_range(const uint8_t* a_packed, const uint8_t* a_scales, const int32_t* expert_counts,
                                 const int32_t* row_offsets, int E, int64_t rows_capacity, int64_t m_total,
                                 const uint8_t* w_packed, const uint8_t* w_scales, int N, int K, int epilogue,
                                 void* c_out, uint8_t* c_scales, int tile_n, int w_layout, int32_t min_rows,
                                 int32_t max_rows, void* ws, size_t ws_bytes, cudaStream_t stream) {
  return grouped_gemm_common(true, a_packed, a_scales, nullptr, expert_counts, row_offsets, E, rows_capacity, m_total,
                             w_packed, w_scales, nullptr, N, K, epilogue, nullptr, c_out, c_scales, tile_n, w_layout,
                             min_rows, max_rows, ws, ws_bytes, stream);
}

// ---- a6 ---------------------------------------------------------------------
int moe_finalize(const void* y_bf16, const int32_t* flat_to_perm, const float* topk_w, int T, int k, int H,
                 int64_t rows_capacity, void* out_bf16, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(T >= 0 && k >= 1 && k <= 1024, NVFP4MOE_ERR_INVALID_ARG, "T %d k %d", T, k);
  NVFP4MOE_REQUIRE(H > 0 && H % 8 == 0, NVFP4MOE_ERR_UNSUPPORTED, "H = %d must be a multiple of 8", H);
  NVFP4MOE_REQUIRE(rows_capacity >= 0, NVFP4MOE_ERR_INVALID_ARG, "rows_capacity < 0");
  if (T == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(y_bf16 && flat_to_perm && topk_w && out_bf16, NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(aligned16(y_bf16) && aligned16(out_bf16), NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_finalize(y_bf16, flat_to_perm, topk_w, T, k, H, rows_capacity, out_bf16, stream),
                     "finalize launch");
}

// ---- grouped routing ----------------------------------------------------------
int moe_route_grouped(const float* logits, const float* select_bias, int T, int E, int k, int n_group, int topk_group,
                      int group_best, int score_fn, int renormalize, float scale, int32_t* topk_idx, float* topk_w,
                      cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(T >= 0, NVFP4MOE_ERR_INVALID_ARG, "T = %d must be >= 0", T);
  NVFP4MOE_REQUIRE(E >= 1 && E <= 1024, NVFP4MOE_ERR_UNSUPPORTED, "E = %d outside [1, 1024]", E);
  NVFP4MOE_REQUIRE(k >= 1 && k <= E && k <= 32, NVFP4MOE_ERR_UNSUPPORTED, "k = %d outside [1, min(E, 32)]", k);
  NVFP4MOE_REQUIRE(n_group >= 1 && n_group <= 32 && E % n_group == 0, NVFP4MOE_ERR_UNSUPPORTED,
                   "n_group = %d outside [1, 32] or no divisor of E = %d", n_group, E);
  NVFP4MOE_REQUIRE(topk_group >= 1 && topk_group <= n_group, NVFP4MOE_ERR_INVALID_ARG,
                   "topk_group = %d outside [1, n_group = %d]", topk_group, n_group);
  NVFP4MOE_REQUIRE(k <= topk_group * (E / n_group), NVFP4MOE_ERR_INVALID_ARG, "k = %d experts of %d groups of %d", k,
                   topk_group, E / n_group);
  NVFP4MOE_REQUIRE((group_best == 1 || group_best == 2) && (n_group == 1 || group_best <= E / n_group),
                   NVFP4MOE_ERR_INVALID_ARG, "group_best = %d with groups of %d", group_best, E / n_group);
  NVFP4MOE_REQUIRE(score_fn == NVFP4MOE_SCORE_SOFTMAX || score_fn == NVFP4MOE_SCORE_SIGMOID,
                   NVFP4MOE_ERR_INVALID_ARG, "score_fn %d", score_fn);
  NVFP4MOE_REQUIRE(scale > -1e30f && scale < 1e30f, NVFP4MOE_ERR_INVALID_ARG, "scale must be finite");
  if (T == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(logits && topk_idx && topk_w, NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(select_bias) |
                     reinterpret_cast<uintptr_t>(topk_idx) | reinterpret_cast<uintptr_t>(topk_w)) & 3) == 0,
                   NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_route_grouped(logits, select_bias, T, E, k, n_group, topk_group, group_best,
                                          score_fn == NVFP4MOE_SCORE_SOFTMAX, renormalize != 0, scale, topk_idx, topk_w,
                                          stream),
                     "route_grouped launch");
}

// ---- few tokens -----------------------------------------------------------------
// One 4-bit matrix (or one of each expert) of the few-token calls.
static int check_matrix(const FewMatrix& w, int n_of, const char* name) {
  const int kq = w.mx ? 128 : 64;
  NVFP4MOE_REQUIRE(w.K > 0 && w.K % kq == 0, NVFP4MOE_ERR_UNSUPPORTED, "%s: %d columns, not a positive multiple of %d", name,
                   w.K, kq);
  NVFP4MOE_REQUIRE(w.N > 0 && w.N % n_of == 0, NVFP4MOE_ERR_UNSUPPORTED, "%s: %d rows, not a positive multiple of %d", name,
                   w.N, n_of);
  NVFP4MOE_REQUIRE(w.packed && w.scales && (w.mx || w.gscale), NVFP4MOE_ERR_INVALID_ARG, "%s: null pointer", name);
  NVFP4MOE_REQUIRE(aligned16(w.packed) && aligned16(w.scales) && (reinterpret_cast<uintptr_t>(w.gscale) & 3) == 0,
                   NVFP4MOE_ERR_INVALID_ARG, "%s: misaligned pointer", name);
  return NVFP4MOE_OK;
}

size_t moe_matvec_workspace_size(int T, int N, int K) {
  if (T < 1 || T > kFewMaxTokens || N < 1 || K < 1) return 0;
  return few_matvec_workspace_bytes(T, N, K);
}

static int matvec_common(const void* x, int64_t x_stride, int T, int x_dtype, const FewMatrix& w, int w_layout, void* out,
                         void* ws, size_t ws_bytes, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(T >= 0, NVFP4MOE_ERR_INVALID_ARG, "T = %d must be >= 0", T);
  NVFP4MOE_REQUIRE(T <= kFewMaxTokens, NVFP4MOE_ERR_UNSUPPORTED, "T = %d above %d", T, kFewMaxTokens);
  NVFP4MOE_REQUIRE(x_dtype == NVFP4MOE_X_BF16 || x_dtype == NVFP4MOE_X_FP16, NVFP4MOE_ERR_INVALID_ARG, "x_dtype %d", x_dtype);
  NVFP4MOE_REQUIRE(w_layout == NVFP4MOE_W_ROWMAJOR || w_layout == NVFP4MOE_W_TILED, NVFP4MOE_ERR_INVALID_ARG,
                   "w_layout %d", w_layout);
  if (int st = check_matrix(w, 128, "w")) return st;
  if (T == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(x && out && aligned16(x) && aligned16(out), NVFP4MOE_ERR_INVALID_ARG, "null or misaligned pointer");
  NVFP4MOE_REQUIRE(T == 1 || (x_stride >= 0 && x_stride % 8 == 0), NVFP4MOE_ERR_INVALID_ARG,
                   "x_stride %lld must be a multiple of 8", (long long)x_stride);
  const size_t need = moe_matvec_workspace_size(T, w.N, w.K);
  NVFP4MOE_REQUIRE(need == 0 || (ws && ws_bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255) == 0),
                   NVFP4MOE_ERR_WORKSPACE, "workspace %zu < %zu or not 256-byte aligned", ws_bytes, need);
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_few_matvec(x, T == 1 ? 0 : x_stride, T, x_dtype == NVFP4MOE_X_FP16, w, out, ws, d.num_sms, stream),
                     "matvec launch");
}

int moe_matvec_nvfp4(const void* x, int64_t x_stride, int T, int x_dtype, const uint8_t* w_packed, const uint8_t* w_scales,
                     const float* w_gscale, int N, int K, int w_layout, void* out, void* ws, size_t ws_bytes,
                     cudaStream_t stream) {
  const FewMatrix w = {w_packed, w_scales, w_gscale, N, K, false, w_layout == NVFP4MOE_W_TILED};
  return matvec_common(x, x_stride, T, x_dtype, w, w_layout, out, ws, ws_bytes, stream);
}

int moe_matvec_mxfp4(const void* x, int64_t x_stride, int T, int x_dtype, const uint8_t* w_packed, const uint8_t* w_scales,
                     int N, int K, int w_layout, void* out, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const FewMatrix w = {w_packed, w_scales, nullptr, N, K, true, w_layout == NVFP4MOE_W_TILED};
  return matvec_common(x, x_stride, T, x_dtype, w, w_layout, out, ws, ws_bytes, stream);
}

size_t moe_experts_workspace_size(int T, int k, int H, int I) {
  if (T < 1 || T > kFewMaxTokens || k < 1 || k > 32 || H < 1 || I < 1) return 0;
  return few_experts_workspace_bytes(T, k, H, I);
}

int moe_experts_launches(int T, int k, int H, int I) {
  if (T < 1 || T > kFewMaxTokens || k < 1 || k > 32 || H < 1 || I < 1) return 0;
  return few_experts_launches(T, k, H, I);
}

static int experts_common(const void* x, int64_t x_stride, const int32_t* topk_idx, const float* topk_w, int T, int k, int E,
                          int I, const FewMatrix& gu, const FewMatrix& dn, int w_layout, void* out, void* ws,
                          size_t ws_bytes, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(T >= 0, NVFP4MOE_ERR_INVALID_ARG, "T = %d must be >= 0", T);
  NVFP4MOE_REQUIRE(T <= kFewMaxTokens, NVFP4MOE_ERR_UNSUPPORTED, "T = %d above %d", T, kFewMaxTokens);
  NVFP4MOE_REQUIRE(E >= 1 && E <= 1024, NVFP4MOE_ERR_UNSUPPORTED, "E = %d outside [1, 1024]", E);
  NVFP4MOE_REQUIRE(k >= 1 && k <= 32, NVFP4MOE_ERR_UNSUPPORTED, "k = %d outside [1, 32]", k);
  NVFP4MOE_REQUIRE(I > 0 && I % 128 == 0 && I < (1 << 30), NVFP4MOE_ERR_UNSUPPORTED, "I = %d must be a positive multiple of 128", I);
  NVFP4MOE_REQUIRE(w_layout == NVFP4MOE_W_ROWMAJOR || w_layout == NVFP4MOE_W_TILED, NVFP4MOE_ERR_INVALID_ARG,
                   "w_layout %d", w_layout);
  if (int st = check_matrix(gu, 256, "w_gu")) return st;
  if (int st = check_matrix(dn, 128, "w_d")) return st;
  if (T == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(x && topk_idx && topk_w && out, NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(aligned16(x) && aligned16(out) &&
                       ((reinterpret_cast<uintptr_t>(topk_idx) | reinterpret_cast<uintptr_t>(topk_w)) & 3) == 0,
                   NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  NVFP4MOE_REQUIRE(T == 1 || (x_stride >= 0 && x_stride % 8 == 0), NVFP4MOE_ERR_INVALID_ARG,
                   "x_stride %lld must be a multiple of 8", (long long)x_stride);
  const size_t need = moe_experts_workspace_size(T, k, gu.K, dn.K);
  NVFP4MOE_REQUIRE(ws && ws_bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255) == 0, NVFP4MOE_ERR_WORKSPACE,
                   "workspace %zu < %zu or not 256-byte aligned", ws_bytes, need);
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  return cuda_status(launch_few_experts(x, T == 1 ? 0 : x_stride, topk_idx, topk_w, T, k, E, gu, dn, out, ws,
                                        d.num_sms, stream),
                     "experts launch");
}

int moe_experts_nvfp4(const void* x_bf16, int64_t x_stride, const int32_t* topk_idx, const float* topk_w, int T, int k, int E,
                      int H, int I, const uint8_t* w_gu_packed, const uint8_t* w_gu_scales, const float* w_gu_gscale,
                      const uint8_t* w_d_packed, const uint8_t* w_d_scales, const float* w_d_gscale, int w_layout,
                      void* out_bf16, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const bool tiled = w_layout == NVFP4MOE_W_TILED;
  const FewMatrix gu = {w_gu_packed, w_gu_scales, w_gu_gscale, I < (1 << 30) ? 2 * I : 0, H, false, tiled};
  const FewMatrix dn = {w_d_packed, w_d_scales, w_d_gscale, H, I, false, tiled};
  return experts_common(x_bf16, x_stride, topk_idx, topk_w, T, k, E, I, gu, dn, w_layout, out_bf16, ws, ws_bytes, stream);
}

int moe_experts_mxfp4(const void* x_bf16, int64_t x_stride, const int32_t* topk_idx, const float* topk_w, int T, int k, int E,
                      int H, int I, const uint8_t* w_gu_packed, const uint8_t* w_gu_scales, const uint8_t* w_d_packed,
                      const uint8_t* w_d_scales, int w_layout, void* out_bf16, void* ws, size_t ws_bytes,
                      cudaStream_t stream) {
  const bool tiled = w_layout == NVFP4MOE_W_TILED;
  const FewMatrix gu = {w_gu_packed, w_gu_scales, nullptr, I < (1 << 30) ? 2 * I : 0, H, true, tiled};
  const FewMatrix dn = {w_d_packed, w_d_scales, nullptr, H, I, true, tiled};
  return experts_common(x_bf16, x_stride, topk_idx, topk_w, T, k, E, I, gu, dn, w_layout, out_bf16, ws, ws_bytes, stream);
}

// ---- latent attention ---------------------------------------------------------
// A strided operand of the latent-attention calls: 16-byte aligned rows.
static bool row_aligned(const void* p, int64_t stride) { return aligned16(p) && stride >= 0 && stride % 8 == 0; }
// Rows of 64 values of T tokens x H heads that do not overlap: one dimension's rows lie within a step of the other.
static bool rows_apart(int64_t T, int64_t token_stride, int64_t H, int64_t head_stride) {
  const int64_t heads = H > 1 ? (H - 1) * head_stride + 64 : 64, tokens = T > 1 ? (T - 1) * token_stride + 64 : 64;
  return (H == 1 || head_stride >= 64) && (T == 1 || token_stride >= 64) &&
         (T == 1 || H == 1 || token_stride >= heads || head_stride >= tokens);
}

int mla_append(const void* latent, int64_t latent_stride, const void* k_rope, int64_t k_rope_stride,
               const void* norm_weight, float eps, const int32_t* positions, const int64_t* slots, int T,
               const float* rope_table, int64_t max_positions, int interleaved, int dtype, void* cache,
               int64_t num_slots, void* rows_out, const void* q_rope, int64_t q_token_stride, int64_t q_head_stride,
               int H, void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(T >= 0 && T <= (1 << 30), NVFP4MOE_ERR_INVALID_ARG, "T = %d outside [0, 2^30]", T);
  NVFP4MOE_REQUIRE(H >= 0 && H <= 1024, NVFP4MOE_ERR_UNSUPPORTED, "H = %d outside [0, 1024]", H);
  NVFP4MOE_REQUIRE(dtype == NVFP4MLA_BF16 || dtype == NVFP4MLA_FP16, NVFP4MOE_ERR_INVALID_ARG, "dtype %d", dtype);
  NVFP4MOE_REQUIRE(interleaved == 0 || interleaved == 1, NVFP4MOE_ERR_INVALID_ARG, "interleaved %d", interleaved);
  NVFP4MOE_REQUIRE(num_slots >= 0 && max_positions >= 1, NVFP4MOE_ERR_INVALID_ARG, "num_slots %lld max_positions %lld",
                   (long long)num_slots, (long long)max_positions);
  NVFP4MOE_REQUIRE(!norm_weight || (eps >= 0.0f && eps < 1e30f), NVFP4MOE_ERR_INVALID_ARG,
                   "eps must be finite and not negative");
  if (T == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(latent && k_rope && positions && slots && rope_table && (cache || num_slots == 0),
                   NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(H == 0 || (q_rope && q_out), NVFP4MOE_ERR_INVALID_ARG, "H = %d without q_rope or q_out", H);
  NVFP4MOE_REQUIRE(row_aligned(latent, latent_stride) && row_aligned(k_rope, k_rope_stride),
                   NVFP4MOE_ERR_INVALID_ARG, "latent and k_rope must be 16-byte aligned with strides %% 8 == 0");
  NVFP4MOE_REQUIRE(H == 0 || (row_aligned(q_rope, q_token_stride) && row_aligned(q_rope, q_head_stride) &&
                              row_aligned(q_out, q_out_token_stride) && row_aligned(q_out, q_out_head_stride)),
                   NVFP4MOE_ERR_INVALID_ARG, "q_rope and q_out must be 16-byte aligned with strides %% 8 == 0");
  NVFP4MOE_REQUIRE(aligned16(norm_weight) && aligned16(rope_table) && aligned16(cache) && aligned16(rows_out) &&
                       (reinterpret_cast<uintptr_t>(positions) & 3) == 0 &&
                       (reinterpret_cast<uintptr_t>(slots) & 7) == 0,
                   NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  NVFP4MOE_REQUIRE(mla_append_blocks(T, H) < (int64_t(1) << 31), NVFP4MOE_ERR_UNSUPPORTED,
                   "T * (1 + ceil(H / 16)) = %lld units are more than a grid of 2^31 - 1 blocks takes",
                   (long long)T * (1 + ceil_div(H, 16)));
  NVFP4MOE_REQUIRE(H == 0 || rows_apart(T, q_out_token_stride, H, q_out_head_stride), NVFP4MOE_ERR_INVALID_ARG,
                   "rows of q_out overlap: strides %lld (tokens) and %lld (heads)", (long long)q_out_token_stride,
                   (long long)q_out_head_stride);
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  MlaAppendArgs a;
  a.latent = latent;
  a.latent_stride = latent_stride;
  a.k_rope = k_rope;
  a.k_rope_stride = k_rope_stride;
  a.norm_weight = norm_weight;
  a.eps = eps;
  a.positions = positions;
  a.slots = slots;
  a.T = T;
  a.table = rope_table;
  a.max_positions = max_positions;
  a.interleaved = interleaved != 0;
  a.fp16 = dtype == NVFP4MLA_FP16;
  a.cache = cache;
  a.num_slots = num_slots;
  a.rows_out = rows_out;
  a.q = q_rope;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.H = H;
  a.q_out = q_out;
  a.qo_token_stride = q_out_token_stride;
  a.qo_head_stride = q_out_head_stride;
  return cuda_status(launch_mla_append(a, stream), "mla_append launch");
}

// Whether two arrays share memory.
static bool share(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a_bytes > 0 && b_bytes > 0 && x < y + uint64_t(b_bytes) && y < x + uint64_t(a_bytes);
}

// Whether an array shares memory with one of n rows that lie `step` >= `row` bytes apart.
static bool share_rows(const void* a, int64_t a_bytes, const void* rows, int64_t n, int64_t row, int64_t step) {
  if (n <= 0 || row <= 0 || a_bytes <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(rows);
  if (x + uint64_t(a_bytes) <= y) return false;
  const uint64_t first = x < y + uint64_t(row) ? 0 : (x - y - uint64_t(row)) / uint64_t(step) + 1;   // that ends after a's begin
  return first < uint64_t(n) && y + first * uint64_t(step) < x + uint64_t(a_bytes);
}

int mla_plan(const int32_t* past_lens, const int32_t* new_lens, int B, int page_size, int32_t* block_tables,
             int64_t table_stride, int max_pages, const int32_t* free_pages, int num_free, const int32_t* free_count, int T,
             int32_t* positions, int64_t* slots, int32_t* cu_seqlens, int32_t* seq_lens, int32_t* granted,
             int32_t* free_count_out, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(B >= 0 && T >= 0 && max_pages >= 0 && num_free >= 0, NVFP4MOE_ERR_INVALID_ARG,
                   "B = %d T = %d max_pages = %d num_free = %d", B, T, max_pages, num_free);
  NVFP4MOE_REQUIRE(page_size >= 16 && (page_size & (page_size - 1)) == 0, NVFP4MOE_ERR_UNSUPPORTED,
                   "page_size = %d must be a power of two >= 16", page_size);
  NVFP4MOE_REQUIRE(table_stride >= max_pages, NVFP4MOE_ERR_INVALID_ARG, "table_stride %lld < max_pages %d",
                   (long long)table_stride, max_pages);
  NVFP4MOE_REQUIRE(free_count && free_count_out && cu_seqlens && (free_pages || num_free == 0) &&
                       (T == 0 || (positions && slots)) &&
                       (B == 0 || (past_lens && new_lens && seq_lens && granted && (block_tables || max_pages == 0))),
                   NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  const void* words[] = {past_lens, new_lens, block_tables, free_pages, free_count, positions, cu_seqlens, seq_lens, granted,
                         free_count_out};
  for (const void* w : words)
    NVFP4MOE_REQUIRE((reinterpret_cast<uintptr_t>(w) & 3) == 0, NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  NVFP4MOE_REQUIRE((reinterpret_cast<uintptr_t>(slots) & 7) == 0, NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  struct Array {
    const char* name;
    const void* at;
    int64_t bytes;
  };
  const Array outs[] = {{"positions", positions, int64_t(T) * 4},     {"slots", slots, int64_t(T) * 8},
                        {"cu_seqlens", cu_seqlens, (int64_t(B) + 1) * 4}, {"seq_lens", seq_lens, int64_t(B) * 4},
                        {"granted", granted, int64_t(B) * 4},         {"free_count_out", free_count_out, 4}};
  const Array ins[] = {{"past_lens", past_lens, int64_t(B) * 4},
                       {"new_lens", new_lens, int64_t(B) * 4},
                       {"free_pages", free_pages, int64_t(num_free) * 4},
                       {"free_count", free_count, 4}};
  for (int i = 0; i < 6; ++i) {
    const Array& o = outs[i];
    for (const Array& in : ins)
      NVFP4MOE_REQUIRE(!share(o.at, o.bytes, in.at, in.bytes) ||
                           (o.at == in.at && ((o.at == seq_lens && in.at == past_lens) || (o.at == granted && in.at == new_lens) ||
                                              (o.at == free_count_out && in.at == free_count))),
                       NVFP4MOE_ERR_INVALID_ARG, "%s overlaps %s", o.name, in.name);
    for (int j = 0; j < i; ++j)
      NVFP4MOE_REQUIRE(!share(o.at, o.bytes, outs[j].at, outs[j].bytes), NVFP4MOE_ERR_INVALID_ARG, "%s overlaps %s", o.name,
                       outs[j].name);
    NVFP4MOE_REQUIRE(!share_rows(o.at, o.bytes, block_tables, B, int64_t(max_pages) * 4, table_stride * 4),
                     NVFP4MOE_ERR_INVALID_ARG, "%s overlaps block_tables", o.name);
  }
  for (const Array& in : ins)
    NVFP4MOE_REQUIRE(!share_rows(in.at, in.bytes, block_tables, B, int64_t(max_pages) * 4, table_stride * 4),
                     NVFP4MOE_ERR_INVALID_ARG, "%s overlaps block_tables", in.name);
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  MlaPlanArgs a;
  a.past = past_lens, a.fresh = new_lens;
  a.B = B, a.shift = __builtin_ctz(unsigned(page_size));
  a.tables = block_tables, a.table_stride = table_stride, a.max_pages = max_pages;
  a.free_pages = free_pages, a.num_free = num_free, a.free_count = free_count;
  a.T = T, a.positions = positions, a.slots = slots;
  a.cu_seqlens = cu_seqlens, a.seq_lens = seq_lens, a.granted = granted, a.free_count_out = free_count_out;
  return cuda_status(launch_mla_plan(a, stream), "mla_plan launch");
}

size_t mla_decode_workspace_size(void) { return mla_decode_workspace_bytes(); }

int mla_decode(const void* q, const void* cache, int num_pages, int page_size, const int32_t* block_tables,
               int64_t table_stride, int max_pages, const int32_t* seq_lens, int B, int Sq, int H, float scale,
               int dtype, void* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(B >= 0 && Sq >= 1 && H >= 1 && max_pages >= 0, NVFP4MOE_ERR_INVALID_ARG,
                   "B = %d Sq = %d H = %d max_pages = %d", B, Sq, H, max_pages);
  NVFP4MOE_REQUIRE(int64_t(Sq) * H < (int64_t(1) << 31) && int64_t(B) * Sq * H < (int64_t(1) << 31),
                   NVFP4MOE_ERR_UNSUPPORTED, "B * Sq * H must be below 2^31");
  NVFP4MOE_REQUIRE(dtype == NVFP4MLA_BF16 || dtype == NVFP4MLA_FP16, NVFP4MOE_ERR_INVALID_ARG, "dtype %d", dtype);
  NVFP4MOE_REQUIRE(scale > 0.0f && scale < 1e30f, NVFP4MOE_ERR_INVALID_ARG, "scale must be positive and finite");
  NVFP4MOE_REQUIRE(page_size >= 16 && (page_size & (page_size - 1)) == 0, NVFP4MOE_ERR_UNSUPPORTED,
                   "page_size = %d must be a power of two >= 16", page_size);
  NVFP4MOE_REQUIRE(num_pages >= 1 && int64_t(num_pages) * page_size < (int64_t(1) << 31), NVFP4MOE_ERR_UNSUPPORTED,
                   "num_pages = %d with pages of %d rows: 1 .. 2^31 - 1 rows", num_pages, page_size);
  NVFP4MOE_REQUIRE(table_stride >= max_pages, NVFP4MOE_ERR_INVALID_ARG, "table_stride %lld < max_pages %d",
                   (long long)table_stride, max_pages);
  if (B == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(q && cache && (block_tables || max_pages == 0) && seq_lens && out && lse,
                   NVFP4MOE_ERR_INVALID_ARG, "null pointer");
  NVFP4MOE_REQUIRE(aligned16(q) && aligned16(cache) && aligned16(out) &&
                       ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(block_tables) |
                         reinterpret_cast<uintptr_t>(seq_lens)) & 3) == 0,
                   NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = mla_decode_workspace_bytes();
  NVFP4MOE_REQUIRE(ws && ws_bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255) == 0, NVFP4MOE_ERR_WORKSPACE,
                   "workspace %zu < %zu or not 256-byte aligned", ws_bytes, need);
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  MlaDecodeArgs a;
  a.q = q;
  a.cache = cache;
  a.num_pages = num_pages;
  a.page = page_size;
  a.tables = block_tables;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.lens = seq_lens;
  a.B = B, a.Sq = Sq, a.H = H;
  a.scale = scale;
  a.fp16 = dtype == NVFP4MLA_FP16;
  a.out = out;
  a.lse = lse;
  a.ws = ws;
  return launch_mla_decode(a, d.num_sms, stream);  // detail already set on failure
}

int mla_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_nope,
                int64_t k_nope_token_stride, int64_t k_nope_head_stride, const void* k_rope,
                int64_t k_rope_token_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                const int32_t* cu_q, const int32_t* cu_k, int B, int Tq, int Tk, int H, float scale, int causal,
                int dtype, void* out, float* lse, cudaStream_t stream) {
  t_detail[0] = 0;
  NVFP4MOE_REQUIRE(B >= 0 && Tq >= 0 && Tk >= 0 && H >= 0, NVFP4MOE_ERR_INVALID_ARG, "B = %d Tq = %d Tk = %d H = %d", B,
                   Tq, Tk, H);
  NVFP4MOE_REQUIRE(int64_t(Tq) * H < (int64_t(1) << 31) && int64_t(Tk) * H < (int64_t(1) << 31) &&
                       (int64_t(Tq) / 256 + B) * H < (int64_t(1) << 31),
                   NVFP4MOE_ERR_UNSUPPORTED, "Tq * H, Tk * H and the blocks (Tq / 256 + B) * H must be below 2^31");
  NVFP4MOE_REQUIRE(dtype == NVFP4MLA_BF16 || dtype == NVFP4MLA_FP16, NVFP4MOE_ERR_INVALID_ARG, "dtype %d", dtype);
  NVFP4MOE_REQUIRE(causal == 0 || causal == 1, NVFP4MOE_ERR_INVALID_ARG, "causal %d", causal);
  NVFP4MOE_REQUIRE(scale > 0.0f && scale < 1e30f, NVFP4MOE_ERR_INVALID_ARG, "scale must be positive and finite");
  if (B == 0 || Tq == 0 || H == 0) return NVFP4MOE_OK;
  NVFP4MOE_REQUIRE(q && cu_q && cu_k && out && lse && (Tk == 0 || (k_nope && k_rope && v)), NVFP4MOE_ERR_INVALID_ARG,
                   "null pointer");
  const int64_t strides[7] = {q_token_stride, q_head_stride, k_nope_token_stride, k_nope_head_stride,
                              k_rope_token_stride, v_token_stride, v_head_stride};
  for (int64_t s : strides)
    NVFP4MOE_REQUIRE(s >= 8 && s % 8 == 0 && s < (int64_t(1) << 38), NVFP4MOE_ERR_INVALID_ARG,
                     "stride %lld must be a positive multiple of 8 below 2^38", (long long)s);
  NVFP4MOE_REQUIRE(aligned16(q) && aligned16(k_nope) && aligned16(k_rope) && aligned16(v) && aligned16(out) &&
                       ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(cu_q) |
                         reinterpret_cast<uintptr_t>(cu_k)) & 3) == 0,
                   NVFP4MOE_ERR_INVALID_ARG, "misaligned pointer");
  DeviceInfo d;
  if (int st = current_device(&d)) return st;
  MlaPrefillArgs a;
  a.q = q, a.q_token_stride = q_token_stride, a.q_head_stride = q_head_stride;
  a.k_nope = k_nope, a.kn_token_stride = k_nope_token_stride, a.kn_head_stride = k_nope_head_stride;
  a.k_rope = k_rope, a.kr_token_stride = k_rope_token_stride;
  a.v = v, a.v_token_stride = v_token_stride, a.v_head_stride = v_head_stride;
  // without keys nothing is loaded, but the tensor maps still describe something
  if (Tk == 0) a.k_nope = a.k_rope = a.v = q;
  a.cu_q = cu_q, a.cu_k = cu_k;
  a.B = B, a.Tq = Tq, a.Tk = Tk, a.H = H;
  a.scale = scale;
  a.causal = causal;
  a.fp16 = dtype == NVFP4MLA_FP16;
  a.out = out;
  a.lse = lse;
  return launch_mla_prefill(a, stream);  // detail already set on failure
}

}  // extern "C"
