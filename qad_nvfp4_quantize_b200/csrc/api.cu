// C ABI entry points (include/nvfp4.h): argument validation, the sm_100
// hardware gate, the device status word, and dispatch to the kernels.
#include <atomic>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "kv_attention.cuh"

namespace {

constexpr int kMaxDevices = 64;

// Library-owned device status word (one per device: module globals are
// instantiated on every device that loads the library).
__device__ int g_device_status = 0;

struct DeviceInfo {
  int checked = 0;     // 0 unknown, 1 supported, -1 unsupported
  int num_sms = 0;
  int* status = nullptr;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

nvfp4_status current_device(DeviceInfo** out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return NVFP4_ERR_CUDA;
  if (dev >= kMaxDevices) return NVFP4_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(g_dev_mu);
  DeviceInfo& d = g_dev[dev];
  if (d.checked == 0) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return NVFP4_ERR_CUDA;
    if (major != 10 || minor != 0) {
      d.checked = -1;
    } else {
      void* p = nullptr;
      if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return NVFP4_ERR_CUDA;
      d.status = static_cast<int*>(p);
      d.num_sms = sms;
      d.checked = 1;
    }
  }
  if (d.checked < 0) return NVFP4_ERR_UNSUPPORTED_DEVICE;
  *out = &d;
  return NVFP4_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

nvfp4_status launched(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

// Shapes of the paged KV cache: whole granules, head sizes with a kernel.
bool kv_shape_ok(int page_size, int head_dim) {
  return (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128) &&
         (head_dim == 64 || head_dim == 128);
}
// Token indexes are 32-bit numbers, up to two tiles of 128 behind a sequence's last token.
constexpr int64_t kMostKvTokens = (int64_t(1) << 31) - 256;
bool kv_sizes_ok(int64_t total, int kv_heads, int batch, int table_width, int64_t num_pages, int page_size) {
  return total >= 0 && total < (int64_t(1) << 31) && kv_heads > 0 && kv_heads <= 1024 && batch >= 0 &&
         batch < (1 << 24) && table_width >= 0 && (int64_t)table_width * page_size <= kMostKvTokens &&
         num_pages >= 0 && num_pages < (int64_t(1) << 31);
}
bool pool_ok(int64_t num_pages, int slots, int table_width, int page_size) {
  return num_pages >= 0 && num_pages < (int64_t(1) << 31) - (1 << 16) && slots >= 0 && table_width >= 0 &&
         page_size >= 1 && (int64_t)table_width * page_size < (int64_t(1) << 31) && table_width <= (1 << 23);
}

// Dynamic global scale: amax pass 1 into the workspace.
nvfp4_status run_amax(const void* x, int64_t n, void* ws, size_t ws_bytes, int num_sms, cudaStream_t s,
                      const uint32_t** partial, int* n_partial) {
  if (!ws || ws_bytes < nvfp4_quantize_workspace_bytes(1, 64) || !aligned16(ws)) return NVFP4_ERR_WORKSPACE;
  const int np = nvfp4::amax_partial_count(n, num_sms);
  uint32_t* part = static_cast<uint32_t*>(ws);
  if (nvfp4::launch_amax_partial(x, n, part, np, s) != cudaSuccess) return NVFP4_ERR_CUDA;
  *partial = part;
  *n_partial = np;
  return NVFP4_OK;
}

std::atomic<uint64_t> g_launches{0};

}  // namespace

void nvfp4::note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

cudaError_t nvfp4::allow_dynamic_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);  // the device gate admits kMaxDevices = 64 devices
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

int nvfp4::current_device_context(int* num_sms, int** status) {
  DeviceInfo* d;
  const nvfp4_status st = current_device(&d);
  if (st == NVFP4_OK) {
    *num_sms = d->num_sms;
    *status = d->status;
  }
  return st;
}

extern "C" {

int nvfp4_version(void) { return 200; }

nvfp4_status nvfp4_check_device(void) {
  DeviceInfo* d;
  return current_device(&d);
}

const char* nvfp4_status_string(nvfp4_status s) {
  switch (s) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_INVALID_ARG: return "invalid argument";
    case NVFP4_ERR_UNSUPPORTED_DEVICE: return "unsupported device (NVFP4 needs sm_100)";
    case NVFP4_ERR_CUDA: return "CUDA error";
    case NVFP4_ERR_WORKSPACE: return "workspace missing or too small";
    case NVFP4_ERR_NONFINITE_INPUT: return "non-finite input";
    case NVFP4_ERR_TIMEOUT: return "device wait timed out";
    case NVFP4_ERR_TOO_LARGE: return "input larger than the no-alloc entry point's static scratch (M*K > 2^30)";
    case NVFP4_ERR_BOUNDS: return "a computed index fell outside its buffer (bounds-checking build)";
    case NVFP4_ERR_PAGE: return "KV cache: an index, offset or length outside its cache, table or pool";
    case NVFP4_ERR_NO_PAGES: return "KV cache: too few free pages";
  }
  return "unknown status";
}

size_t nvfp4_scale_bytes(int64_t rows, int64_t K) {
  if (rows < 0 || K <= 0 || K % 64) return 0;
  return (size_t)((rows + 127) / 128) * (size_t)(K / 64) * 512u;
}

size_t nvfp4_quantize_workspace_bytes(int64_t M, int64_t K) {
  (void)M;
  (void)K;
  // partial maxima, then the two grid-barrier words (padded to 256 bytes)
  return (size_t)nvfp4::kMaxPartials * sizeof(uint32_t) + 256;
}

nvfp4_status nvfp4_quantize(const void* x, int64_t M, int64_t K, nvfp4_mode mode, const float* g_in,
                            uint8_t* codes, uint8_t* scales, float* g_out, uint8_t* fos_choice,
                            void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  if (M < 0 || K <= 0 || K % 64 ||
      (mode != NVFP4_MODE_MAX && mode != NVFP4_MODE_FOUR_OVER_SIX && mode != NVFP4_MODE_MSE))
    return NVFP4_ERR_INVALID_ARG;
  if (M > 0 && (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned16(scales)))
    return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const uint32_t* partial = nullptr;
  int np = 0;
  const int m = (int)mode;
  if (!g_in) {
    if (!workspace || workspace_bytes < nvfp4_quantize_workspace_bytes(M, K) || !aligned16(workspace))
      return NVFP4_ERR_WORKSPACE;
    // one launch: amax, grid barrier and quantization with X kept on chip
    const cudaError_t e = nvfp4::launch_quantize_fused(x, M, K, m, static_cast<uint32_t*>(workspace), codes,
                                                       scales, g_out, fos_choice, d->status, d->num_sms, s);
    if (e != cudaErrorNotSupported) return launched(e);
    st = run_amax(x, M * K, workspace, workspace_bytes, d->num_sms, s, &partial, &np);
    if (st != NVFP4_OK) return st;
  }
  return launched(nvfp4::launch_quantize(x, M, K, m, partial, np, g_in, codes, scales, g_out, fos_choice,
                                         d->status, d->num_sms, s));
}

nvfp4_status nvfp4_fake_quant(const void* x, int64_t M, int64_t K, nvfp4_mode mode, const float* g_frozen,
                              const uint8_t* scales_frozen, void* y, void* workspace, size_t workspace_bytes,
                              nvfp4_stream_t stream) {
  if (M < 0 || K <= 0 || K % 64 || (mode != NVFP4_MODE_MAX && mode != NVFP4_MODE_FOUR_OVER_SIX))
    return NVFP4_ERR_INVALID_ARG;
  if (scales_frozen && !g_frozen) return NVFP4_ERR_INVALID_ARG;
  if (M > 0 && (!x || !y || !aligned16(x) || !aligned16(y) || x == y)) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const uint32_t* partial = nullptr;
  int np = 0;
  const bool fos = mode == NVFP4_MODE_FOUR_OVER_SIX;
  if (!g_frozen) {
    if (!workspace || workspace_bytes < nvfp4_quantize_workspace_bytes(M, K) || !aligned16(workspace))
      return NVFP4_ERR_WORKSPACE;
    const cudaError_t e =
        nvfp4::launch_fake_quant_fused(x, M, K, fos, static_cast<uint32_t*>(workspace), y, d->status, d->num_sms, s);
    if (e != cudaErrorNotSupported) return launched(e);
    st = run_amax(x, M * K, workspace, workspace_bytes, d->num_sms, s, &partial, &np);
    if (st != NVFP4_OK) return st;
  }
  return launched(nvfp4::launch_fake_quant(x, M, K, fos, partial, np, g_frozen, scales_frozen, y, d->status,
                                           d->num_sms, s));
}

nvfp4_status nvfp4_gemm(const uint8_t* Aq, const uint8_t* As, const float* ga, const uint8_t* Bq,
                        const uint8_t* Bs, const float* gb, int64_t M, int64_t N, int64_t K, void* C,
                        nvfp4_stream_t stream) {
  if (M < 0 || N <= 0 || K <= 0 || K % 64 || N % 16 || M >= (1ll << 31) || N >= (1ll << 31))
    return NVFP4_ERR_INVALID_ARG;
  if (!Bq || !Bs || !gb || !aligned16(Bq) || !aligned16(Bs)) return NVFP4_ERR_INVALID_ARG;
  if (M > 0 && (!Aq || !As || !ga || !C || !aligned16(Aq) || !aligned16(As) || !aligned16(C)))
    return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(nvfp4::launch_gemm(Aq, As, ga, Bq, Bs, gb, M, N, K, C, d->status, d->num_sms, s));
}

nvfp4_status nvfp4_convert_e2m1(const float* in, int64_t n, uint8_t* out, nvfp4_stream_t stream) {
  if (n < 0 || (n > 0 && (!in || !out))) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  if (n == 0) return NVFP4_OK;
  return launched(nvfp4::launch_convert(in, n, out, false, d->num_sms, reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_convert_e4m3(const float* in, int64_t n, uint8_t* out, nvfp4_stream_t stream) {
  if (n < 0 || (n > 0 && (!in || !out))) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  if (n == 0) return NVFP4_OK;
  return launched(nvfp4::launch_convert(in, n, out, true, d->num_sms, reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_topk_kl(const void* teacher, const void* student, int64_t rows, int64_t V, int k, float* loss,
                           int32_t* idx, float* grad, nvfp4_stream_t stream) {
  if (rows < 0 || V <= 0 || V % 8 || k < 1 || k > V || (grad && !idx)) return NVFP4_ERR_INVALID_ARG;
  if (rows > 0 && (!teacher || !student || !loss || !aligned16(teacher) || !aligned16(student)))
    return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  return launched(nvfp4::launch_topk_kl(teacher, student, rows, V, k, loss, idx, grad, d->status, d->num_sms,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t M, int64_t K,
                              void* y, nvfp4_stream_t stream) {
  if (M < 0 || K <= 0 || K % 64) return NVFP4_ERR_INVALID_ARG;
  if (M > 0 && (!codes || !scales || !g || !y || !aligned16(codes) || !aligned16(y))) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  if (M == 0) return NVFP4_OK;
  return launched(nvfp4::launch_dequantize(codes, scales, g, M, K, y, d->status, d->num_sms, reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_fake_quant_backward(const void* x, const void* grad_y, int64_t M, int64_t K, nvfp4_mode mode,
                                       const float* g_frozen, const uint8_t* scales_frozen, void* grad_x,
                                       void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  if (M < 0 || K <= 0 || K % 64 || (mode != NVFP4_MODE_MAX && mode != NVFP4_MODE_FOUR_OVER_SIX))
    return NVFP4_ERR_INVALID_ARG;
  if (scales_frozen && !g_frozen) return NVFP4_ERR_INVALID_ARG;
  if (M > 0 && (!x || !grad_y || !grad_x || !aligned16(x) || !aligned16(grad_y) || !aligned16(grad_x) ||
                grad_x == x || grad_x == grad_y))
    return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const uint32_t* partial = nullptr;
  int np = 0;
  const bool fos = mode == NVFP4_MODE_FOUR_OVER_SIX;
  if (!g_frozen) {
    if (!workspace || workspace_bytes < nvfp4_quantize_workspace_bytes(M, K) || !aligned16(workspace))
      return NVFP4_ERR_WORKSPACE;
    const cudaError_t e = nvfp4::launch_fake_quant_bwd_fused(x, grad_y, M, K, fos, static_cast<uint32_t*>(workspace),
                                                             grad_x, d->status, d->num_sms, s);
    if (e != cudaErrorNotSupported) return launched(e);
    st = run_amax(x, M * K, workspace, workspace_bytes, d->num_sms, s, &partial, &np);
    if (st != NVFP4_OK) return st;
  }
  return launched(nvfp4::launch_fake_quant_bwd(x, grad_y, M, K, fos, partial, np, g_frozen, scales_frozen, grad_x,
                                               d->status, d->num_sms, s));
}

size_t nvfp4_kv_page_bytes(int page_size, int head_dim) {
  if (!kv_shape_ok(page_size, head_dim)) return 0;
  return (size_t)(page_size / nvfp4::kGranule) * nvfp4::granule_bytes(head_dim);
}

size_t nvfp4_paged_attention_workspace_bytes(void) { return nvfp4::kv_attention_workspace_bytes(); }

size_t nvfp4_kv_compact_workspace_bytes(int64_t num_pages) {
  return num_pages < 0 ? 0 : nvfp4::kv_compact_workspace_bytes(num_pages);
}

nvfp4_status nvfp4_kv_append(const void* k, const void* v, int64_t row_stride, int64_t total, int kv_heads,
                             int head_dim, const int32_t* cu_q, const int32_t* kv_len, int batch,
                             const int32_t* block_table, int table_width, uint8_t* pages, int64_t num_pages,
                             int page_size, const float* k_g, const float* v_g, nvfp4_mode mode,
                             nvfp4_stream_t stream) {
  if (!kv_shape_ok(page_size, head_dim) || !kv_sizes_ok(total, kv_heads, batch, table_width, num_pages, page_size) ||
      (mode != NVFP4_MODE_MAX && mode != NVFP4_MODE_FOUR_OVER_SIX))
    return NVFP4_ERR_INVALID_ARG;
  if (row_stride % 8 || row_stride < (int64_t)kv_heads * head_dim) return NVFP4_ERR_INVALID_ARG;
  if (total > 0 && batch > 0 &&
      (!k || !v || !cu_q || !kv_len || !block_table || !pages || !k_g || !v_g || !aligned16(k) || !aligned16(v) ||
       !aligned16(pages)))
    return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  const nvfp4::KvIndex ix{cu_q, kv_len, block_table, batch, table_width, page_size, kv_heads, total, num_pages,
                           __builtin_ctz(page_size / nvfp4::kGranule)};
  return launched(nvfp4::launch_kv_append(k, v, row_stride, head_dim, ix, pages, k_g, v_g,
                                          mode == NVFP4_MODE_FOUR_OVER_SIX, d->status, d->num_sms,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

static nvfp4_status run_attention(const void* q, int64_t q_stride, int64_t total, int q_heads, int kv_heads,
                                  int head_dim, const int32_t* cu_q, const int32_t* kv_len, int batch,
                                  const int32_t* block_table, int table_width, const uint8_t* pages,
                                  int64_t num_pages, int page_size, const float* k_g, const float* v_g, float scale,
                                  int causal, int64_t window, int64_t max_q, void* out, float* lse, void* workspace,
                                  size_t workspace_bytes, nvfp4_stream_t stream, int64_t wait_cycles, int withheld) {
  if (!kv_shape_ok(page_size, head_dim) || !kv_sizes_ok(total, kv_heads, batch, table_width, num_pages, page_size))
    return NVFP4_ERR_INVALID_ARG;
  if (q_heads <= 0 || q_heads % kv_heads || q_heads / kv_heads > 128) return NVFP4_ERR_INVALID_ARG;
  if (total * (q_heads / kv_heads) >= (int64_t(1) << 30)) return NVFP4_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || scale > 3.0e38f || window < 0 || max_q < 0) return NVFP4_ERR_INVALID_ARG;
  if (q_stride % 8 || q_stride < (int64_t)q_heads * head_dim) return NVFP4_ERR_INVALID_ARG;
  if (total > 0 && batch > 0) {
    if (!q || !cu_q || !kv_len || !block_table || !pages || !k_g || !v_g || !out || !aligned16(q) ||
        !aligned16(pages) || !aligned16(out) || q == out)
      return NVFP4_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < nvfp4::kv_attention_workspace_bytes() || !aligned16(workspace))
      return NVFP4_ERR_WORKSPACE;
  }
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  nvfp4::AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.ix = nvfp4::KvIndex{cu_q, kv_len, block_table, batch, table_width, page_size, kv_heads, total, num_pages,
                           __builtin_ctz(page_size / nvfp4::kGranule)};
  a.pages = pages;
  a.k_g = k_g;
  a.v_g = v_g;
  a.scale = scale;
  a.group = q_heads / kv_heads;
  a.causal = causal != 0;
  // no position exceeds 2^31: a window beyond that hides nothing, and position - window must not pass 64 bits
  a.window = window < (int64_t(1) << 31) ? window : 0;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = d->status;
  a.wait_cycles = wait_cycles;
  a.withheld = withheld;
  return launched(nvfp4::launch_kv_attention(a, head_dim, max_q, workspace, d->num_sms,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_paged_attention(const void* q, int64_t q_stride, int64_t total, int q_heads, int kv_heads,
                                   int head_dim, const int32_t* cu_q, const int32_t* kv_len, int batch,
                                   const int32_t* block_table, int table_width, const uint8_t* pages,
                                   int64_t num_pages, int page_size, const float* k_g, const float* v_g, float scale,
                                   int causal, int64_t window, int64_t max_q, void* out, float* lse, void* workspace,
                                   size_t workspace_bytes, nvfp4_stream_t stream) {
  return run_attention(q, q_stride, total, q_heads, kv_heads, head_dim, cu_q, kv_len, batch, block_table, table_width,
                       pages, num_pages, page_size, k_g, v_g, scale, causal, window, max_q, out, lse, workspace,
                       workspace_bytes, stream, nvfp4::kAttnWaitCycles, 0);
}

nvfp4_status nvfp4_selftest_attention_timeout(const void* q, int64_t q_stride, int64_t total, int q_heads,
                                              int kv_heads, int head_dim, const int32_t* cu_q, const int32_t* kv_len,
                                              int batch, const int32_t* block_table, int table_width,
                                              const uint8_t* pages, int64_t num_pages, int page_size,
                                              const float* k_g, const float* v_g, float scale, int causal,
                                              int64_t window, int64_t max_q, void* out, float* lse, void* workspace,
                                              size_t workspace_bytes, uint64_t timeout_ns, nvfp4_stream_t stream) {
  if (timeout_ns == 0 || timeout_ns > 10000000000ull) return NVFP4_ERR_INVALID_ARG;  // (0, 10 s]
  return run_attention(q, q_stride, total, q_heads, kv_heads, head_dim, cu_q, kv_len, batch, block_table, table_width,
                       pages, num_pages, page_size, k_g, v_g, scale, causal, window, max_q, out, lse, workspace,
                       workspace_bytes, stream, 2 * (int64_t)timeout_ns, 1);  // at about 2 cycles a nanosecond
}

nvfp4_status nvfp4_kv_copy_pages(uint8_t* pages, int64_t num_pages, int64_t page_bytes, const int32_t* src,
                                 const int32_t* dst, int64_t n, nvfp4_stream_t stream) {
  if (num_pages < 0 || page_bytes <= 0 || page_bytes % 16 || page_bytes > (int64_t(1) << 30) || n < 0 ||
      n >= (int64_t(1) << 31))
    return NVFP4_ERR_INVALID_ARG;
  if (n > 0 && (!pages || !src || !dst || !aligned16(pages))) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  return launched(nvfp4::launch_kv_copy(pages, num_pages, page_bytes, src, dst, n, d->status, d->num_sms,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_kv_fork(int32_t* refs, int64_t num_pages, int32_t* block_table, int slots, int table_width,
                           int32_t* seq_len, int page_size, const int32_t* parent, const int32_t* child, int n,
                           int32_t* src, int32_t* dst, nvfp4_stream_t stream) {
  if (!pool_ok(num_pages, slots, table_width, page_size) || n < 0 || n > (1 << 20)) return NVFP4_ERR_INVALID_ARG;
  if (n > 0 && (!refs || !block_table || !seq_len || !parent || !child || !src || !dst || src == dst))
    return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  const nvfp4::PoolArgs a{refs, block_table, seq_len, num_pages, slots, table_width, page_size};
  return launched(nvfp4::launch_kv_fork(a, parent, child, n, src, dst, d->status,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_kv_free(int32_t* refs, int64_t num_pages, int32_t* block_table, int slots, int table_width,
                           int32_t* seq_len, int page_size, const int32_t* which, int n, nvfp4_stream_t stream) {
  if (!pool_ok(num_pages, slots, table_width, page_size) || n < 0) return NVFP4_ERR_INVALID_ARG;
  if (n > 0 && (!refs || !block_table || !seq_len || !which)) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  const nvfp4::PoolArgs a{refs, block_table, seq_len, num_pages, slots, table_width, page_size};
  return launched(nvfp4::launch_kv_free(a, which, n, d->status, reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_kv_compact(const int32_t* refs, int64_t num_pages, const int32_t* block_table, int slots,
                              int table_width, const int32_t* seq_len, int page_size, int32_t* refs_out,
                              int32_t* table_out, int32_t* src, int32_t* dst, int32_t* live, void* workspace,
                              size_t workspace_bytes, nvfp4_stream_t stream) {
  if (!pool_ok(num_pages, slots, table_width, page_size) || num_pages < 1) return NVFP4_ERR_INVALID_ARG;
  if (!refs || !refs_out || !src || !dst || !live || src == dst) return NVFP4_ERR_INVALID_ARG;
  if (slots > 0 && table_width > 0 && (!block_table || !table_out || !seq_len)) return NVFP4_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < nvfp4::kv_compact_workspace_bytes(num_pages)) return NVFP4_ERR_WORKSPACE;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  const nvfp4::PoolArgs a{const_cast<int32_t*>(refs), const_cast<int32_t*>(block_table),
                          const_cast<int32_t*>(seq_len), num_pages, slots, table_width, page_size};
  return launched(nvfp4::launch_kv_compact(a, refs_out, table_out, src, dst, live, workspace, d->status, d->num_sms,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_get_device_status(nvfp4_stream_t stream, int clear, nvfp4_status* out) {
  if (!out) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return NVFP4_ERR_CUDA;
  int v = 0;
  if (cudaMemcpy(&v, d->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (clear && cudaMemset(d->status, 0, sizeof(int)) != cudaSuccess) return NVFP4_ERR_CUDA;
  *out = static_cast<nvfp4_status>(v);
  return NVFP4_OK;
}

uint64_t nvfp4_kernel_launches(void) { return g_launches.load(std::memory_order_relaxed); }

nvfp4_status nvfp4_selftest_gemm_timeout(const uint8_t* Aq, const uint8_t* As, const float* ga, const uint8_t* Bq,
                                          const uint8_t* Bs, const float* gb, int64_t M, int64_t N, int64_t K,
                                          void* C, uint64_t timeout_ns, nvfp4_stream_t stream) {
  if (timeout_ns == 0 || timeout_ns > 10000000000ull) return NVFP4_ERR_INVALID_ARG;  // (0, 10 s]
  if (M <= 0 || N <= 0 || K <= 0 || K % 64 || N % 16 || M >= (1ll << 31) || N >= (1ll << 31))
    return NVFP4_ERR_INVALID_ARG;
  if (!Aq || !As || !ga || !Bq || !Bs || !gb || !C || !aligned16(Aq) || !aligned16(As) || !aligned16(Bq) ||
      !aligned16(Bs) || !aligned16(C))
    return NVFP4_ERR_INVALID_ARG;
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  return launched(nvfp4::launch_gemm(Aq, As, ga, Bq, Bs, gb, M, N, K, C, d->status, d->num_sms,
                                     reinterpret_cast<cudaStream_t>(stream), timeout_ns, 1));
}

nvfp4_status nvfp4_selftest_timeout(uint64_t timeout_ns, nvfp4_stream_t stream) {
  if (timeout_ns > 10000000000ull) return NVFP4_ERR_INVALID_ARG;  // at most 10 s
  DeviceInfo* d;
  nvfp4_status st = current_device(&d);
  if (st != NVFP4_OK) return st;
  return launched(nvfp4::launch_selftest_timeout(timeout_ns, d->status, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
