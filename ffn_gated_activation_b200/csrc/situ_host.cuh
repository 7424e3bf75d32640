// Host code shared by the library's translation units: the last error, the
// launch cap, cached device properties, argument checks and launch helpers.
// One instance of each per library (C++17 inline), none of it exported.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "situ_glu.h"

#include "situ_device.cuh"

#pragma GCC visibility push(hidden)

inline thread_local char tl_last_error[512] = "";

inline situ_status_t fail(situ_status_t status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(tl_last_error, sizeof tl_last_error, fmt, ap);
  va_end(ap);
  return status;
}

inline std::atomic<int> g_max_ctas{0};

constexpr int kMaxDevices = 64;
inline std::atomic<int> g_sm_count[kMaxDevices];

inline situ_status_t device_sm_count(int* sms) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return fail(SITU_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(err));
  if (dev >= 0 && dev < kMaxDevices) {
    const int cached = g_sm_count[dev].load(std::memory_order_relaxed);
    if (cached > 0) {
      *sms = cached;
      return SITU_OK;
    }
  }
  int n = 0;
  err = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess || n <= 0)
    return fail(SITU_ERR_CUDA, "cudaDeviceGetAttribute(SM count): %s", cudaGetErrorString(err));
  if (dev >= 0 && dev < kMaxDevices) g_sm_count[dev].store(n, std::memory_order_relaxed);
  *sms = n;
  return SITU_OK;
}

inline bool finite_positive(double x) { return std::isfinite(x) && x > 0.0; }

inline int elem_size(situ_dtype_t d) { return d == SITU_DTYPE_BF16 ? 2 : 4; }

inline bool valid_dtype(int d) { return d == SITU_DTYPE_BF16 || d == SITU_DTYPE_F32; }

// Byte range [lo, hi) spanned by a row-pitched matrix.
struct Span {
  uintptr_t lo, hi;
};

inline Span matrix_span(const void* base, int64_t rows, int64_t pitch_elems, int64_t width_elems, int es) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
  const uint64_t bytes = (static_cast<uint64_t>(rows - 1) * pitch_elems + width_elems) * es;
  return {lo, lo + bytes};
}

inline bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// rows * pitch + width fits in int64 bytes.
inline bool span_fits(int64_t rows, int64_t pitch, int64_t width, int es) {
  if (width > INT64_MAX / es) return false;  // one row alone
  const int64_t limit = INT64_MAX / es - width;
  return rows <= 1 || (pitch <= limit / (rows - 1));
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Per-call constants of the element arithmetic and the gate's exponent form.
inline void fill_coeffs(double beta, int has_lb, double lb, Coeffs* c, int* gate_mode) {
  const double kLog2eD = 1.4426950408889634;
  c->beta = static_cast<float>(beta);
  c->kt = static_cast<float>(2.0 * kLog2eD / beta);
  c->lb = has_lb ? static_cast<float>(lb) : 1.0f;
  c->inv_lb = has_lb ? static_cast<float>(1.0 / lb) : 1.0f;
  c->ku = has_lb ? static_cast<float>(2.0 * kLog2eD / lb) : 0.0f;
  c->bb = static_cast<float>(has_lb ? beta * lb : beta);
  *gate_mode = beta == 4.0 ? kGateSquare : beta == 2.0 ? kGateEqual : beta == 1.0 ? kGateRoot : kGateGeneric;
}

// CTAs of a kernel that one SM holds, asked of the runtime once per (device,
// kernel, launch shape).
inline situ_status_t ctas_per_sm(const void* kernel, int threads, int smem, int* per_sm) {
  struct Entry {
    int dev;
    const void* kernel;
    int threads, smem, per_sm;
  };
  static std::mutex mu;
  static Entry seen[512];
  static int n_seen = 0;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return fail(SITU_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(err));
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n_seen; ++i) {
    const Entry& e = seen[i];
    if (e.kernel == kernel && e.threads == threads && e.smem == smem && e.dev == dev) {
      *per_sm = e.per_sm;
      return SITU_OK;
    }
  }
  err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, kernel, threads, smem);
  if (err != cudaSuccess || *per_sm <= 0)
    return fail(SITU_ERR_CUDA, "occupancy query: %s", cudaGetErrorString(err));
  if (n_seen < 512) seen[n_seen++] = {dev, kernel, threads, smem, *per_sm};
  return SITU_OK;
}

inline situ_status_t launch_grid(const void* kernel, int threads, int smem, int64_t tokens, int* grid) {
  int sms = 0;
  situ_status_t st = device_sm_count(&sms);
  if (st != SITU_OK) return st;
  int per_sm = 0;
  st = ctas_per_sm(kernel, threads, smem, &per_sm);
  if (st != SITU_OK) return st;
  int64_t g = static_cast<int64_t>(sms) * per_sm;
  const int cap = g_max_ctas.load(std::memory_order_relaxed);
  if (cap > 0 && g > cap) g = cap;
  if (g > tokens) g = tokens;
  *grid = static_cast<int>(g);
  return SITU_OK;
}

// Opt a kernel in to more than 48 KB of dynamic shared memory, once per
// (device, kernel, size).
inline situ_status_t ensure_smem(const void* kernel, int bytes) {
  struct Entry {
    int dev;
    const void* kernel;
    int bytes;
  };
  static std::mutex mu;
  static Entry seen[256];
  static int n_seen = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(SITU_ERR_CUDA, "cudaGetDevice failed");
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n_seen; ++i)
    if (seen[i].dev == dev && seen[i].kernel == kernel && seen[i].bytes >= bytes) return SITU_OK;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err != cudaSuccess) return fail(SITU_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(err));
  if (n_seen < 256) seen[n_seen++] = {dev, kernel, bytes};
  return SITU_OK;
}

inline situ_status_t check_launch(const char* what) {
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return fail(SITU_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(err));
  return SITU_OK;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// The status words of the other translation units' kernels on the current
// device, read (and, with `clear`, reset) after a synchronisation; -1 on a CUDA
// error.
int norm_device_status(int clear);
int moe_device_status(int clear);
int nvfp4_device_status(int clear);

#pragma GCC visibility pop

// This translation unit's status word, as above.
namespace {
[[maybe_unused]] int unit_device_status(int clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_status, sizeof v) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_device_status, &zero, sizeof zero) != cudaSuccess) return -1;
  }
  return v;
}
}  // namespace
