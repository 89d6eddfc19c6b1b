// qmm_api.cu -- the extern "C" entry points of libqmm.so: argument validation
// (host only, before any CUDA call), device checks and dispatch to the
// kernel launchers. The operations themselves are defined in include/qmm.h.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <mutex>
#include <string>

#include "kv_layout.cuh"
#include "qmm_common.cuh"
#include "qmm_internal.h"

namespace qmm {

static thread_local std::string t_last_error;

qmm_status set_error(qmm_status st, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  t_last_error = buf;
  return st;
}

qmm_status cuda_check(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return QMM_OK;
  return set_error(QMM_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_dev_mu;
DevInfo g_dev[kMaxDevices];
bool g_dev_known[kMaxDevices];

// Attributes of the current device (queried once per device, then cached).
qmm_status current_device(DevInfo *out) {
  int d = -1;
  cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess) return cuda_check(e, "cudaGetDevice");
  if (d < 0 || d >= kMaxDevices) return set_error(QMM_ERR_DEVICE, "device ordinal %d out of range", d);
  {
    std::lock_guard<std::mutex> lock(g_dev_mu);
    if (!g_dev_known[d]) {
      DevInfo info;
      info.device = d;
      e = cudaDeviceGetAttribute(&info.cc_major, cudaDevAttrComputeCapabilityMajor, d);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&info.cc_minor, cudaDevAttrComputeCapabilityMinor, d);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&info.sms, cudaDevAttrMultiProcessorCount, d);
      if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&info.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, d);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&info.l2_bytes, cudaDevAttrL2CacheSize, d);
      if (e != cudaSuccess) return cuda_check(e, "cudaDeviceGetAttribute");
      g_dev[d] = info;
      g_dev_known[d] = true;
    }
    *out = g_dev[d];
  }
  if (out->cc_major != 10 || out->cc_minor != 0)
    return set_error(QMM_ERR_DEVICE, "device %d has compute capability %d.%d; this library is built for sm_100a (10.0)",
                     d, out->cc_major, out->cc_minor);
  return QMM_OK;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Common checks of (M, N, K, block). `max_m` < 0 means unbounded M.
qmm_status check_shape(const char *fn, int64_t M, int64_t N, int64_t K, int block, int64_t max_m) {
  if (block != QMM_BLOCK) return set_error(QMM_ERR_BLOCK, "%s: block=%d, only 32 is supported", fn, block);
  if (M < 0 || N < 0 || K < 0)
    return set_error(QMM_ERR_SHAPE, "%s: negative size M=%lld N=%lld K=%lld", fn, (long long)M, (long long)N,
                     (long long)K);
  if (K % QMM_BLOCK != 0) return set_error(QMM_ERR_SHAPE, "%s: K=%lld is not a multiple of 32", fn, (long long)K);
  if (K > QMM_MAX_K) return set_error(QMM_ERR_SHAPE, "%s: K=%lld exceeds %d", fn, (long long)K, QMM_MAX_K);
  if (max_m >= 0 && M > max_m)
    return set_error(QMM_ERR_SHAPE, "%s: M=%lld exceeds %lld", fn, (long long)M, (long long)max_m);
  if (N > (int64_t(1) << 40)) return set_error(QMM_ERR_SHAPE, "%s: N=%lld too large", fn, (long long)N);
  return QMM_OK;
}

qmm_status check_ptr(const char *fn, const char *name, const void *p, bool needed, uintptr_t align) {
  if (!needed) return QMM_OK;
  if (p == nullptr) return set_error(QMM_ERR_NULL, "%s: %s is NULL", fn, name);
  if (!aligned(p, align))
    return set_error(QMM_ERR_ALIGN, "%s: %s=%p is not %u-byte aligned", fn, name, p, (unsigned)align);
  return QMM_OK;
}

#define QMM_TRY(expr)                  \
  do {                                 \
    qmm_status _st = (expr);           \
    if (_st != QMM_OK) return _st;     \
  } while (0)

qmm_status zero_fill(float *Y, int64_t count, cudaStream_t s) {
  return cuda_check(cudaMemsetAsync(Y, 0, static_cast<size_t>(count) * sizeof(float), s), "cudaMemsetAsync");
}

}  // namespace

static qmm_status q8_gemv_impl(int64_t M, int64_t N, int64_t K, int block, const void *W, const float *X,
                               float *Y, qmm_stream_t stream, uint32_t user_flags) {
  const char *fn = "qmm_q8_gemv";
  t_last_error.clear();
  QMM_TRY(check_shape(fn, M, N, K, block, QMM_MAX_DECODE_M));
  if (user_flags & ~uint32_t(QMM_FLAG_EARLY_WEIGHTS))
    return set_error(QMM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, user_flags);
  if (M == 0 || N == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "W", W, K > 0, 16));
  QMM_TRY(check_ptr(fn, "X", X, K > 0, 16));
  QMM_TRY(check_ptr(fn, "Y", Y, true, 4));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return zero_fill(Y, M * N, s);
  uint32_t flags = kLaunchPdl | ((user_flags & QMM_FLAG_EARLY_WEIGHTS) ? kPrefetchBeforeWait : 0u);
  return launch_q8_gemv(dev, static_cast<int>(M), N, static_cast<int>(K), W, X, Y, s, flags);
}

static qmm_status quantize_q8_0_impl(int64_t M, int64_t K, int block, const float *X, void *XB, qmm_stream_t stream) {
  const char *fn = "qmm_quantize_act_q8_0";
  t_last_error.clear();
  QMM_TRY(check_shape(fn, M, 0, K, block, -1));
  if (M == 0 || K == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "X", X, true, 16));
  QMM_TRY(check_ptr(fn, "XB", XB, true, 16));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  return launch_quantize_act_q8_0(dev, M, static_cast<int>(K), X, static_cast<uint8_t *>(XB),
                                  reinterpret_cast<cudaStream_t>(stream), kLaunchPdl);
}

static qmm_status q8q8_q8_0_impl(int64_t M, int64_t N, int64_t K, int block, const void *W, const void *XB, float *Y,
                                 uint32_t user_flags, qmm_stream_t stream) {
  const char *fn = "qmm_q8q8_gemv_q8_0";
  t_last_error.clear();
  QMM_TRY(check_shape(fn, M, N, K, block, QMM_MAX_DECODE_M));
  if (user_flags & ~uint32_t(QMM_FLAG_EARLY_WEIGHTS))
    return set_error(QMM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, user_flags);
  if (M == 0 || N == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "W", W, K > 0, 16));
  QMM_TRY(check_ptr(fn, "XB", XB, K > 0, 16));
  QMM_TRY(check_ptr(fn, "Y", Y, true, 4));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return zero_fill(Y, M * N, s);
  uint32_t flags = kLaunchPdl | ((user_flags & QMM_FLAG_EARLY_WEIGHTS) ? kPrefetchBeforeWait : 0u);
  return launch_q8q8_gemv_q8_0(dev, static_cast<int>(M), N, static_cast<int>(K), W, static_cast<const uint8_t *>(XB),
                               Y, s, flags);
}

static qmm_status auto_impl(int64_t M, int64_t N, int64_t K, int block, const void *W, const float *X, float *Y,
                            int8_t *QX, float *DX, uint32_t user_flags, qmm_stream_t stream) {
  const char *fn = "qmm_q8_gemv_auto";
  t_last_error.clear();
  QMM_TRY(check_shape(fn, M, N, K, block, QMM_MAX_DECODE_M));
  if (user_flags & ~uint32_t(QMM_FLAG_EARLY_WEIGHTS))
    return set_error(QMM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, user_flags);
  if (M == 0 || N == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "W", W, K > 0, 16));
  QMM_TRY(check_ptr(fn, "X", X, K > 0, 16));
  QMM_TRY(check_ptr(fn, "QX", QX, K > 0, 16));
  QMM_TRY(check_ptr(fn, "DX", DX, K > 0, 4));
  QMM_TRY(check_ptr(fn, "Y", Y, true, 4));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return zero_fill(Y, M * N, s);
  uint32_t flags = kLaunchPdl | ((user_flags & QMM_FLAG_EARLY_WEIGHTS) ? kPrefetchBeforeWait : 0u);
  return launch_q8_gemv_auto(dev, static_cast<int>(M), N, static_cast<int>(K), W, X, Y, QX, DX, s, flags);
}

static qmm_status multi_impl(int64_t M, int64_t K, int block, int nproj, const int64_t *N, const void *const *W,
                             const float *X, float *const *Y, uint32_t user_flags, qmm_stream_t stream) {
  const char *fn = "qmm_q8_gemv_multi";
  t_last_error.clear();
  if (nproj < 1 || nproj > QMM_MAX_PROJ) return set_error(QMM_ERR_SHAPE, "%s: nproj=%d outside 1..%d", fn, nproj, QMM_MAX_PROJ);
  if (!N || !W || !Y) return set_error(QMM_ERR_NULL, "%s: N, W and Y arrays are required", fn);
  if (user_flags & ~uint32_t(QMM_FLAG_EARLY_WEIGHTS))
    return set_error(QMM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, user_flags);
  int64_t n[QMM_MAX_PROJ];
  const void *w[QMM_MAX_PROJ];
  float *y[QMM_MAX_PROJ];
  int k = 0;
  for (int i = 0; i < nproj; ++i) {
    QMM_TRY(check_shape(fn, M, N[i], K, block, QMM_MAX_DECODE_M));
    if (N[i] == 0 || M == 0) continue;
    QMM_TRY(check_ptr(fn, "W[i]", W[i], K > 0, 16));
    QMM_TRY(check_ptr(fn, "Y[i]", Y[i], true, 4));
    n[k] = N[i];
    w[k] = W[i];
    y[k] = Y[i];
    ++k;
  }
  if (k == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "X", X, K > 0, 16));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) {
    for (int i = 0; i < k; ++i) QMM_TRY(zero_fill(y[i], M * n[i], s));
    return QMM_OK;
  }
  uint32_t flags = kLaunchPdl | ((user_flags & QMM_FLAG_EARLY_WEIGHTS) ? kPrefetchBeforeWait : 0u);
  return launch_q8_gemv_multi(dev, static_cast<int>(M), static_cast<int>(K), k, n, w, X, y, s, flags);
}

static qmm_status quantize_impl(int64_t M, int64_t K, int block, const float *X, int8_t *QX, float *DX,
                                qmm_stream_t stream) {
  const char *fn = "qmm_quantize_act_q8";
  t_last_error.clear();
  QMM_TRY(check_shape(fn, M, 0, K, block, -1));
  if (M == 0 || K == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "X", X, true, 16));
  QMM_TRY(check_ptr(fn, "QX", QX, true, 16));
  QMM_TRY(check_ptr(fn, "DX", DX, true, 4));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  return launch_quantize_act_q8(dev, M, static_cast<int>(K), X, QX, DX, reinterpret_cast<cudaStream_t>(stream),
                                kLaunchPdl);
}

static qmm_status q8q8_impl(int64_t M, int64_t N, int64_t K, int block, const void *W, const int8_t *QX,
                            const float *DX, float *Y, int32_t *isum, qmm_stream_t stream, uint32_t user_flags) {
  const char *fn = isum ? "qmm_q8q8_block_dots" : "qmm_q8q8_gemv";
  t_last_error.clear();
  QMM_TRY(check_shape(fn, M, N, K, block, QMM_MAX_DECODE_M));
  if (user_flags & ~uint32_t(QMM_FLAG_EARLY_WEIGHTS))
    return set_error(QMM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, user_flags);
  if (M == 0 || N == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "W", W, K > 0, 16));
  QMM_TRY(check_ptr(fn, "QX", QX, K > 0, 16));
  if (isum) {
    QMM_TRY(check_ptr(fn, "isum", isum, K > 0, 4));
  } else {
    QMM_TRY(check_ptr(fn, "DX", DX, K > 0, 4));
    QMM_TRY(check_ptr(fn, "Y", Y, true, 4));
  }
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return isum ? QMM_OK : zero_fill(Y, M * N, s);
  if (isum) return launch_q8q8_block_dots(dev, static_cast<int>(M), N, static_cast<int>(K), W, QX, nullptr, isum, s);
  uint32_t flags = kLaunchPdl | ((user_flags & QMM_FLAG_EARLY_WEIGHTS) ? kPrefetchBeforeWait : 0u);
  return launch_q8q8_gemv(dev, static_cast<int>(M), N, static_cast<int>(K), W, QX, DX, Y, s, flags);
}

static qmm_status q8q8_fused_impl(int64_t M, int64_t N, int64_t K, int block, const void *W, const float *X,
                                  int8_t *QX, float *DX, float *Y, qmm_stream_t stream, uint32_t user_flags) {
  const char *fn = "qmm_q8q8_gemv_fused";
  t_last_error.clear();
  QMM_TRY(check_shape(fn, M, N, K, block, QMM_MAX_DECODE_M));
  if (user_flags & ~uint32_t(QMM_FLAG_EARLY_WEIGHTS))
    return set_error(QMM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, user_flags);
  if (M == 0 || N == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "W", W, K > 0, 16));
  QMM_TRY(check_ptr(fn, "X", X, K > 0, 16));
  QMM_TRY(check_ptr(fn, "QX", QX, K > 0, 16));
  QMM_TRY(check_ptr(fn, "DX", DX, K > 0, 4));
  QMM_TRY(check_ptr(fn, "Y", Y, true, 4));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return zero_fill(Y, M * N, s);
  uint32_t flags = kLaunchPdl | ((user_flags & QMM_FLAG_EARLY_WEIGHTS) ? kPrefetchBeforeWait : 0u);
  return launch_q8q8_gemv_fused(dev, static_cast<int>(M), N, static_cast<int>(K), W, X, QX, DX, Y, s, flags);
}

static qmm_status fused_dots_impl(int64_t M, int64_t N, int64_t K, int block, const void *W, const float *X,
                                  int8_t *QX, float *DX, float *Y, int32_t *isum, qmm_stream_t stream) {
  const char *fn = "qmm_q8q8_gemv_fused_dots";
  t_last_error.clear();
  QMM_TRY(check_shape(fn, M, N, K, block, QMM_MAX_DECODE_M));
  if (M == 0 || N == 0 || K == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "W", W, true, 16));
  QMM_TRY(check_ptr(fn, "X", X, true, 16));
  QMM_TRY(check_ptr(fn, "QX", QX, true, 16));
  QMM_TRY(check_ptr(fn, "DX", DX, true, 4));
  QMM_TRY(check_ptr(fn, "Y", Y, true, 4));
  QMM_TRY(check_ptr(fn, "isum", isum, true, 4));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  return launch_q8q8_gemv_fused_dots(dev, static_cast<int>(M), N, static_cast<int>(K), W, X, QX, DX, Y, isum,
                                     reinterpret_cast<cudaStream_t>(stream));
}

static qmm_status dots_q8_0_impl(int64_t M, int64_t N, int64_t K, int block, const void *W, const void *XB,
                                 int32_t *isum, qmm_stream_t stream) {
  const char *fn = "qmm_q8q8_block_dots_q8_0";
  t_last_error.clear();
  QMM_TRY(check_shape(fn, M, N, K, block, QMM_MAX_DECODE_M));
  if (M == 0 || N == 0 || K == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "W", W, true, 16));
  QMM_TRY(check_ptr(fn, "XB", XB, true, 16));
  QMM_TRY(check_ptr(fn, "isum", isum, true, 4));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  return launch_q8q8_block_dots(dev, static_cast<int>(M), N, static_cast<int>(K), W, nullptr,
                                static_cast<const uint8_t *>(XB), isum, reinterpret_cast<cudaStream_t>(stream));
}

static qmm_status withheld_impl(int kernel, int64_t M, int64_t N, int64_t K, int block, const void *W, const void *X,
                                float *Y, uint64_t wait_ns, qmm_stream_t stream) {
  const char *fn = "qmm_test_withheld_copy";
  t_last_error.clear();
  if (kernel != 0 && kernel != 1) return set_error(QMM_ERR_SHAPE, "%s: kernel=%d, expected 0 or 1", fn, kernel);
  QMM_TRY(check_shape(fn, M, N, K, block, kernel == 0 ? QMM_MAX_DECODE_M : 32));
  if (M < 1 || N < 1 || K < 32) return set_error(QMM_ERR_SHAPE, "%s: M, N must be >= 1 and K >= 32", fn);
  if (wait_ns < 1000 || wait_ns > 2000000000ull)
    return set_error(QMM_ERR_SHAPE, "%s: wait_ns=%llu outside 1e3 .. 2e9", fn, (unsigned long long)wait_ns);
  QMM_TRY(check_ptr(fn, "W", W, true, 16));
  QMM_TRY(check_ptr(fn, "X", X, true, 16));
  QMM_TRY(check_ptr(fn, "Y", Y, true, 4));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (kernel == 0)
    return launch_q8_gemv_withheld(dev, static_cast<int>(M), N, static_cast<int>(K), W, static_cast<const float *>(X), Y,
                                   wait_ns, s);
  return launch_prefill_small_withheld(dev, QMM_Q8_0, M, N, static_cast<int>(K), W, static_cast<const uint16_t *>(X), Y,
                                       wait_ns, s);
}

static qmm_status q4_gemv_impl(int64_t M, int64_t N, int64_t K, int block, const void *W, const float *X, float *Y,
                               uint32_t user_flags, qmm_stream_t stream) {
  const char *fn = "qmm_q4_gemv";
  t_last_error.clear();
  QMM_TRY(check_shape(fn, M, N, K, block, QMM_MAX_DECODE_M));
  if (user_flags & ~uint32_t(QMM_FLAG_EARLY_WEIGHTS))
    return set_error(QMM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, user_flags);
  if (M == 0 || N == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "W", W, K > 0, 16));
  QMM_TRY(check_ptr(fn, "X", X, K > 0, 16));
  QMM_TRY(check_ptr(fn, "Y", Y, true, 4));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return zero_fill(Y, M * N, s);
  uint32_t flags = kLaunchPdl | ((user_flags & QMM_FLAG_EARLY_WEIGHTS) ? kPrefetchBeforeWait : 0u);
  return launch_q4_gemv(dev, static_cast<int>(M), N, static_cast<int>(K), W, X, Y, s, flags);
}

static qmm_status gateup_impl(int64_t M, int64_t N, int64_t K, int block, const void *Wg, const void *Wu,
                              const float *X, float *G, float *U, float *Y, qmm_stream_t stream, bool unfused,
                              uint32_t user_flags) {
  const char *fn = unfused ? "qmm_q4_gateup_unfused" : "qmm_q4_swiglu_gateup";
  t_last_error.clear();
  QMM_TRY(check_shape(fn, M, N, K, block, QMM_MAX_DECODE_M));
  if (user_flags & ~uint32_t(QMM_FLAG_EARLY_WEIGHTS))
    return set_error(QMM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, user_flags);
  if (M == 0 || N == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "Wg", Wg, K > 0, 16));
  QMM_TRY(check_ptr(fn, "Wu", Wu, K > 0, 16));
  QMM_TRY(check_ptr(fn, "X", X, K > 0, 16));
  QMM_TRY(check_ptr(fn, "Y", Y, true, 4));
  if (unfused) {
    QMM_TRY(check_ptr(fn, "G", G, true, 4));
    QMM_TRY(check_ptr(fn, "U", U, true, 4));
  }
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) {
    if (unfused) {
      QMM_TRY(zero_fill(G, M * N, s));
      QMM_TRY(zero_fill(U, M * N, s));
    }
    return zero_fill(Y, M * N, s);
  }
  if (unfused)
    return launch_q4_gateup_unfused(dev, static_cast<int>(M), N, static_cast<int>(K), Wg, Wu, X, G, U, Y, s);
  uint32_t flags = kLaunchPdl | ((user_flags & QMM_FLAG_EARLY_WEIGHTS) ? kPrefetchBeforeWait : 0u);
  return launch_q4_gateup(dev, static_cast<int>(M), N, static_cast<int>(K), Wg, Wu, X, Y, s, flags);
}

static qmm_status prefill_impl(int wtype, int64_t M, int64_t N, int64_t K, int block, const void *W,
                               const uint16_t *X, float *Y, qmm_stream_t stream, uint32_t user_flags) {
  const char *fn = "qmm_quant_matmul_prefill";
  t_last_error.clear();
  if (wtype != QMM_Q8_0 && wtype != QMM_Q4_0) return set_error(QMM_ERR_DTYPE, "%s: unknown weight type %d", fn, wtype);
  QMM_TRY(check_shape(fn, M, N, K, block, -1));
  if (M > (int64_t(1) << 24)) return set_error(QMM_ERR_SHAPE, "%s: M=%lld too large", fn, (long long)M);
  if (user_flags & ~uint32_t(QMM_FLAG_EARLY_WEIGHTS))
    return set_error(QMM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, user_flags);
  if (M == 0 || N == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "W", W, K > 0, 16));
  QMM_TRY(check_ptr(fn, "X", X, K > 0, 16));
  QMM_TRY(check_ptr(fn, "Y", Y, true, 4));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return zero_fill(Y, M * N, s);
  const uint32_t flags = kLaunchPdl | ((user_flags & QMM_FLAG_EARLY_WEIGHTS) ? kPrefetchBeforeWait : 0u);
  return launch_prefill(dev, wtype, M, N, static_cast<int>(K), W, X, Y, s, flags);
}

// ---- quantised key/value cache ---------------------------------------------

// Checks of a cache's form; fills *f.
static qmm_status check_kv_form(const char *fn, int ktype, int vtype, int64_t Hkv, int64_t D, int block, int64_t pages,
                                int64_t page, KvForm *f) {
  if (block != QMM_BLOCK) return set_error(QMM_ERR_BLOCK, "%s: block=%d, only 32 is supported", fn, block);
  for (int t : {ktype, vtype})
    if (t != QMM_Q8_0 && t != QMM_Q4_0) return set_error(QMM_ERR_DTYPE, "%s: unknown cache type %d", fn, t);
  if (Hkv < 1 || Hkv > QMM_KV_MAX_HEADS)
    return set_error(QMM_ERR_SHAPE, "%s: Hkv=%lld outside 1..%d", fn, (long long)Hkv, QMM_KV_MAX_HEADS);
  if (D != 64 && D != 96 && D != 128 && D != 192 && D != 256)
    return set_error(QMM_ERR_SHAPE, "%s: D=%lld is not 64, 96, 128, 192 or 256", fn, (long long)D);
  if (page < 16 || page > 65536 || (page & (page - 1)))
    return set_error(QMM_ERR_SHAPE, "%s: page=%lld is not a power of two from 16 to 65536", fn, (long long)page);
  if (pages < 0 || pages > INT32_MAX)
    return set_error(QMM_ERR_SHAPE, "%s: pages=%lld outside 0..2^31-1", fn, (long long)pages);
  f->nb = static_cast<int>(D / 32);
  f->heads = static_cast<int>(Hkv);
  f->page = static_cast<int>(page);
  f->kq8 = ktype == QMM_Q8_0;
  f->vq8 = vtype == QMM_Q8_0;
  f->pages = pages;
  return QMM_OK;
}

static qmm_status check_dtype(const char *fn, int dtype) {
  if (dtype != QMM_F32 && dtype != QMM_BF16) return set_error(QMM_ERR_DTYPE, "%s: unknown element type %d", fn, dtype);
  return QMM_OK;
}

// Strides in elements: rows have to stay on 16-byte boundaries.
static qmm_status check_stride(const char *fn, const char *name, int64_t stride, int dtype) {
  if (stride < 0 || stride > (int64_t(1) << 40))
    return set_error(QMM_ERR_SHAPE, "%s: stride %s=%lld outside 0..2^40", fn, name, (long long)stride);
  if (stride * (dtype == QMM_F32 ? 4 : 2) % 16)
    return set_error(QMM_ERR_ALIGN, "%s: stride %s=%lld elements is not a multiple of 16 bytes", fn, name,
                     (long long)stride);
  return QMM_OK;
}

static qmm_status kv_write_impl(int ktype, int vtype, int dtype, int64_t T, int64_t Hkv, int64_t D, int block,
                                int64_t pages, int64_t page, const void *K, int64_t k_tok, int64_t k_head,
                                const void *V, int64_t v_tok, int64_t v_head, const int64_t *slots, void *cache,
                                qmm_stream_t stream) {
  const char *fn = "qmm_kv_write";
  t_last_error.clear();
  KvForm f;
  QMM_TRY(check_kv_form(fn, ktype, vtype, Hkv, D, block, pages, page, &f));
  QMM_TRY(check_dtype(fn, dtype));
  if (T < 0 || T > INT32_MAX) return set_error(QMM_ERR_SHAPE, "%s: T=%lld outside 0..2^31-1", fn, (long long)T);
  QMM_TRY(check_stride(fn, "k_tok", k_tok, dtype));
  QMM_TRY(check_stride(fn, "k_head", k_head, dtype));
  QMM_TRY(check_stride(fn, "v_tok", v_tok, dtype));
  QMM_TRY(check_stride(fn, "v_head", v_head, dtype));
  if (T == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "K", K, true, 16));
  QMM_TRY(check_ptr(fn, "V", V, true, 16));
  QMM_TRY(check_ptr(fn, "slots", slots, true, 8));
  QMM_TRY(check_ptr(fn, "cache", cache, pages > 0, 16));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  return launch_kv_write(dev, f, dtype, T, K, k_tok, k_head, V, v_tok, v_head, slots, cache,
                         reinterpret_cast<cudaStream_t>(stream));
}

static qmm_status kv_read_impl(int ktype, int vtype, int dtype, int64_t T, int64_t Hkv, int64_t D, int block,
                               int64_t pages, int64_t page, const int64_t *slots, const void *cache, void *K, void *V,
                               qmm_stream_t stream) {
  const char *fn = "qmm_kv_read";
  t_last_error.clear();
  KvForm f;
  QMM_TRY(check_kv_form(fn, ktype, vtype, Hkv, D, block, pages, page, &f));
  QMM_TRY(check_dtype(fn, dtype));
  if (T < 0 || T > INT32_MAX) return set_error(QMM_ERR_SHAPE, "%s: T=%lld outside 0..2^31-1", fn, (long long)T);
  if (T == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "slots", slots, true, 8));
  QMM_TRY(check_ptr(fn, "cache", cache, pages > 0, 16));
  QMM_TRY(check_ptr(fn, "K", K, true, 16));
  QMM_TRY(check_ptr(fn, "V", V, true, 16));
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  return launch_kv_read(dev, f, dtype, T, slots, cache, K, V, reinterpret_cast<cudaStream_t>(stream));
}

static qmm_status check_kv_queries(const char *fn, int64_t B, int64_t M, int64_t Hq, int64_t Hkv) {
  if (B < 0 || B > QMM_KV_MAX_BATCH)
    return set_error(QMM_ERR_SHAPE, "%s: B=%lld outside 0..%d", fn, (long long)B, QMM_KV_MAX_BATCH);
  if (M < 0 || M > QMM_KV_MAX_QUERIES)
    return set_error(QMM_ERR_SHAPE, "%s: M=%lld outside 0..%d", fn, (long long)M, QMM_KV_MAX_QUERIES);
  if (Hq < 1 || Hq % Hkv != 0 || Hq / Hkv > QMM_KV_MAX_RATIO)
    return set_error(QMM_ERR_SHAPE, "%s: Hq=%lld is not 1..%d times Hkv=%lld", fn, (long long)Hq, QMM_KV_MAX_RATIO,
                     (long long)Hkv);
  return QMM_OK;
}

static qmm_status kv_attn_impl(int ktype, int vtype, int dtype, int64_t B, int64_t M, int64_t Hq, int64_t Hkv,
                               int64_t D, int block, int64_t pages, int64_t page, const void *Q, int64_t q_seq,
                               int64_t q_tok, int64_t q_head, const void *cache, const int32_t *table,
                               int64_t table_stride, int64_t max_pages, const int32_t *lens, float scale,
                               int64_t window, void *Y, void *ws, int64_t ws_bytes, qmm_stream_t stream, const char *fn,
                               uint64_t wait_ns, bool withhold) {
  t_last_error.clear();
  KvForm f;
  QMM_TRY(check_kv_form(fn, ktype, vtype, Hkv, D, block, pages, page, &f));
  QMM_TRY(check_dtype(fn, dtype));
  QMM_TRY(check_kv_queries(fn, B, M, Hq, Hkv));
  QMM_TRY(check_stride(fn, "q_seq", q_seq, dtype));
  QMM_TRY(check_stride(fn, "q_tok", q_tok, dtype));
  QMM_TRY(check_stride(fn, "q_head", q_head, dtype));
  if (max_pages < 0 || max_pages >= (int64_t(1) << 30) / page)
    return set_error(QMM_ERR_SHAPE, "%s: max_pages=%lld with page=%lld reaches 2^30 tokens", fn, (long long)max_pages,
                     (long long)page);
  if (table_stride < 0 || table_stride > (int64_t(1) << 40))
    return set_error(QMM_ERR_SHAPE, "%s: table_stride=%lld outside 0..2^40", fn, (long long)table_stride);
  if (window < 0) return set_error(QMM_ERR_SHAPE, "%s: window=%lld is negative", fn, (long long)window);
  if (!isfinite(scale)) return set_error(QMM_ERR_SHAPE, "%s: scale is not finite", fn);
  if (B == 0 || M == 0) return QMM_OK;
  QMM_TRY(check_ptr(fn, "Q", Q, true, 16));
  QMM_TRY(check_ptr(fn, "cache", cache, pages > 0, 16));
  QMM_TRY(check_ptr(fn, "table", table, max_pages > 0, 4));
  QMM_TRY(check_ptr(fn, "lens", lens, true, 4));
  QMM_TRY(check_ptr(fn, "Y", Y, true, 16));
  QMM_TRY(check_ptr(fn, "ws", ws, true, 16));
  const int64_t need = 4 * kv_attn_workspace_floats(B, static_cast<int>(M), static_cast<int>(Hq),
                                                    static_cast<int>(Hkv), static_cast<int>(D));
  if (ws_bytes < need)
    return set_error(QMM_ERR_SHAPE, "%s: ws_bytes=%lld, %lld are needed", fn, (long long)ws_bytes, (long long)need);
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  KvAttnArgs a{};
  a.q = Q;
  a.cache = static_cast<const uint8_t *>(cache);
  a.table = table;
  a.lens = lens;
  a.out = Y;
  a.ws = static_cast<float *>(ws);
  a.q_seq = q_seq;
  a.q_tok = q_tok;
  a.q_head = q_head;
  a.table_stride = table_stride;
  a.batch = static_cast<int>(B);
  a.m = static_cast<int>(M);
  a.hq = static_cast<int>(Hq);
  a.max_pages = static_cast<int>(max_pages);
  a.window = window >= (int64_t(1) << 30) ? 0 : static_cast<int>(window);  // longer than any sequence: none
  a.scale = scale;
  a.wait_ns = wait_ns;
  a.withhold = withhold;
  return launch_kv_attn(dev, f, dtype, a, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace qmm

using namespace qmm;

extern "C" {

QMM_API qmm_status qmm_q8_gemv(int64_t M, int64_t N, int64_t K, int block, const void *W, const float *X,
                               float *Y, qmm_stream_t stream) {
  return q8_gemv_impl(M, N, K, block, W, X, Y, stream, 0u);
}

QMM_API qmm_status qmm_q8_gemv_ex(int64_t M, int64_t N, int64_t K, int block, const void *W, const float *X,
                                  float *Y, uint32_t flags, qmm_stream_t stream) {
  return q8_gemv_impl(M, N, K, block, W, X, Y, stream, flags);
}

QMM_API qmm_status qmm_quantize_act_q8_0(int64_t M, int64_t K, int block, const float *X, void *XB,
                                         qmm_stream_t stream) {
  return quantize_q8_0_impl(M, K, block, X, XB, stream);
}

QMM_API qmm_status qmm_q8q8_gemv_q8_0(int64_t M, int64_t N, int64_t K, int block, const void *W, const void *XB,
                                      float *Y, uint32_t flags, qmm_stream_t stream) {
  return q8q8_q8_0_impl(M, N, K, block, W, XB, Y, flags, stream);
}

QMM_API qmm_status qmm_q8_gemv_auto(int64_t M, int64_t N, int64_t K, int block, const void *W, const float *X,
                                    float *Y, int8_t *QX, float *DX, uint32_t flags, qmm_stream_t stream) {
  return auto_impl(M, N, K, block, W, X, Y, QX, DX, flags, stream);
}

QMM_API qmm_status qmm_q8_gemv_multi(int64_t M, int64_t K, int block, int nproj, const int64_t *N,
                                     const void *const *W, const float *X, float *const *Y, uint32_t flags,
                                     qmm_stream_t stream) {
  return multi_impl(M, K, block, nproj, N, W, X, Y, flags, stream);
}

QMM_API qmm_status qmm_quantize_act_q8(int64_t M, int64_t K, int block, const float *X, int8_t *QX, float *DX,
                                       qmm_stream_t stream) {
  return quantize_impl(M, K, block, X, QX, DX, stream);
}

QMM_API qmm_status qmm_q8q8_gemv(int64_t M, int64_t N, int64_t K, int block, const void *W, const int8_t *QX,
                                 const float *DX, float *Y, qmm_stream_t stream) {
  return q8q8_impl(M, N, K, block, W, QX, DX, Y, nullptr, stream, 0u);
}

QMM_API qmm_status qmm_q8q8_gemv_ex(int64_t M, int64_t N, int64_t K, int block, const void *W, const int8_t *QX,
                                    const float *DX, float *Y, uint32_t flags, qmm_stream_t stream) {
  return q8q8_impl(M, N, K, block, W, QX, DX, Y, nullptr, stream, flags);
}

QMM_API qmm_status qmm_q8q8_gemv_fused(int64_t M, int64_t N, int64_t K, int block, const void *W, const float *X,
                                       int8_t *QX, float *DX, float *Y, uint32_t flags, qmm_stream_t stream) {
  return q8q8_fused_impl(M, N, K, block, W, X, QX, DX, Y, stream, flags);
}

QMM_API qmm_status qmm_q8q8_block_dots(int64_t M, int64_t N, int64_t K, int block, const void *W, const int8_t *QX,
                                       int32_t *isum, qmm_stream_t stream) {
  return q8q8_impl(M, N, K, block, W, QX, nullptr, nullptr, isum, stream, 0u);
}

QMM_API qmm_status qmm_q8q8_gemv_fused_dots(int64_t M, int64_t N, int64_t K, int block, const void *W,
                                            const float *X, int8_t *QX, float *DX, float *Y, int32_t *isum,
                                            qmm_stream_t stream) {
  return fused_dots_impl(M, N, K, block, W, X, QX, DX, Y, isum, stream);
}

QMM_API qmm_status qmm_q8q8_block_dots_q8_0(int64_t M, int64_t N, int64_t K, int block, const void *W, const void *XB,
                                            int32_t *isum, qmm_stream_t stream) {
  return dots_q8_0_impl(M, N, K, block, W, XB, isum, stream);
}

QMM_API qmm_status qmm_test_withheld_copy(int kernel, int64_t M, int64_t N, int64_t K, int block, const void *W,
                                          const void *X, float *Y, uint64_t wait_ns, qmm_stream_t stream) {
  return withheld_impl(kernel, M, N, K, block, W, X, Y, wait_ns, stream);
}

QMM_API qmm_status qmm_q4_swiglu_gateup(int64_t M, int64_t N, int64_t K, int block, const void *Wg, const void *Wu,
                                        const float *X, float *Y, qmm_stream_t stream) {
  return gateup_impl(M, N, K, block, Wg, Wu, X, nullptr, nullptr, Y, stream, false, 0u);
}

QMM_API qmm_status qmm_q4_swiglu_gateup_ex(int64_t M, int64_t N, int64_t K, int block, const void *Wg,
                                           const void *Wu, const float *X, float *Y, uint32_t flags,
                                           qmm_stream_t stream) {
  return gateup_impl(M, N, K, block, Wg, Wu, X, nullptr, nullptr, Y, stream, false, flags);
}

QMM_API qmm_status qmm_q4_gemv(int64_t M, int64_t N, int64_t K, int block, const void *W, const float *X, float *Y,
                               uint32_t flags, qmm_stream_t stream) {
  return q4_gemv_impl(M, N, K, block, W, X, Y, flags, stream);
}

QMM_API qmm_status qmm_q4_gateup_unfused(int64_t M, int64_t N, int64_t K, int block, const void *Wg, const void *Wu,
                                         const float *X, float *G, float *U, float *Y, qmm_stream_t stream) {
  return gateup_impl(M, N, K, block, Wg, Wu, X, G, U, Y, stream, true, 0u);
}

QMM_API qmm_status qmm_quant_matmul_prefill(int wtype, int64_t M, int64_t N, int64_t K, int block, const void *W,
                                            const uint16_t *X, float *Y, qmm_stream_t stream) {
  return prefill_impl(wtype, M, N, K, block, W, X, Y, stream, 0u);
}

QMM_API qmm_status qmm_quant_matmul_prefill_ex(int wtype, int64_t M, int64_t N, int64_t K, int block, const void *W,
                                               const uint16_t *X, float *Y, uint32_t flags, qmm_stream_t stream) {
  return prefill_impl(wtype, M, N, K, block, W, X, Y, stream, flags);
}

QMM_API qmm_status qmm_prefill_plan(int wtype, int64_t M, int64_t N, int64_t K, int block, int32_t *plan) {
  const char *fn = "qmm_prefill_plan";
  t_last_error.clear();
  if (plan == nullptr) return set_error(QMM_ERR_NULL, "%s: plan is NULL", fn);
  if (wtype != QMM_Q8_0 && wtype != QMM_Q4_0) return set_error(QMM_ERR_DTYPE, "%s: unknown weight type %d", fn, wtype);
  QMM_TRY(check_shape(fn, M, N, K, block, -1));
  if (M < 1 || N < 1 || K < 32) return set_error(QMM_ERR_SHAPE, "%s: M, N must be >= 1 and K >= 32", fn);
  if (M > (int64_t(1) << 24)) return set_error(QMM_ERR_SHAPE, "%s: M=%lld too large", fn, (long long)M);
  DevInfo dev;
  QMM_TRY(current_device(&dev));
  PrefillPlan pl{};
  QMM_TRY(launch_prefill(dev, wtype, M, N, static_cast<int>(K), nullptr, nullptr, nullptr, nullptr, 0u, &pl));
  plan[0] = pl.mt;
  plan[1] = pl.split;
  plan[2] = pl.stages;
  plan[3] = pl.ctas;
  plan[4] = pl.kind;
  return QMM_OK;
}

QMM_API qmm_status qmm_kv_page_bytes(int ktype, int vtype, int64_t Hkv, int64_t D, int block, int64_t page,
                                     int64_t *bytes) {
  const char *fn = "qmm_kv_page_bytes";
  t_last_error.clear();
  if (bytes == nullptr) return set_error(QMM_ERR_NULL, "%s: bytes is NULL", fn);
  KvForm f;
  QMM_TRY(check_kv_form(fn, ktype, vtype, Hkv, D, block, 0, page, &f));
  *bytes = static_cast<int64_t>(f.heads) * (f.page / kKvGroup) * f.group_bytes();
  return QMM_OK;
}

QMM_API qmm_status qmm_kv_write(int ktype, int vtype, int dtype, int64_t T, int64_t Hkv, int64_t D, int block,
                                int64_t pages, int64_t page, const void *K, int64_t k_tok, int64_t k_head,
                                const void *V, int64_t v_tok, int64_t v_head, const int64_t *slots, void *cache,
                                qmm_stream_t stream) {
  return kv_write_impl(ktype, vtype, dtype, T, Hkv, D, block, pages, page, K, k_tok, k_head, V, v_tok, v_head, slots,
                       cache, stream);
}

QMM_API qmm_status qmm_kv_read(int ktype, int vtype, int dtype, int64_t T, int64_t Hkv, int64_t D, int block,
                               int64_t pages, int64_t page, const int64_t *slots, const void *cache, void *K, void *V,
                               qmm_stream_t stream) {
  return kv_read_impl(ktype, vtype, dtype, T, Hkv, D, block, pages, page, slots, cache, K, V, stream);
}

QMM_API qmm_status qmm_kv_attn(int ktype, int vtype, int dtype, int64_t B, int64_t M, int64_t Hq, int64_t Hkv,
                               int64_t D, int block, int64_t pages, int64_t page, const void *Q, int64_t q_seq,
                               int64_t q_tok, int64_t q_head, const void *cache, const int32_t *table,
                               int64_t table_stride, int64_t max_pages, const int32_t *lens, float scale,
                               int64_t window, void *Y, void *ws, int64_t ws_bytes, qmm_stream_t stream) {
  return kv_attn_impl(ktype, vtype, dtype, B, M, Hq, Hkv, D, block, pages, page, Q, q_seq, q_tok, q_head, cache, table,
                      table_stride, max_pages, lens, scale, window, Y, ws, ws_bytes, stream, "qmm_kv_attn", kWaitLimitNs,
                      false);
}

QMM_API qmm_status qmm_test_kv_withheld_copy(int ktype, int vtype, int dtype, int64_t B, int64_t M, int64_t Hq,
                                             int64_t Hkv, int64_t D, int block, int64_t pages, int64_t page,
                                             const void *Q, int64_t q_seq, int64_t q_tok, int64_t q_head,
                                             const void *cache, const int32_t *table, int64_t table_stride,
                                             int64_t max_pages, const int32_t *lens, float scale, int64_t window,
                                             void *Y, void *ws, int64_t ws_bytes, uint64_t wait_ns,
                                             qmm_stream_t stream) {
  const char *fn = "qmm_test_kv_withheld_copy";
  if (wait_ns < 1000 || wait_ns > 2000000000ull)
    return set_error(QMM_ERR_SHAPE, "%s: wait_ns=%llu outside 1e3 .. 2e9", fn, (unsigned long long)wait_ns);
  return kv_attn_impl(ktype, vtype, dtype, B, M, Hq, Hkv, D, block, pages, page, Q, q_seq, q_tok, q_head, cache, table,
                      table_stride, max_pages, lens, scale, window, Y, ws, ws_bytes, stream, fn, wait_ns, true);
}

QMM_API qmm_status qmm_kv_attn_workspace(int64_t B, int64_t M, int64_t Hq, int64_t Hkv, int64_t D, int64_t *bytes) {
  const char *fn = "qmm_kv_attn_workspace";
  t_last_error.clear();
  if (bytes == nullptr) return set_error(QMM_ERR_NULL, "%s: bytes is NULL", fn);
  KvForm f;
  QMM_TRY(check_kv_form(fn, QMM_Q4_0, QMM_Q4_0, Hkv, D, QMM_BLOCK, 0, 16, &f));
  QMM_TRY(check_kv_queries(fn, B, M, Hq, Hkv));
  *bytes = 4 * kv_attn_workspace_floats(B, static_cast<int>(M), static_cast<int>(Hq), static_cast<int>(Hkv),
                                        static_cast<int>(D));
  return QMM_OK;
}

QMM_API const char *qmm_last_error_string(void) { return t_last_error.c_str(); }

QMM_API const char *qmm_version(void) { return "qmm 0.1.0 sm_100a"; }

QMM_API qmm_status qmm_device_status(uint32_t *bits) {
  if (bits == nullptr) return set_error(QMM_ERR_NULL, "qmm_device_status: bits is NULL");
  *bits = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_check(e, "cudaDeviceSynchronize");
  uint32_t b = 0;
  e = q8_gemv_status(&b);
  if (e != cudaSuccess) return cuda_check(e, "status read");
  *bits |= b;
  e = q4_gateup_status(&b);
  if (e != cudaSuccess) return cuda_check(e, "status read");
  *bits |= b;
  e = prefill_status(&b);
  if (e != cudaSuccess) return cuda_check(e, "status read");
  *bits |= b;
  e = kv_cache_status(&b);
  if (e != cudaSuccess) return cuda_check(e, "status read");
  *bits |= b;
  e = kv_attn_status(&b);
  if (e != cudaSuccess) return cuda_check(e, "status read");
  *bits |= b;
  if (*bits) return set_error(QMM_ERR_DEVICE_CHECK, "qmm_device_status: a kernel recorded a failure (bits 0x%x)", *bits);
  return QMM_OK;
}

}  // extern "C"
