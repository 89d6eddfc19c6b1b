// kv_cache.cu -- quantised key/value cache: writing new tokens and reading
// tokens back (include/qmm.h, "Quantised key/value cache"; kv_layout.cuh).
#include <algorithm>

#include "kv_layout.cuh"
#include "qmm_common.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

__device__ uint32_t g_kv_status;

__device__ __forceinline__ float load_elem(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_elem(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_elem(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

struct KvRows {
  int64_t tok, head;  // strides in elements
};

// The token of a slot: its page, group and place, or page -1 for a slot that is
// left out (negative) or does not exist (recorded).
__device__ __forceinline__ int64_t slot_page(const KvForm &f, int64_t slot) {
  if (slot < 0) return -1;
  if (slot >= f.pages * f.page) {
    atomicOr(&g_kv_status, kDevBadIndex);
    return -1;
  }
  return slot / f.page;
}

// One warp per row (token, head, keys or values); lane j holds element j of a block.
template <typename T>
__global__ void __launch_bounds__(256) kv_write_kernel(KvForm f, int64_t rows, const T *K, KvRows ks, const T *V,
                                                       KvRows vs, const int64_t *slots, uint8_t *cache) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t r = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; r < rows; r += nwarps) {
    const bool val = r & 1;
    const int head = static_cast<int>((r >> 1) % f.heads);
    const int64_t tok = (r >> 1) / f.heads;
    const int64_t slot = slots[tok];
    const int64_t pg = slot_page(f, slot);
    if (pg < 0) continue;
    const int in = static_cast<int>(slot - pg * f.page), place = in % kKvGroup;
    const bool q8 = val ? f.vq8 : f.kq8;
    uint8_t *part = cache + f.group_at(pg, head, in / kKvGroup) + (val ? kv_part_bytes(f.nb, f.kq8) : 0);
    const T *row = val ? V + tok * vs.tok + head * vs.head : K + tok * ks.tok + head * ks.head;
    for (int b = 0; b < f.nb; ++b) {
      const float x = load_elem(row + b * 32 + lane);
      const uint32_t mag = __float_as_uint(fabsf(x));
      const uint32_t top = __reduce_max_sync(0xffffffffu, mag);
      int code;
      float d;
      if (q8) {
        d = __fdiv_rn(__uint_as_float(top), 127.0f);
        const float id = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
        code = static_cast<int>(fminf(fmaxf(roundf(__fmul_rn(x, id)), -127.0f), 127.0f));
        part[val ? kv_val_code_at(f.nb, true, place, b, lane) : kv_key_code_at(f.nb, true, place, b, lane)] =
            static_cast<uint8_t>(code);
      } else {
        const uint32_t who = __ballot_sync(0xffffffffu, mag == top);
        const float m = __shfl_sync(0xffffffffu, x, __ffs(who) - 1);
        d = m * -0.125f;
        const float id = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
        code = static_cast<int>(fminf(fmaxf(__fadd_rn(__fmul_rn(x, id), 8.5f), 0.0f), 15.0f));
        const int high = __shfl_down_sync(0xffffffffu, code, 16);
        if (lane < 16)
          part[val ? kv_val_code_at(f.nb, false, place, b, lane) : kv_key_code_at(f.nb, false, place, b, lane)] =
              static_cast<uint8_t>(code | high << 4);
      }
      if (lane == 0)
        *reinterpret_cast<uint16_t *>(part + kv_scale_at(f.nb, q8, place, b)) = __half_as_ushort(__float2half_rn(d));
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) kv_read_kernel(KvForm f, int64_t rows, T *K, T *V, const int64_t *slots,
                                                      const uint8_t *cache) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t r = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; r < rows; r += nwarps) {
    const bool val = r & 1;
    const int head = static_cast<int>((r >> 1) % f.heads);
    const int64_t tok = (r >> 1) / f.heads;
    const int64_t slot = slots[tok];
    const int64_t pg = slot_page(f, slot);
    if (pg < 0) continue;
    const int in = static_cast<int>(slot - pg * f.page), place = in % kKvGroup;
    const bool q8 = val ? f.vq8 : f.kq8;
    const uint8_t *part = cache + f.group_at(pg, head, in / kKvGroup) + (val ? kv_part_bytes(f.nb, f.kq8) : 0);
    T *row = (val ? V : K) + (tok * f.heads + head) * f.nb * 32;
    for (int b = 0; b < f.nb; ++b) {
      const float d = half_bits_to_float(*reinterpret_cast<const uint16_t *>(part + kv_scale_at(f.nb, q8, place, b)));
      const int x = q8 ? lane : lane & 15;
      const uint8_t byte = part[val ? kv_val_code_at(f.nb, q8, place, b, x) : kv_key_code_at(f.nb, q8, place, b, x)];
      const int code = q8 ? static_cast<int8_t>(byte) : (lane < 16 ? byte & 15 : byte >> 4) - 8;
      store_elem(row + b * 32 + lane, static_cast<float>(code) * d);
    }
  }
}

cudaLaunchConfig_t config(const DevInfo &dev, int64_t rows, cudaStream_t stream, cudaLaunchAttribute *attr) {
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(256);
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((rows + 7) / 8, static_cast<int64_t>(dev.sms) * 16)));
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

qmm_status launch_kv_write(const DevInfo &dev, const KvForm &f, int dtype, int64_t T, const void *K, int64_t kst,
                           int64_t ksh, const void *V, int64_t vst, int64_t vsh, const int64_t *slots, void *cache,
                           cudaStream_t stream) {
  const int64_t rows = 2 * T * f.heads;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = config(dev, rows, stream, &attr);
  uint8_t *c = static_cast<uint8_t *>(cache);
  const KvRows ks{kst, ksh}, vs{vst, vsh};
  cudaError_t e =
      dtype == QMM_F32
          ? cudaLaunchKernelEx(&cfg, kv_write_kernel<float>, f, rows, static_cast<const float *>(K), ks,
                               static_cast<const float *>(V), vs, slots, c)
          : cudaLaunchKernelEx(&cfg, kv_write_kernel<__nv_bfloat16>, f, rows, static_cast<const __nv_bfloat16 *>(K), ks,
                               static_cast<const __nv_bfloat16 *>(V), vs, slots, c);
  return cuda_check(e, "kv_write launch");
}

qmm_status launch_kv_read(const DevInfo &dev, const KvForm &f, int dtype, int64_t T, const int64_t *slots,
                          const void *cache, void *K, void *V, cudaStream_t stream) {
  const int64_t rows = 2 * T * f.heads;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = config(dev, rows, stream, &attr);
  const uint8_t *c = static_cast<const uint8_t *>(cache);
  cudaError_t e = dtype == QMM_F32
                      ? cudaLaunchKernelEx(&cfg, kv_read_kernel<float>, f, rows, static_cast<float *>(K),
                                           static_cast<float *>(V), slots, c)
                      : cudaLaunchKernelEx(&cfg, kv_read_kernel<__nv_bfloat16>, f, rows, static_cast<__nv_bfloat16 *>(K),
                                           static_cast<__nv_bfloat16 *>(V), slots, c);
  return cuda_check(e, "kv_read launch");
}

cudaError_t kv_cache_status(uint32_t *bits) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_kv_status, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_kv_status, &zero, sizeof(uint32_t));
  return e;
}

}  // namespace qmm
