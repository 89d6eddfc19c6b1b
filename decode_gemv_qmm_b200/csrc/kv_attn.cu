// kv_attn.cu -- decode attention over the quantised key/value cache
// (include/qmm.h, qmm_kv_attn; the cache's bytes: kv_layout.cuh).
#include <algorithm>

#include "kv_layout.cuh"
#include "qmm_common.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

__device__ uint32_t g_attn_status;

__device__ __forceinline__ float load_elem(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_elem(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_elem(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float cached(const KvForm &f, const uint8_t *part, bool val, int place, int b, int lane) {
  const bool q8 = val ? f.vq8 : f.kq8;
  const float d = half_bits_to_float(*reinterpret_cast<const uint16_t *>(part + kv_scale_at(f.nb, q8, place, b)));
  const int x = q8 ? lane : lane & 15;
  const uint8_t byte = part[val ? kv_val_code_at(f.nb, q8, place, b, x) : kv_key_code_at(f.nb, q8, place, b, x)];
  return static_cast<float>(q8 ? static_cast<int8_t>(byte) : (lane < 16 ? byte & 15 : byte >> 4) - 8) * d;
}

// One warp per query row (sequence, token, head): keys one after the other with
// the running maximum and sum of the softmax; lane j holds dim j of each block.
template <typename T>
__global__ void __launch_bounds__(128) kv_attn_kernel(KvForm f, KvAttnArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (row >= static_cast<int64_t>(a.batch) * a.m * a.hq) return;
  const int h = static_cast<int>(row % a.hq), i = static_cast<int>(row / a.hq % a.m);
  const int s = static_cast<int>(row / a.hq / a.m);
  const int head = h / (a.hq / f.heads);
  const T *q = static_cast<const T *>(a.q) + s * a.q_seq + i * a.q_tok + h * a.q_head;
  float qv[8], acc[8];
  for (int b = 0; b < 8; ++b) {
    qv[b] = b < f.nb ? load_elem(q + b * 32 + lane) : 0.0f;
    acc[b] = 0.0f;
  }
  int64_t len = a.lens[s];
  const int64_t most = static_cast<int64_t>(a.max_pages) * f.page;
  if (len < 0 || len > most) {
    atomicOr(&g_attn_status, kDevBadIndex);
    len = len < 0 ? 0 : most;
  }
  const int64_t last = len - a.m + i;
  const int64_t low = a.window > 0 && last - a.window + 1 > 0 ? last - a.window + 1 : 0;
  float top = -INFINITY, sum = 0.0f;
  for (int64_t j = low; j <= last; ++j) {
    const int pg = a.table[s * a.table_stride + j / f.page];
    if (pg < 0 || pg >= f.pages) {
      atomicOr(&g_attn_status, kDevBadIndex);
      continue;
    }
    const int in = static_cast<int>(j % f.page), place = in % kKvGroup;
    const uint8_t *kpart = a.cache + f.group_at(pg, head, in / kKvGroup);
    const uint8_t *vpart = kpart + kv_part_bytes(f.nb, f.kq8);
    float dot = 0.0f;
    for (int b = 0; b < 8; ++b)
      if (b < f.nb) dot = fmaf(qv[b], cached(f, kpart, false, place, b, lane), dot);
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    dot *= a.scale;
    const float next = fmaxf(top, dot), keep = expf(top - next), p = expf(dot - next);
    top = next;
    sum = sum * keep + p;
    for (int b = 0; b < 8; ++b)
      if (b < f.nb) acc[b] = fmaf(p, cached(f, vpart, true, place, b, lane), acc[b] * keep);
  }
  T *out = static_cast<T *>(a.out) + row * f.nb * 32;
  for (int b = 0; b < 8; ++b)
    if (b < f.nb) store_elem(out + b * 32 + lane, sum > 0.0f ? acc[b] / sum : 0.0f);
}

}  // namespace

qmm_status launch_kv_attn(const DevInfo &dev, const KvForm &f, int dtype, const KvAttnArgs &a, cudaStream_t stream) {
  (void)dev;
  const int64_t rows = static_cast<int64_t>(a.batch) * a.m * a.hq;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(128);
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 3) / 4));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_check(dtype == QMM_F32 ? cudaLaunchKernelEx(&cfg, kv_attn_kernel<float>, f, a)
                                     : cudaLaunchKernelEx(&cfg, kv_attn_kernel<__nv_bfloat16>, f, a),
                    "kv_attn launch");
}

int64_t kv_attn_workspace_floats(int64_t batch, int m, int hq, int hkv, int d) {
  (void)batch, (void)m, (void)hq, (void)hkv, (void)d;
  return 8;
}

cudaError_t kv_attn_status(uint32_t *bits) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_attn_status, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(uint32_t));
  return e;
}

}  // namespace qmm
