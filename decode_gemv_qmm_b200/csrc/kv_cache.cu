// kv_cache.cu -- quantised key/value cache: writing new tokens and reading
// tokens back (include/qmm.h, "Quantised key/value cache"; kv_layout.cuh).
//
// Both move bytes: a row of D elements against its D/2 + D/16 (Q4_0) or D + D/16
// (Q8_0) bytes, with a few operations an element, so memory bounds them once
// every load and store is wide and many are in flight. A thread takes one eighth
// of a 32-block, dims 4q .. 4q+3 and 16+4q .. 16+4q+3 (q < 4): two vectors of
// four elements in the rows, and in the cache one word (keys, Q4_0), two words
// that follow each other (keys, Q8_0) or the same bytes in two places (values);
// the four threads of a block follow each other, the blocks of a row too, so a
// warp's accesses fill whole sectors on either side. Keys and values are the two
// halves of the grid: a warp has one kind only.
#include <algorithm>

#include "kv_layout.cuh"
#include "qmm_common.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

__device__ uint32_t g_kv_status;

// Four elements of a row.
__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float *p, float4 v) { __stcs(reinterpret_cast<float4 *>(p), v); }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  __stcs(reinterpret_cast<uint2 *>(p),
         make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b)));
}

struct KvRows {
  int64_t tok, head;  // strides in elements
};

// What a thread works on: eighth q of block b of the row (token, head).
struct KvItem {
  int64_t tok;
  int head, b, q;
};

template <int NB>
__device__ __forceinline__ KvItem item_of(int64_t i, int heads) {
  KvItem it;
  it.q = static_cast<int>(i & 3);
  const int64_t block = i >> 2, row = block / NB;
  it.b = static_cast<int>(block - row * NB);
  it.tok = row / heads;
  it.head = static_cast<int>(row - it.tok * heads);
  return it;
}

// The part (keys' or values') of the group that a slot's token lies in, and its
// place there; nullptr for a slot that is left out (negative) or does not exist
// (recorded).
__device__ __forceinline__ uint8_t *part_of(const KvForm &f, uint8_t *cache, int64_t slot, int head, bool val, int *place) {
  if (slot < 0) return nullptr;
  const int shift = 31 - __clz(f.page);
  const int64_t pg = slot >> shift;
  if (pg >= f.pages) {
    atomicOr(&g_kv_status, kDevBadIndex);
    return nullptr;
  }
  const int in = static_cast<int>(slot & (f.page - 1));
  *place = in % kKvGroup;
  return cache + f.group_at(pg, head, in / kKvGroup) + (val ? kv_part_bytes(f.nb, f.kq8) : 0);
}

// Offsets of the eighth's bytes: `at`, and for values (the second half of the
// four dims) `at + next`.
template <int NB>
__device__ __forceinline__ int bytes_of(bool q8, bool val, int place, int b, int q, int *next) {
  const KvRun r = kv_run(NB, q8, b);
  if (!val) {
    const int row = 8 * (place >> 3) + 2 * (place & 3) + ((place >> 2) & 1), unit = q8 ? 8 : 4;
    *next = 4;
    return r.first * unit * 64 + ((row * 4 + q) * r.n + b - r.first) * unit;
  }
  const int unit = q8 ? 4 : 2, g = 2 * q;
  const bool halves = r.n * unit == 8;
  *next = r.n * unit;
  return r.first * unit * 128 + (halves ? ((g >> 2) * 64 + place * 4 + (g & 3)) * 8 : (place * 8 + g) * r.n * unit) +
         (b - r.first) * unit;
}

// Four codes as bytes of a word.
__device__ __forceinline__ uint32_t pack4(const int *c) {
  return (c[0] & 0xff) | (c[1] & 0xff) << 8 | (c[2] & 0xff) << 16 | static_cast<uint32_t>(c[3] & 0xff) << 24;
}

template <int NB, typename T>
__global__ void __launch_bounds__(256) kv_write_kernel(KvForm f, int64_t items, const T *K, KvRows ks, const T *V,
                                                       KvRows vs, const int64_t *slots, uint8_t *cache) {
  pdl_launch_dependents();
  pdl_wait();
  const bool val = blockIdx.y;
  const bool q8 = val ? f.vq8 : f.kq8;
  const T *rows = val ? V : K;
  const KvRows st = val ? vs : ks;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  // whole warps take part in a round: the four threads of a block are in one
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i - (threadIdx.x & 31) < items; i += step) {
    const bool there = i < items;
    const KvItem it = item_of<NB>(there ? i : items - 1, f.heads);
    const int64_t slot = __ldg(slots + it.tok);
    const T *row = rows + it.tok * st.tok + it.head * st.head + it.b * 32 + it.q * 4;
    const float4 lo = load4(row), hi = load4(row + 16);
    const float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    int c[8];
    float d;
    if (q8) {
      d = __fdiv_rn(top, 127.0f);
      const float id = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        c[j] = static_cast<int>(fminf(fmaxf(roundf(__fmul_rn(x[j], id)), -127.0f), 127.0f));
    } else {
      // the first of the largest gives the sign: the least of 2 dim + sign
      uint32_t first = 64;
#pragma unroll
      for (int j = 7; j >= 0; --j)
        if (fabsf(x[j]) == top) first = 2 * ((j & 4) * 4 + it.q * 4 + (j & 3)) + (__float_as_uint(x[j]) >> 31);
      first = min(first, __shfl_xor_sync(0xffffffffu, first, 1));
      first = min(first, __shfl_xor_sync(0xffffffffu, first, 2));
      d = first & 1 ? top * 0.125f : top * -0.125f;
      const float id = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        c[j] = static_cast<int>(fminf(fmaxf(__fadd_rn(__fmul_rn(x[j], id), 8.5f), 0.0f), 15.0f));
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] |= c[j + 4] << 4;
    }
    int place = 0;
    uint8_t *part = there ? part_of(f, cache, slot, it.head, val, &place) : nullptr;
    if (part == nullptr) continue;
    int next;
    uint8_t *at = part + bytes_of<NB>(q8, val, place, it.b, it.q, &next);
    if (!val) {
      if (q8)
        *reinterpret_cast<uint2 *>(at) = make_uint2(pack4(c), pack4(c + 4));
      else
        *reinterpret_cast<uint32_t *>(at) = pack4(c);
    } else if (q8) {
      const int a[8] = {c[0], c[1], c[4], c[5], c[2], c[3], c[6], c[7]};
      *reinterpret_cast<uint32_t *>(at) = pack4(a);
      *reinterpret_cast<uint32_t *>(at + next) = pack4(a + 4);
    } else {
      const uint32_t w = pack4(c);
      *reinterpret_cast<uint16_t *>(at) = static_cast<uint16_t>(w);
      *reinterpret_cast<uint16_t *>(at + next) = static_cast<uint16_t>(w >> 16);
    }
    if (it.q == 0)
      *reinterpret_cast<uint16_t *>(part + kv_scale_at(NB, q8, place, it.b)) = __half_as_ushort(__float2half_rn(d));
  }
}

template <int NB, typename T>
__global__ void __launch_bounds__(256) kv_read_kernel(KvForm f, int64_t items, T *K, T *V, const int64_t *slots,
                                                      uint8_t *cache) {
  pdl_launch_dependents();
  pdl_wait();
  const bool val = blockIdx.y;
  const bool q8 = val ? f.vq8 : f.kq8;
  T *rows = val ? V : K;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < items; i += step) {
    const KvItem it = item_of<NB>(i, f.heads);
    int place = 0, next;
    const uint8_t *part = part_of(f, cache, __ldg(slots + it.tok), it.head, val, &place);
    if (part == nullptr) continue;
    const uint8_t *at = part + bytes_of<NB>(q8, val, place, it.b, it.q, &next);
    const float d = half_bits_to_float(*reinterpret_cast<const uint16_t *>(part + kv_scale_at(NB, q8, place, it.b)));
    float x[8];
    if (q8) {
      const uint32_t w0 = *reinterpret_cast<const uint32_t *>(at), w1 = *reinterpret_cast<const uint32_t *>(at + next);
      // values: bytes are dims 0, 1, 16, 17 and 2, 3, 18, 19
      const uint32_t lo = val ? __byte_perm(w0, w1, 0x5410) : w0, hi = val ? __byte_perm(w0, w1, 0x7632) : w1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = static_cast<float>(static_cast<int8_t>(lo >> (8 * j)));
        x[j + 4] = static_cast<float>(static_cast<int8_t>(hi >> (8 * j)));
      }
    } else {
      const uint32_t w = val ? *reinterpret_cast<const uint16_t *>(at) |
                                   static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(at + next)) << 16
                             : *reinterpret_cast<const uint32_t *>(at);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = static_cast<float>(static_cast<int>(w >> (8 * j) & 15) - 8);
        x[j + 4] = static_cast<float>(static_cast<int>(w >> (8 * j + 4) & 15) - 8);
      }
    }
    T *row = rows + (it.tok * f.heads + it.head) * (NB * 32) + it.b * 32 + it.q * 4;
    store4(row, make_float4(x[0] * d, x[1] * d, x[2] * d, x[3] * d));
    store4(row + 16, make_float4(x[4] * d, x[5] * d, x[6] * d, x[7] * d));
  }
}

template <typename... P, typename... A>
cudaError_t launch(const DevInfo &dev, int64_t items, cudaStream_t stream, void (*kernel)(P...), A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(256);
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((items + 255) / 256, static_cast<int64_t>(dev.sms) * 4)), 2);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int NB, typename T>
cudaError_t write_rows(const DevInfo &dev, const KvForm &f, int64_t items, const void *K, KvRows ks, const void *V,
                       KvRows vs, const int64_t *slots, void *cache, cudaStream_t stream) {
  return launch(dev, items, stream, kv_write_kernel<NB, T>, f, items, static_cast<const T *>(K), ks,
                static_cast<const T *>(V), vs, slots, static_cast<uint8_t *>(cache));
}

template <int NB, typename T>
cudaError_t read_rows(const DevInfo &dev, const KvForm &f, int64_t items, const int64_t *slots, const void *cache, void *K,
                      void *V, cudaStream_t stream) {
  return launch(dev, items, stream, kv_read_kernel<NB, T>, f, items, static_cast<T *>(K), static_cast<T *>(V), slots,
                static_cast<uint8_t *>(const_cast<void *>(cache)));
}

// call<NB, element type>(...) for a cache's head size.
#define QMM_KV_FORM(call, ...)                                                                                    \
  (f.nb == 2   ? (dtype == QMM_F32 ? call<2, float>(__VA_ARGS__) : call<2, __nv_bfloat16>(__VA_ARGS__))           \
   : f.nb == 3 ? (dtype == QMM_F32 ? call<3, float>(__VA_ARGS__) : call<3, __nv_bfloat16>(__VA_ARGS__))           \
   : f.nb == 4 ? (dtype == QMM_F32 ? call<4, float>(__VA_ARGS__) : call<4, __nv_bfloat16>(__VA_ARGS__))           \
   : f.nb == 6 ? (dtype == QMM_F32 ? call<6, float>(__VA_ARGS__) : call<6, __nv_bfloat16>(__VA_ARGS__))           \
               : (dtype == QMM_F32 ? call<8, float>(__VA_ARGS__) : call<8, __nv_bfloat16>(__VA_ARGS__)))

}  // namespace

qmm_status launch_kv_write(const DevInfo &dev, const KvForm &f, int dtype, int64_t T, const void *K, int64_t kst,
                           int64_t ksh, const void *V, int64_t vst, int64_t vsh, const int64_t *slots, void *cache,
                           cudaStream_t stream) {
  const KvRows ks{kst, ksh}, vs{vst, vsh};
  const int64_t items = T * f.heads * f.nb * 4;
  return cuda_check(QMM_KV_FORM(write_rows, dev, f, items, K, ks, V, vs, slots, cache, stream), "kv_write launch");
}

qmm_status launch_kv_read(const DevInfo &dev, const KvForm &f, int dtype, int64_t T, const int64_t *slots,
                          const void *cache, void *K, void *V, cudaStream_t stream) {
  const int64_t items = T * f.heads * f.nb * 4;
  return cuda_check(QMM_KV_FORM(read_rows, dev, f, items, slots, cache, K, V, stream), "kv_read launch");
}

cudaError_t kv_cache_status(uint32_t *bits) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_kv_status, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_kv_status, &zero, sizeof(uint32_t));
  return e;
}

}  // namespace qmm
