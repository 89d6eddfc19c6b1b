// kv_cache.cu -- quantised key/value cache: writing new tokens and reading
// tokens back (include/qmm.h, "Quantised key/value cache"; kv_layout.cuh).
//
// Both move bytes: a row of D elements against its D/2 + D/16 (Q4_0) or D + D/16
// (Q8_0) bytes, with a few operations an element. A thread takes quarter q of a
// run of blocks (kv_layout.cuh): dims 4q .. 4q+3 and 16+4q .. 16+4q+3 of its 4, 2
// or 1 blocks, which are up to 16 bytes that follow each other in the cache, for
// keys and for values; the four quarters of a run follow each other, so a warp's
// accesses fill whole sectors on either side. Its head, run and quarter stay the
// same over its tokens, so a token costs an address and the conversions (one
// eighth of a block a thread, with every address worked out anew, took 130 us
// where this takes 64 us for 65536 tokens, 8 heads of 128, Q4_0, bf16). Keys
// and values are the two halves of the grid.
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

// Blocks of a launch for each SM (65536 tokens read: 90 us with 2, 67 with 8, 64 with 16).
constexpr int kKvBlocks = 16;

// What a thread works on, the same for all its tokens: quarter q of a run of a head.
struct KvUnit {
  int head, q, first, n;  // the run's first block, its blocks
  int64_t tok, step;      // the thread's first token, and how far the next one is
  bool there;
};

// Units of a token lie on the threads of a block, as many tokens as fit; where
// one token's do not fit, the grid's z counts blocks of them.
template <int NB, bool Q8>
__device__ __forceinline__ KvUnit unit_of(int heads) {
  constexpr int kRuns = kv_runs(NB, Q8);
  const int units = heads * kRuns * 4, per = units <= 256 ? 256 / units : 1;
  const int tid = threadIdx.x, slot = units <= 256 ? tid / units : 0;
  const int u = units <= 256 ? tid - slot * units : blockIdx.z * 256 + tid;
  KvUnit k;
  k.q = u & 3;
  const int run = (u >> 2) % kRuns;
  k.head = (u >> 2) / kRuns;
  k.first = kv_run_first(NB, Q8, run);
  k.n = kv_run_blocks(NB, Q8, run);
  k.tok = static_cast<int64_t>(blockIdx.x) * per + slot;
  k.step = static_cast<int64_t>(gridDim.x) * per;
  k.there = slot < per && u < units && (units > 256 || blockIdx.z == 0);
  return k;
}

// Where a token's bytes of a unit are: the part of its group, and its place there.
// False for a slot that is left out (negative) or does not exist (recorded).
struct KvAt {
  int64_t part;
  int place;
};
__device__ __forceinline__ bool at_slot(const KvForm &f, int64_t slot, int head, bool val, KvAt *at) {
  if (slot < 0) return false;
  const int shift = 31 - __clz(f.page);
  const int64_t pg = slot >> shift;
  if (pg >= f.pages) {
    atomicOr(&g_kv_status, kDevBadIndex);
    return false;
  }
  const int in = static_cast<int>(slot) & (f.page - 1);
  at->place = in % kKvGroup;
  at->part = f.group_at(pg, head, in / kKvGroup) + (val ? kv_part_bytes(f.nb, f.kq8) : 0);
  return true;
}

// Offset in the part of a unit's bytes, n * (Q8 ? 8 : 4) of them.
template <bool Q8>
__device__ __forceinline__ int unit_at(const KvUnit &k, bool val, int place) {
  constexpr int kBytes = Q8 ? 8 : 4;  // of a quarter block
  const int base = k.first * kBytes * 64;
  if (!val) return base + ((8 * (place >> 3) + 2 * (place & 3) + ((place >> 2) & 1)) * 4 + k.q) * k.n * kBytes;
  if (k.n * kBytes == 16) return base + ((k.q >> 1) * 32 + place * 2 + (k.q & 1)) * 16;
  return base + (place * 4 + k.q) * k.n * kBytes;
}

// A unit's words, by blocks: Q4_0 one of a block (low nibbles dims 4q + e, high
// ones 16 + 4q + e, byte e), Q8_0 two (dims 4q + e; 16 + 4q + e). Values lie by
// pairs of dims, so the halves of two words are exchanged, either way.
template <bool Q8>
__device__ __forceinline__ void by_blocks(uint32_t (&w)[4], int n, bool val) {
  if (!val) return;
  const uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
  if (Q8) {
    if (n == 2)
      w[0] = __byte_perm(a, c, 0x5410), w[1] = __byte_perm(a, c, 0x7632), w[2] = __byte_perm(b, d, 0x5410), w[3] = __byte_perm(b, d, 0x7632);
    else
      w[0] = __byte_perm(a, b, 0x5410), w[1] = __byte_perm(a, b, 0x7632);
  } else if (n == 4) {
    w[0] = __byte_perm(a, c, 0x5410), w[1] = __byte_perm(a, c, 0x7632), w[2] = __byte_perm(b, d, 0x5410), w[3] = __byte_perm(b, d, 0x7632);
  } else if (n == 2) {
    w[0] = __byte_perm(a, b, 0x5410), w[1] = __byte_perm(a, b, 0x7632);
  }
}
template <bool Q8>
__device__ __forceinline__ void by_pairs(uint32_t (&w)[4], int n, bool val) {
  if (!val) return;
  const uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
  if (n == (Q8 ? 2 : 4))
    w[0] = __byte_perm(a, b, 0x5410), w[2] = __byte_perm(a, b, 0x7632), w[1] = __byte_perm(c, d, 0x5410), w[3] = __byte_perm(c, d, 0x7632);
  else if (Q8 || n == 2)
    w[0] = __byte_perm(a, b, 0x5410), w[1] = __byte_perm(a, b, 0x7632);
}

// 16384 tokens, 8 heads of 128, Q4_0, bf16: 28.0 us, 2.1 times the bytes' 13.1 (29.2
// with the sums one by one; 29.3 with bf16 extremes in pairs). Neither memory (28% of
// its rate) nor issue slots (54%) are full: 80 registers leave three blocks an SM, and
// a thread waits for all its loads before it converts.
template <int NB, bool Q8, typename T>
__device__ __forceinline__ void write_units(const KvForm &f, int64_t tokens, const T *rows, KvRows st, bool val,
                                            const int64_t *slots, uint8_t *cache) {
  constexpr int kMost = Q8 ? 2 : 4;  // blocks of a unit
  const KvUnit k = unit_of<NB, Q8>(f.heads);
  // whole warps take part in a round: the four quarters of a run are in one
  const int64_t rounds = (tokens + k.step - 1) / k.step;
  int64_t tok = k.tok;
  for (int64_t i = 0; i < rounds; ++i, tok += k.step) {
    const bool there = k.there && tok < tokens;
    const int64_t slot = there ? __ldg(slots + tok) : -1;
    float x[kMost][8];
    const T *row = rows + tok * st.tok + k.head * st.head + k.first * 32 + k.q * 4;
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
      if (there && j < k.n) lo = load4(row + j * 32), hi = load4(row + j * 32 + 16);
      x[j][0] = lo.x, x[j][1] = lo.y, x[j][2] = lo.z, x[j][3] = lo.w;
      x[j][4] = hi.x, x[j][5] = hi.y, x[j][6] = hi.z, x[j][7] = hi.w;
    }
    // The blocks' extremes, over the four quarters: for Q8_0 the largest
    // magnitude, for Q4_0 the value that has it (of two, the first).
    float top[kMost];
    bool tie = false;
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      float up = Q8 ? fabsf(x[j][0]) : x[j][0], down = x[j][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) {
        up = fmaxf(up, Q8 ? fabsf(x[j][e]) : x[j][e]);
        if (!Q8) down = fminf(down, x[j][e]);
      }
      up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 1));
      up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 2));
      if (!Q8) {
        down = fminf(down, __shfl_xor_sync(0xffffffffu, down, 1));
        down = fminf(down, __shfl_xor_sync(0xffffffffu, down, 2));
        tie |= there && j < k.n && up == -down;  // zeros too: theirs may be of either sign
      }
      top[j] = Q8 || up >= -down ? up : down;
    }
    if (!Q8 && __any_sync(0xffffffffu, tie)) {
#pragma unroll
      for (int j = 0; j < kMost; ++j) {  // the least of 2 dim + sign
        uint32_t first = 64;
#pragma unroll
        for (int e = 7; e >= 0; --e)
          if (fabsf(x[j][e]) == fabsf(top[j])) first = 2 * ((e & 4) * 4 + k.q * 4 + (e & 3)) + (__float_as_uint(x[j][e]) >> 31);
        first = min(first, __shfl_xor_sync(0xffffffffu, first, 1));
        first = min(first, __shfl_xor_sync(0xffffffffu, first, 2));
        top[j] = first & 1 ? -fabsf(top[j]) : fabsf(top[j]);
      }
    }
    // Quarter j works out block j's scale and its inverse for all four.
    float mine = top[0];
#pragma unroll
    for (int j = 1; j < kMost; ++j)
      if (k.q == j) mine = top[j];
    const float scale = Q8 ? __fdiv_rn(mine, 127.0f) : mine * -0.125f;
    const float inverse = scale != 0.0f ? __fdiv_rn(1.0f, scale) : 0.0f;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      const float id = __shfl_sync(0xffffffffu, inverse, (threadIdx.x & 28) + j);
      uint32_t c[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        // The products one by one: a packed product before a packed sum gave other
        // bytes for bf16 rows (as one rounding of both would), and each is rounded here.
        const float2 y = make_float2(__fmul_rn(x[j][e], id), __fmul_rn(x[j][e + 1], id));
        if (Q8) {  // half away from zero: the number below 0.5 takes halves up and nothing else; |y| < 127.5; where not, see below
          c[e] = static_cast<uint32_t>(__float2int_rz(__fadd_rn(y.x, copysignf(0.49999997f, y.x))));
          c[e + 1] = static_cast<uint32_t>(__float2int_rz(__fadd_rn(y.y, copysignf(0.49999997f, y.y))));
        } else {  // truncated: the sum with 2^23, rounded towards zero, ends in the code
          float2 z = __fadd2_rn(y, make_float2(8.5f, 8.5f));
          z = __fadd2_rz(make_float2(fminf(z.x, 15.5f), fminf(z.y, 15.5f)), make_float2(8388608.0f, 8388608.0f));
          c[e] = __float_as_uint(z.x), c[e + 1] = __float_as_uint(z.y);
        }
      }
      const uint32_t lo = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
      const uint32_t hi = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
      if (Q8)
        w[(2 * j) & 3] = lo, w[(2 * j + 1) & 3] = hi;
      else
        w[j & 3] = (lo & 0x0f0f0f0fu) | (hi << 4 & 0xf0f0f0f0u);
    }
    // Where 1 / d overflows (d below 2^-128) or d is not finite, the rule's clamp acts.
    if (Q8 && __any_sync(0xffffffffu, isinf(inverse) || !isfinite(scale))) {
#pragma unroll
      for (int j = 0; j < kMost; ++j) {
        const float id = __shfl_sync(0xffffffffu, inverse, (threadIdx.x & 28) + j);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float r = fminf(fmaxf(roundf(__fmul_rn(x[j][4 * h + e], id)), -127.0f), 127.0f);
            v |= (static_cast<uint32_t>(static_cast<int>(r)) & 255u) << (8 * e);
          }
          w[(2 * j + h) & 3] = v;
        }
      }
    }
    KvAt at;
    if (!there || !at_slot(f, slot, k.head, val, &at)) continue;
    uint8_t *part = cache + at.part, *to = part + unit_at<Q8>(k, val, at.place);
    by_pairs<Q8>(w, k.n, val);
    if (k.n == kMost)
      *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    else if (Q8 || k.n == 2)
      *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t *>(to) = w[0];
    if (k.q < k.n)
      *reinterpret_cast<uint16_t *>(part + kv_scale_at(NB, Q8, at.place, k.first + k.q)) =
          __half_as_ushort(__float2half_rn(scale));
  }
}

template <int NB, bool Q8, typename T>
__device__ __forceinline__ void read_units(const KvForm &f, int64_t tokens, T *rows, bool val, const int64_t *slots,
                                           const uint8_t *cache) {
  constexpr int kMost = Q8 ? 2 : 4;
  const KvUnit k = unit_of<NB, Q8>(f.heads);
  if (!k.there) return;
  int64_t slot = k.tok < tokens ? __ldg(slots + k.tok) : -1;
  for (int64_t tok = k.tok; tok < tokens; tok += k.step) {
    const int64_t now = slot;
    if (tok + k.step < tokens) slot = __ldg(slots + tok + k.step);
    KvAt at;
    if (!at_slot(f, now, k.head, val, &at)) continue;
    const uint8_t *part = cache + at.part, *from = part + unit_at<Q8>(k, val, at.place);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (k.n == kMost) {
      const uint4 v = *reinterpret_cast<const uint4 *>(from);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if (Q8 || k.n == 2) {
      const uint2 v = *reinterpret_cast<const uint2 *>(from);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t *>(from);
    }
    float d[kMost];
#pragma unroll
    for (int j = 0; j < kMost; ++j)
      d[j] = j < k.n ? half_bits_to_float(*reinterpret_cast<const uint16_t *>(part + kv_scale_at(NB, Q8, at.place, k.first + j)))
                     : 0.0f;
    by_blocks<Q8>(w, k.n, val);
    T *row = rows + (tok * f.heads + k.head) * (NB * 32) + k.first * 32 + k.q * 4;
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      if (j >= k.n) continue;
      float x[8];
      if (Q8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // 2^23 + 128 + c, from the byte c + 128
          x[e] = __uint_as_float(__byte_perm(w[(2 * j) & 3] ^ 0x80808080u, 0x4b000000u, 0x7440 + e)) - 8388736.0f;
          x[e + 4] = __uint_as_float(__byte_perm(w[(2 * j + 1) & 3] ^ 0x80808080u, 0x4b000000u, 0x7440 + e)) - 8388736.0f;
        }
      } else {
        const uint32_t lo = w[j & 3] & 0x0f0f0f0fu, hi = w[j & 3] >> 4 & 0x0f0f0f0fu;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // 2^23 + c
          x[e] = __uint_as_float(__byte_perm(lo, 0x4b000000u, 0x7440 + e)) - 8388616.0f;
          x[e + 4] = __uint_as_float(__byte_perm(hi, 0x4b000000u, 0x7440 + e)) - 8388616.0f;
        }
      }
      store4(row + j * 32, make_float4(x[0] * d[j], x[1] * d[j], x[2] * d[j], x[3] * d[j]));
      store4(row + j * 32 + 16, make_float4(x[4] * d[j], x[5] * d[j], x[6] * d[j], x[7] * d[j]));
    }
  }
}

template <int NB, typename T>
__global__ void __launch_bounds__(256) kv_write_kernel(KvForm f, int64_t tokens, const T *K, KvRows ks, const T *V,
                                                       KvRows vs, const int64_t *slots, uint8_t *cache) {
  pdl_launch_dependents();
  pdl_wait();
  const bool val = blockIdx.y;
  if (val ? f.vq8 : f.kq8)
    write_units<NB, true>(f, tokens, val ? V : K, val ? vs : ks, val, slots, cache);
  else
    write_units<NB, false>(f, tokens, val ? V : K, val ? vs : ks, val, slots, cache);
}

template <int NB, typename T>
__global__ void __launch_bounds__(256) kv_read_kernel(KvForm f, int64_t tokens, T *K, T *V, const int64_t *slots,
                                                      const uint8_t *cache) {
  pdl_launch_dependents();
  pdl_wait();
  const bool val = blockIdx.y;
  if (val ? f.vq8 : f.kq8)
    read_units<NB, true>(f, tokens, val ? V : K, val, slots, cache);
  else
    read_units<NB, false>(f, tokens, val ? V : K, val, slots, cache);
}

template <int NB, typename... P, typename... A>
cudaError_t launch(const DevInfo &dev, const KvForm &f, int64_t tokens, cudaStream_t stream, void (*kernel)(P...), A... args) {
  // units of a token, by the type with the more of them (the other's blocks find none)
  const int units = f.heads * 4 * kv_runs(NB, f.kq8 || f.vq8), most = std::min(kv_runs(NB, true), kv_runs(NB, false));
  const int64_t per = std::max(1, 256 / (f.heads * 4 * (f.kq8 && f.vq8 ? kv_runs(NB, true) : most)));
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(256);
  const int64_t want = (tokens + per - 1) / per, z = (units + 255) / 256;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(want, std::max<int64_t>(1, dev.sms * kKvBlocks / z))), 2,
                     static_cast<unsigned>(z));
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int NB, typename T>
cudaError_t write_rows(const DevInfo &dev, const KvForm &f, int64_t tokens, const void *K, KvRows ks, const void *V,
                       KvRows vs, const int64_t *slots, void *cache, cudaStream_t stream) {
  return launch<NB>(dev, f, tokens, stream, kv_write_kernel<NB, T>, f, tokens, static_cast<const T *>(K), ks,
                static_cast<const T *>(V), vs, slots, static_cast<uint8_t *>(cache));
}

template <int NB, typename T>
cudaError_t read_rows(const DevInfo &dev, const KvForm &f, int64_t tokens, const int64_t *slots, const void *cache, void *K,
                      void *V, cudaStream_t stream) {
  return launch<NB>(dev, f, tokens, stream, kv_read_kernel<NB, T>, f, tokens, static_cast<T *>(K), static_cast<T *>(V), slots,
                    static_cast<const uint8_t *>(cache));
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
  return cuda_check(QMM_KV_FORM(write_rows, dev, f, T, K, ks, V, vs, slots, cache, stream), "kv_write launch");
}

qmm_status launch_kv_read(const DevInfo &dev, const KvForm &f, int dtype, int64_t T, const int64_t *slots,
                          const void *cache, void *K, void *V, cudaStream_t stream) {
  return cuda_check(QMM_KV_FORM(read_rows, dev, f, T, slots, cache, K, V, stream), "kv_read launch");
}

cudaError_t kv_cache_status(uint32_t *bits) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_kv_status, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_kv_status, &zero, sizeof(uint32_t));
  return e;
}

}  // namespace qmm
