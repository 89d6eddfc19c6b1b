// kv_attn.cuh -- the decode attention kernel over the quantised key/value cache
// (include/qmm.h, qmm_kv_attn; the cache's bytes: kv_layout.cuh), instantiated
// for each head size by kv_attn_d*.cu.
#pragma once

#include <algorithm>

#include "kv_layout.cuh"
#include "qmm_common.cuh"
#include "qmm_internal.h"

namespace qmm {

// ---- arithmetic on fragments ------------------------------------------------

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D = A . B + C, 16 x 8 x 16, fp16 operands, fp32 sums.
__device__ __forceinline__ float4 mma_f16(const uint4 &a, uint32_t b0, uint32_t b1, const float4 &c) {
  float4 d;
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d.x), "=f"(d.y), "=f"(d.z), "=f"(d.w)
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y), "f"(c.z), "f"(c.w));
  return d;
}

// The same with bf16 operands.
__device__ __forceinline__ float4 mma_bf16(const uint4 &a, uint32_t b0, uint32_t b1, const float4 &c) {
  float4 d;
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d.x), "=f"(d.y), "=f"(d.z), "=f"(d.w)
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y), "f"(c.z), "f"(c.w));
  return d;
}

// Two fp32 values as fp16 pairs hi + lo: 22 bits of each, when they are neither
// above 65504 nor so small that lo falls below fp16's 2^-24.
__device__ __forceinline__ void split_f16(float2 x, __half2 &hi, __half2 &lo) {
  hi = __float22half2_rn(x);
  lo = __float22half2_rn(__ffma2_rn(__half22float2(hi), make_float2(-1.0f, -1.0f), x));
}

// Transposes an 8 x 8 tile of 16-bit values: lane (g, t) has row g, columns 2t and
// 2t + 1, and gets column g, rows 2t and 2t + 1.
__device__ __forceinline__ __half2 transpose8(__half2 x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(h2_bits(x)));
  return bits_h2(y);
}

// Codes as fp16 pairs, exact: 0x6400 | c is 1024 + c. The constants come as
// launch arguments: an instruction takes one immediate, and constants that the
// compiler sees cost a second operation (measured: 64 of 487 instructions of 16
// keys).
struct KvMagic {
  uint32_t k1024, sixteenth, minus72;  // fp16 pairs; 0x64 is also the high byte of 1024 + c
};
//   Q4_0: low nibbles of bytes 0 and 2 of w; high nibbles of bytes 0 and 2
__device__ __forceinline__ uint32_t q4_low(uint32_t w, const KvMagic &k) {
  return h2_bits(__hsub2(bits_h2((w & 0x000f000fu) | k.k1024), bits_h2(0x64086408u)));  // - 1032
}
__device__ __forceinline__ uint32_t q4_high(uint32_t w, const KvMagic &k) {
  return h2_bits(__hfma2(bits_h2((w & 0x00f000f0u) | k.k1024), bits_h2(k.sixteenth), bits_h2(k.minus72)));
}
//   Q8_0: two bytes of w (already xor 0x80808080: code + 128) chosen by kSel
template <uint32_t kSel>
__device__ __forceinline__ uint32_t q8_pair(uint32_t w, const KvMagic &k) {
  return h2_bits(__hsub2(bits_h2(__byte_perm(w, k.k1024, kSel)), bits_h2(0x64806480u)));  // - 1152
}

__device__ __forceinline__ uint2 lds_u2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// ---- configuration ----------------------------------------------------------

// Floats of one partial result: rows x (D + maximum and sum).
__host__ __device__ constexpr int64_t kv_attn_slot_floats(int rows, int d) { return static_cast<int64_t>(rows) * (d + 2); }

constexpr int kKvMaxBlocks = 160;  // most blocks of a launch
constexpr int kKvMaxWarps = 8;     // most warps of a block
// What beginning an item costs a warp, in groups of keys (16 sequences of 6 to 100
// tokens: 15.6 us with 4, 21.6 us with 2; 64 long ones: 101.8 and 103.3 us).
constexpr int kKvItemCost = 4;

// Scratch: two marks and two partial results of each block, two outputs of each warp.
__host__ __device__ constexpr int64_t kv_attn_scratch_floats(int rows, int d) {
  return kKvMaxBlocks * (4 + 2 * kv_attn_slot_floats(rows, d) + 2 * kKvMaxWarps * rows * (d + 8));
}

template <int NB, bool KQ8, bool VQ8, int OCT, bool FINE>
struct KvCfg {
  static constexpr int kD = NB * 32;
  static constexpr int kKeyPart = kv_part_bytes(NB, KQ8);
  static constexpr int kGroupBytes = kKeyPart + kv_part_bytes(NB, VQ8);
  static constexpr int kRows = 8 * OCT;
  static constexpr int kPiece = kRows * (kD + 8);         // floats of a warp's partial outputs (8 between rows: banks)
  static constexpr int kTerms = FINE ? 2 : 1;             // fp16 terms of a query or weight
  static constexpr int kQBytes = OCT * NB * kTerms * 512;  // a warp's query fragments
  static constexpr int kBudget = 216 * 1024;  // of 227 KB; the rest is the static arrays
  static constexpr int warp_bytes(int tg, int stages) { return kQBytes + stages * tg * kGroupBytes; }
  // Warps of a block, one block an SM. 12 and 16 warps of fewer registers and
  // shorter steps were as fast or slower.
  static constexpr int kNW = 8 * warp_bytes(1, 2) <= kBudget ? 8 : 4;
  // Groups of a step, as many as leave the sums in registers (ptxas reports 255 of
  // them and 12 to 28 bytes spilled for one octet of fp32 rows of 128, Q4_0): 64
  // ragged sequences of up to 8192 tokens take 102, 117, 144 us with 4, 2, 1 (one
  // octet of rows), 131072 keys of one 55, 63, 76 us. A step's ring stage is 9 KB at
  // most, so that two to four are in flight.
  static constexpr int kMaxTG = OCT == 1 ? 4 : OCT == 2 ? 2 : 1;
  static constexpr bool fits(int tg) { return tg * kGroupBytes <= 9216 && kNW * warp_bytes(tg, 2) <= kBudget; }
  static constexpr int kTG = kMaxTG >= 4 && fits(4) ? 4 : kMaxTG >= 2 && fits(2) ? 2 : 1;
  static constexpr int stages() {
    int n = 2;
    while ((n < 4 || warp_bytes(kTG, n) < kPiece * 4) && kNW * warp_bytes(kTG, n + 1) <= kBudget) ++n;
    return n;
  }
  static constexpr int kStages = stages();
  static constexpr int kStageBytes = kTG * kGroupBytes;
  static constexpr int kSmem = kNW * warp_bytes(kTG, kStages);
  static_assert(kSmem <= kBudget, "stages do not fit");
  static_assert(warp_bytes(kTG, kStages) >= kPiece * 4, "a warp's partial result does not fit");
  static_assert(kStages * kTG <= 32, "a bit for each group in the ring");
  static_assert(kNW <= kKvMaxWarps, "scratch is sized for fewer warps");
};

// A launch's constants.
struct KvLaunch {
  KvForm f;
  KvAttnArgs a;
  int ratio, rows, tiles;  // query heads of a key/value head; rows M ratio of one; tiles of kRows rows
  int min_units;           // least units of the line for a warp
  int bf16;
  KvMagic magic;
  uint64_t epoch;          // this call's mark, not 0
};

// Groups of 16 tokens that the queries of sequence s see: [first, first + n).
struct KvSeq {
  int len, first, n;
};

__device__ __forceinline__ KvSeq kv_seq(const KvLaunch &p, int s, uint32_t *status) {
  int len = __ldg(p.a.lens + s);
  const int most = p.a.max_pages * p.f.page;
  if (len < 0 || len > most) {
    atomicOr(status, kDevBadIndex);
    len = len < 0 ? 0 : most;
  }
  const int low = p.a.window > 0 ? max(0, len - p.a.m + 1 - p.a.window) : 0;
  KvSeq q;
  q.len = len;
  q.first = low / kKvGroup;
  q.n = len > 0 ? (len + kKvGroup - 1) / kKvGroup - q.first : 0;
  return q;
}

// Units of the line that an item of n groups takes.
__device__ __forceinline__ int64_t kv_units(int n) { return n ? n + kKvItemCost : 0; }

__device__ __forceinline__ void kv_store(const KvLaunch &p, int64_t at, float4 v) {
  if (p.bf16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.a.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
  } else {
    *reinterpret_cast<float4 *>(static_cast<float *>(p.a.out) + at) = v;
  }
}

__device__ __forceinline__ void kv_store(const KvLaunch &p, int64_t at, float2 v) {
  if (p.bf16)
    *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.a.out) + at) = __floats2bfloat162_rn(v.x, v.y);
  else
    *reinterpret_cast<float2 *>(static_cast<float *>(p.a.out) + at) = v;
}

// Output offset of row r (of one key/value head's M x ratio rows).
__device__ __forceinline__ int64_t kv_out_at(const KvLaunch &p, int s, int head, int r, int d) {
  const int i = r / p.ratio, h = r - i * p.ratio;
  return ((static_cast<int64_t>(s) * p.a.m + i) * p.a.hq + head * p.ratio + h) * d;
}

// a / b of numbers >= 0, without the slow 64-bit division where they are small.
static __device__ __noinline__ int64_t kv_div(int64_t a, int64_t b) {
  if ((static_cast<uint64_t>(a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// A line of `total` units over `blocks`: the first `more` have one more than `each`.
struct KvShare {
  int64_t each, more;
  __device__ __forceinline__ int64_t begin(int i) const { return i * each + min(static_cast<int64_t>(i), more); }
  // the block that has place `at`
  __device__ __forceinline__ int block_of(int64_t at) const {
    const int64_t wide = more * (each + 1);
    return static_cast<int>(at < wide ? kv_div(at, each + 1) : more + kv_div(at - wide, each));
  }
};

// Reads of partial results that another block wrote: the clobber keeps the
// compiler from moving them over the wait for that block's mark.
__device__ __forceinline__ float2 kv_load2(const float *p) {
  float2 v;
  asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 kv_load4(const float *p) {
  float4 v;
  asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Four dims of a row, added up over partial results (maximum, sum; outputs), a
// batch of them at a time so that their loads are in flight together.
struct KvSum {
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  template <int N>
  __device__ __forceinline__ void add(const float2 (&ml)[N], const float4 (&v)[N]) {
    float next = m;
#pragma unroll
    for (int i = 0; i < N; ++i) next = fmaxf(next, ml[i].x);
    const float ref = next == -INFINITY ? 0.0f : next, keep = exp2_approx(m - ref);
    m = next;
    l *= keep, o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float k = exp2_approx(ml[i].x - ref);
      l = fmaf(k, ml[i].y, l);
      o.x = fmaf(k, v[i].x, o.x), o.y = fmaf(k, v[i].y, o.y), o.z = fmaf(k, v[i].z, o.z), o.w = fmaf(k, v[i].w, o.w);
    }
  }
};

// A run's value codes of a group, this lane's: two dims of each half block of tokens
// t + 4 e, as many blocks as the run has.
template <int NB, bool VQ8>
__device__ __forceinline__ void kv_value_words(uint32_t (&vw)[4][2], uint32_t part, int run) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wide = VQ8 ? 4 : 2, bytes = kv_run_blocks(NB, VQ8, run) * wide;
  part += kv_run_first(NB, VQ8, run) * 128 * wide;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (bytes == 8) {
      const uint2 v = lds_u2(part + ((g >> 2) * 64 + t * 4 + (g & 3)) * 8 + e * 128);
      vw[e][0] = v.x, vw[e][1] = v.y;
    } else if (bytes == 4) {
      vw[e][0] = lds_u32(part + (t * 8 + g) * 4 + e * 128);
    } else {
      vw[e][0] = lds_u16(part + (t * 8 + g) * 2 + e * 64);
    }
  }
}

// The codes of the run's block r as fp16: columns of 4 tiles, tokens in pairs.
template <bool VQ8>
__device__ __forceinline__ void kv_value_tiles(uint32_t (&vb)[4][2], const uint32_t (&vw)[4][2], int r, const KvMagic &magic) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (VQ8) {
      const uint32_t w0 = vw[2 * h][r & 1] ^ 0x80808080u, w1 = vw[2 * h + 1][r & 1] ^ 0x80808080u;
      const uint32_t x = __byte_perm(w0, w1, 0x5140), y = __byte_perm(w0, w1, 0x7362);
      vb[0][h] = q8_pair<0x5150>(x, magic), vb[2][h] = q8_pair<0x5352>(x, magic);
      vb[1][h] = q8_pair<0x5150>(y, magic), vb[3][h] = q8_pair<0x5352>(y, magic);
    } else {
      const uint32_t x = __byte_perm(vw[2 * h][r >> 1], vw[2 * h + 1][r >> 1], r & 1 ? 0x7632 : 0x5410);
      const uint32_t x8 = x >> 8;
      vb[0][h] = q4_low(x, magic), vb[1][h] = q4_high(x, magic);
      vb[2][h] = q4_low(x8, magic), vb[3][h] = q4_high(x8, magic);
    }
  }
}

// yes ? a : b, as a selection of registers: the compiler makes a chain of them over an
// array's elements an index into a copy of the array in local memory.
__device__ __forceinline__ float2 choose(bool yes, float2 a, float2 b) {
  float2 r;
  asm("{.reg .pred p; setp.ne.s32 p, %6, 0; selp.f32 %0, %2, %4, p; selp.f32 %1, %3, %5, p;}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "r"(static_cast<int>(yes)));
  return r;
}

__device__ __forceinline__ uint32_t bf2_bits(float2 x) {
  const __nv_bfloat162 b = __float22bfloat162_rn(x);
  return *reinterpret_cast<const uint32_t *>(&b);
}

// Adds a step's weights times values to the sums, whatever the values' scales: p d_v is
// formed in fp32 and taken as three bf16 terms (24 bits, and fp32's range, so that no
// weight loses bits to another); codes are exact in bf16 too. A weight of 0 takes
// nothing from its value, infinite or NaN; weights of keys that a row sees are kept
// from 0 where such a value is among them (`odd`), so that it gets there.
// z: weights times 2^13 of rows 8 o + 2t and the next, for key (g >> 1) + 4 (g & 1) + 8 j
// of group gi; acc: 2^up_exp times the sums; parts: the first group's values; ok: a bit
// for each group that is there.
template <int NB, bool VQ8, int kGroupBytes, int OCT, int TG>
__device__ __forceinline__ void kv_add_apart(float2 (&acc)[OCT][NB * 4], const float2 (&z)[OCT][TG][2], uint32_t parts,
                                             uint32_t ok, int key0, int up_exp, bool odd, const int2 (&last)[OCT],
                                             const int2 (&low)[OCT], const KvMagic &magic) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const float unit = __uint_as_float(static_cast<uint32_t>(up_exp - 13 + 127) << 23);
#pragma unroll 1
  for (int gi = 0; gi < TG; ++gi) {
    if (!(ok >> gi & 1)) continue;
    const uint32_t part = parts + gi * kGroupBytes;
    float2 w[OCT][2];  // transposed: row g, tokens t + 8 j and t + 4 + 8 j
#pragma unroll
    for (int o = 0; o < OCT; ++o)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float2 x = z[o][0][j];
#pragma unroll
        for (int k = 1; k < TG; ++k) x = choose(k == gi, z[o][k][j], x);
        x = make_float2(x.x * unit, x.y * unit);
        if (odd) {
          const int key = key0 + gi * kKvGroup + (g >> 1) + 4 * (g & 1) + 8 * j;
          if (key <= last[o].x && key >= low[o].x) x.x = fmaxf(x.x, 1e-30f);
          if (key <= last[o].y && key >= low[o].y) x.y = fmaxf(x.y, 1e-30f);
        }
        const uint32_t a = __float_as_uint(x.x), b = __float_as_uint(x.y);
        const uint32_t up = h2_bits(transpose8(bits_h2(__byte_perm(a, b, 0x7632))));
        const uint32_t down = h2_bits(transpose8(bits_h2(__byte_perm(a, b, 0x5410))));
        w[o][j] = make_float2(__uint_as_float(__byte_perm(down, up, 0x5410)), __uint_as_float(__byte_perm(down, up, 0x7632)));
      }
#pragma unroll
    for (int run = 0; run < kv_runs(NB, VQ8); ++run) {
      uint32_t vw[4][2];
      kv_value_words<NB, VQ8>(vw, part, run);
#pragma unroll
      for (int r = 0; r < (VQ8 ? 2 : 4); ++r) {
        if (r >= kv_run_blocks(NB, VQ8, run)) continue;
        const int b = kv_run_first(NB, VQ8, run) + r;
        uint32_t vb[4][2];
        kv_value_tiles<VQ8>(vb, vw, r, magic);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) vb[i][j] = bf2_bits(__half22float2(bits_h2(vb[i][j])));
        const uint2 scales = lds_u2(part + kv_scale_at(NB, VQ8, t, b));
#pragma unroll
        for (int o = 0; o < OCT; ++o) {
          uint32_t terms[3][2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 d = __half22float2(bits_h2(j ? scales.y : scales.x));
            float2 x = make_float2(w[o][j].x != 0.0f ? w[o][j].x * d.x : 0.0f, w[o][j].y != 0.0f ? w[o][j].y * d.y : 0.0f);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const uint32_t y = bf2_bits(x);
              terms[i][j] = y;
              // (an infinity is its own first term)
              x.x = isinf(x.x) ? 0.0f : x.x - __uint_as_float(y << 16);
              x.y = isinf(x.y) ? 0.0f : x.y - __uint_as_float(y & 0xffff0000u);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 2; i >= 0; --i)
              c = mma_bf16(make_uint4(vb[2 * h][0], vb[2 * h + 1][0], vb[2 * h][1], vb[2 * h + 1][1]), terms[i][0], terms[i][1], c);
            float2 &p = acc[o][b * 4 + 2 * h], &q = acc[o][b * 4 + 2 * h + 1];
            p = make_float2(p.x + c.x, p.y + c.y), q = make_float2(q.x + c.z, q.y + c.w);
          }
        }
      }
    }
  }
}

// The same as a call, its arrays in local memory: for two octets of heads of 192 and 256,
// whose sums leave no registers for it in the middle of a step (16 rows of 256, Q8_0,
// fp32, 8 x 8192 keys of 8 heads, no step of which calls it: 168 us in line, 151 so).
template <int NB, int OCT, int TG>
struct KvApart {
  float2 acc[OCT][NB * 4], z[OCT][TG][2];
  int2 last[OCT], low[OCT];
};
template <int NB, bool VQ8, int kGroupBytes, int OCT, int TG>
__device__ __noinline__ void kv_add_apart_call(KvApart<NB, OCT, TG> &s, uint32_t parts, uint32_t ok, int key0, int up_exp,
                                               bool odd, const KvMagic &magic) {
  kv_add_apart<NB, VQ8, kGroupBytes>(s.acc, s.z, parts, ok, key0, up_exp, odd, s.last, s.low, magic);
}

// ---- the kernel -------------------------------------------------------------
//
// Work is a line on which the items, an item being (sequence, head, tile of
// query rows), lie one after the other, each as long as its groups of keys and
// what beginning it costs. Every warp takes an equal run of the line, whatever
// the sequences' lengths, and works alone: it brings its groups by bulk copies
// into a ring of its own, across the ends of items, and holds the running
// maximum, sum and outputs of its keys. An item that one warp has whole is
// finished there; the others' partial results are joined by the block that has
// the item, or by the last of the item's blocks to be done (always in the
// line's order: the same sums every time).
//
// Products run on the tensor cores (mma.m16n8k16) with the cached codes, exact
// fp16 integers, as the 16-row operand and an octet of query rows as the 8
// columns: scores are keys x rows, outputs dims x rows, so a conversion serves
// every octet and no column is wasted on terms. fp32 queries (FINE) and the
// weights that go with them are two fp16 terms (22 bits together), each a product
// of its own into the same sums; bf16 queries and their weights are one (the
// weights' remainders would take 2 to 6% of short calls and 8 to 25% of long ones,
// and bring the outputs' error, 1.674e-3 of their norm, to bf16's own 1.672e-3). A
// key's block scale multiplies the finished 32-dim dot in fp32; a value's block scale
// goes into the weight, p d_v, in fp16 with the product's own remainder (FINE), or, in
// steps whose scales lie far apart or are not finite, in fp32 (kv_add_apart).
// The weights change sides between the two products by 8 x 8 transposes. Each
// step's sums are added to fp32 registers outside the tensor core, whose own sums
// need not be rounded to nearest.
//
// What bounds it: at short contexts the chain of latencies (7.6 us for 33 tokens
// of two heads: 2 us to know the lengths and find the work, 1 us for the first
// copies, 1 to 2 us a step and again for joining); at long ones instructions. 16
// keys of a head of 128, Q4_0, fp32 queries, are 370 instructions of a warp: 132
// on the 2-cycle ALU, 111 in fp16 (2 cycles), 32 products of 8 cycles, which overlap
// by a third; some 710 cycles together. One sequence of 131072 tokens, 8 heads: 54.6
// us, 2.8 TB/s of cache (29 us without the arithmetic), of which some 13 us are the
// call's own: with one step a warp (8192 tokens) it takes 16.2 us, and a step more
// takes 3 us. 16 x 8192 tokens, 8 heads of 256, Q8_0, one query row, where a byte needs
// half the instructions: 110 us, 5.2 TB/s, 79% of the measured copy rate.
template <int NB, bool KQ8, bool VQ8, int OCT, bool FINE>
__device__ __forceinline__ void kv_attn_body(const KvLaunch &p, uint32_t *status) {
  using C = KvCfg<NB, KQ8, VQ8, OCT, FINE>;
  constexpr int NW = C::kNW, TG = C::kTG, S = C::kStages, D = C::kD, TERMS = C::kTerms;
  constexpr int kThreads = NW * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[NW * S];
  __shared__ int64_t scan[kThreads + 1];
  // A partial result: groups [a, b) of an item's n; its maxima and sums are in
  // piece_ml, its outputs in the warp's own shared memory if they are the warp's
  // last, else in the scratch.
  struct Piece {
    int seq, head, tile, a, b, n;
    const float *out;
  };
  // A warp's place on the line: an item's groups [a, b) of n, and the units behind them.
  struct Place {
    int seq, head, tile, len, first, n, a, b;
    int64_t left;
  };
  __shared__ Place puts[NW];  // where the copies are
  struct Job {  // what is added up: an item's pieces (as bits), or its blocks' results from a first block on
    int seq, head, tile, a;
    uint32_t pieces;
    int n;
    bool whole;
  };
  __shared__ Piece pieces[2 * NW];
  __shared__ float2 piece_ml[2 * NW][C::kRows];
  __shared__ Job jobs[2 * NW], joins[2];
  __shared__ KvShare kept_share;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const KvMagic magic = p.magic;
  uint8_t *own = smem + warp * C::warp_bytes(TG, S);
  uint4 *qfrag = reinterpret_cast<uint4 *>(own);  // [OCT][NB][TERMS][32]
  uint8_t *ring = own + C::kQBytes;
  const uint32_t qfrag_s = smem_u32(qfrag) + lane * 16, ring_s = smem_u32(ring);
  uint64_t *bar = bars + warp * S;

  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(bar + i, 1);
    fence_mbar_init();
  }
  if (tid < 2 * NW) pieces[tid].seq = -1;
  pdl_launch_dependents();
  pdl_wait();

  // The line: scan[i] is where the sequences of thread i begin on it. Up to 32
  // sequences every warp sees for itself.
  const int64_t per_seq = static_cast<int64_t>(p.f.heads) * p.tiles;
  const int chunk = (p.a.batch + kThreads - 1) / kThreads;
  int64_t total;
  {
    const bool few = p.a.batch <= 32;
    const int at = few ? lane : tid, s0 = min(p.a.batch, at * chunk), s1 = min(p.a.batch, s0 + chunk);
    int64_t incl = 0;
    bool none = false;
    for (int s = s0; s < s1; ++s) {
      const int n = kv_seq(p, s, status).n;
      incl += kv_units(n) * per_seq;
      none |= n == 0;
    }
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (few) {
      total = __shfl_sync(0xffffffffu, incl, 31);
      none = __any_sync(0xffffffffu, none);
      if (warp == 0) scan[lane + 1] = incl;
      if (tid == 0) scan[0] = 0;
      if (tid >= 32) scan[tid + 1] = total;
      __syncthreads();
    } else {
      scan[tid + 1] = incl;
      if (tid == 0) scan[0] = 0;
      none = __syncthreads_or(none);
      int64_t before = 0;
      for (int w = 0; w < warp; ++w) before += scan[w * 32 + 32];
      __syncthreads();
      scan[tid + 1] = incl + before;
      __syncthreads();
      total = scan[kThreads];
    }
    if (none)  // rows of sequences without keys
      for (int s = blockIdx.x; s < p.a.batch; s += gridDim.x) {
        if (kv_seq(p, s, status).n) continue;
        const int64_t n = static_cast<int64_t>(p.a.m) * p.a.hq * D;
        for (int64_t e = tid * 4; e < n; e += kThreads * 4) kv_store(p, s * n + e, make_float4(0.f, 0.f, 0.f, 0.f));
      }
  }

  // Blocks that work, this block's run of the line, and this warp's part of it.
  const int64_t least = static_cast<int64_t>(p.min_units) * NW;
  int blocks = gridDim.x;
  if (total < blocks * least) blocks = static_cast<int>(kv_div(total + least - 1, least));
  volatile uint64_t *marks = reinterpret_cast<volatile uint64_t *>(p.a.ws);  // two of each block
  constexpr int64_t kSlot = kv_attn_slot_floats(C::kRows, D);
  float *block_slots = p.a.ws + kKvMaxBlocks * 4 + 2 * blockIdx.x * kSlot;
  float *warp_slots = p.a.ws + kKvMaxBlocks * (4 + 2 * kSlot) + 2 * NW * blockIdx.x * C::kPiece;
  if (blockIdx.x >= blocks) return;
  KvShare share;
  share.each = kv_div(total, blocks);
  share.more = total - share.each * blocks;
  if (tid == 0) kept_share = share;  // (for the end: not in registers over the work)
  const int64_t from = share.begin(blockIdx.x), span = share.begin(blockIdx.x + 1) - from;

  // The part of the item at hand that begins `skip` units into it.
  auto enter = [&](Place &c, int64_t skip) {
    const int64_t a = max(skip - kKvItemCost, int64_t(0));
    const int64_t b = min(static_cast<int64_t>(c.n), max(skip + c.left - kKvItemCost, int64_t(0)));
    c.a = static_cast<int>(a);
    c.b = static_cast<int>(b);
    c.left -= min(kv_units(c.n) - skip, c.left);
  };
  auto look = [&](Place &c) {
    const KvSeq q = kv_seq(p, c.seq, status);
    c.len = q.len, c.first = q.first, c.n = q.n;
  };
  // The next item with groups for this warp; c.b == c.a at the end.
  auto next = [&](Place &c) {
    c.a = c.b = 0;
    while (c.left > 0 && c.b == c.a) {
      if (++c.tile == p.tiles) {
        c.tile = 0;
        if (++c.head == p.f.heads) {
          c.head = 0;
          do {
            if (++c.seq >= p.a.batch) {
              c.left = 0;
              return;
            }
            look(c);
          } while (c.n == 0);
        }
      }
      enter(c, 0);
    }
  };
  Place use{};
  {
    const int64_t pos = from + span * warp / NW;  // (NW is a power of two)
    use.left = from + span * (warp + 1) / NW - pos;
    if (use.left > 0) {
      int64_t base;
      if (p.a.batch <= 32) {
        use.seq = __popc(__ballot_sync(0xffffffffu, scan[lane + 1] <= pos));
        base = scan[use.seq];
      } else {
        int lo = 0, hi = kThreads;  // scan[lo] <= pos < scan[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (scan[mid] <= pos)
            lo = mid;
          else
            hi = mid;
        }
        base = scan[lo];
        use.seq = lo * chunk;
      }
      look(use);
      while (pos >= base + kv_units(use.n) * per_seq) {
        base += kv_units(use.n) * per_seq;
        ++use.seq;
        look(use);
      }
      const int64_t units = kv_units(use.n);
      const int item = static_cast<int>(kv_div(pos - base, units));
      use.head = item / p.tiles;
      use.tile = item - use.head * p.tiles;
      enter(use, pos - base - item * units);
    }
  }

  const int per_page = p.f.page / kKvGroup, page_shift = 31 - __clz(per_page);
  const uint64_t policy = l2_evict_first_policy();
  if (lane == 0) puts[warp] = use;
  __syncwarp();
  uint32_t filled = 0, used = 0;  // stages of the ring so far
  uint32_t ok_bits = 0;           // groups in the ring whose page exists
  bool dead = false;              // a wait ran out

  // The copies run ahead of the work, over the ends of items. Each lane has the
  // address of one of the next 32 groups of the item at hand (put_at counts
  // those copied, put_n those there are, put_ok marks the ones whose page exists).
  const uint8_t *src = nullptr;
  int put_at = 0, put_n = 0, put_grp = use.first + use.a, put_end = use.first + use.b;
  uint32_t put_ok = 0;
  // Fill the ring's free stages, a step of TG groups each.
  auto fill = [&]() {
    while (filled - used < S) {
      if (put_at >= put_n) {
        put_grp += put_n;
        put_n = put_at = 0;
        Place put = puts[warp];
        if (put_grp >= put_end) {
          if (put.left <= 0) return;
          next(put);
          __syncwarp();
          if (lane == 0) puts[warp] = put;
          __syncwarp();
          put_grp = put.first + put.a;
          put_end = put.first + put.b;
          if (put_grp >= put_end) return;
        }
        const int grp = put_grp + lane;
        put_n = min(put_end - put_grp, 32);
        bool ok = false;
        if (lane < put_n) {
          const int page = __ldg(p.a.table + put.seq * p.a.table_stride + (grp >> page_shift));
          ok = page >= 0 && page < p.f.pages;
          if (!ok) atomicOr(status, kDevBadIndex);
          src = p.a.cache + ((static_cast<int64_t>(page) * p.f.heads + put.head) * per_page + (grp & (per_page - 1))) *
                                C::kGroupBytes;
        }
        put_ok = __ballot_sync(0xffffffffu, ok);
      }
      const int st = filled % S;
      const uint32_t ok = put_ok >> put_at & ((1u << TG) - 1);
      const int mine = lane - put_at;
      if (mine == 0) mbar_arrive_expect_tx(bar + st, __popc(ok) * C::kGroupBytes);
      __syncwarp();
      const bool held = p.a.withhold && blockIdx.x == 0 && filled == 0;
      if (mine >= 0 && mine < TG && (put_ok >> lane & 1) && !held)
        bulk_g2s(ring + st * C::kStageBytes + mine * C::kGroupBytes, src, C::kGroupBytes, bar + st, policy);
      ok_bits = (ok_bits & ~(((1u << TG) - 1) << (st * TG))) | ok << (st * TG);
      ++filled;
      put_at += TG;
    }
  };

  // The query rows 8 o + g of an item, four dims of each half block a lane.
  auto load_rows = [&](float4 (&rows)[OCT][NB][2]) {
#pragma unroll
    for (int o = 0; o < OCT; ++o) {
      const int row = use.tile * C::kRows + o * 8 + g;
      const bool there = row < p.rows;
      const int i = there ? row / p.ratio : 0, h = there ? row - i * p.ratio : 0;
      const int64_t at = use.seq * p.a.q_seq + i * p.a.q_tok +
                         (static_cast<int64_t>(use.head) * p.ratio + h) * p.a.q_head + 4 * t;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int64_t e = at + b * 32 + half * 16;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (there) {
            if (FINE) {
              v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.a.q) + e);
            } else {
              const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.a.q) + e);
              v = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                              __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
            }
          }
          rows[o][b][half] = v;
        }
    }
  };

  while (true) {
    if (use.a == use.b) {
      if (use.left <= 0) break;
      next(use);
      if (use.a == use.b) break;
    }
    float4 rows[OCT][NB][2];
    load_rows(rows);
    if (!dead) fill();  // (the first item: nothing is on its way yet)
    // of rows 8 o + 2t and 8 o + 2t + 1
    float2 top[OCT], sum[OCT], factor[OCT];
    int2 last[OCT], low[OCT];
    float2 acc[OCT][NB * 4];  // dims 2g, 16 + 2g, 2g + 1, 17 + 2g of each block

    // ---- query rows as fragments ----
    // Each row is brought to [2^14, 2^15) by a power of two so that both terms
    // stay in fp16's range; its inverse, with the softmax's scale and log2(e),
    // is the factor of the row's scores, positive: the scale's sign goes into
    // the row.
    __syncwarp();
#pragma unroll
    for (int o = 0; o < OCT; ++o) {
      float big = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float4 v = rows[o][b][half];
          big = fmaxf(big, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
        }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // exponent of the largest, at least -100 (smaller rows keep fewer bits of scores that are 0 anyway)
      const int ex = max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -100);
      float up = __uint_as_float(static_cast<uint32_t>(14 - ex + 127) << 23);
      // (at least the smallest normal number: times minus infinity it has to stay that)
      const float f = p.a.scale == 0.0f ? 1.0f
                                        : fmaxf(fabsf(p.a.scale) * 1.44269504088896f *
                                                    __uint_as_float(static_cast<uint32_t>(ex - 14 + 127) << 23),
                                                1.17549435e-38f);
      factor[o] = make_float2(__shfl_sync(0xffffffffu, f, 8 * t), __shfl_sync(0xffffffffu, f, 8 * t + 4));
      if (p.a.scale <= 0.0f) up = p.a.scale < 0.0f ? -up : 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        __half2 hi[4], lo[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float4 v = rows[o][b][half];
          const float2 even = make_float2(v.x * up, v.z * up), odd = make_float2(v.y * up, v.w * up);
          split_f16(even, hi[2 * half], lo[2 * half]);
          split_f16(odd, hi[2 * half + 1], lo[2 * half + 1]);
        }
        uint4 *f = qfrag + (o * NB + b) * TERMS * 32 + lane;
        f[0] = make_uint4(h2_bits(hi[0]), h2_bits(hi[1]), h2_bits(hi[2]), h2_bits(hi[3]));
        if (FINE) f[32] = make_uint4(h2_bits(lo[0]), h2_bits(lo[1]), h2_bits(lo[2]), h2_bits(lo[3]));
      }
      top[o] = make_float2(-INFINITY, -INFINITY);
      sum[o] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int n = 0; n < NB * 4; ++n) acc[o][n] = make_float2(0.0f, 0.0f);
      const int row = use.tile * C::kRows + o * 8 + 2 * t, off = use.len - p.a.m;
      last[o] = make_int2(off + min(row / p.ratio, p.a.m - 1), off + min((row + 1) / p.ratio, p.a.m - 1));
      low[o] = p.a.window > 0 ? make_int2(max(0, last[o].x - p.a.window + 1), max(0, last[o].y - p.a.window + 1))
                              : make_int2(0, 0);
    }
    __syncwarp();
    const int low_all = p.a.window > 0 ? max(0, use.len - p.a.m - p.a.window + 1) : 0;
    const int grp_end = use.first + use.b;
    // a lane's 16 bytes of a step's value scales
    constexpr int kLooks = TG * NB * 2;
    static_assert(kLooks <= 32, "a step's value scales in one load of a warp");
    const int look = lane % kLooks;
    const uint32_t look_off = look / (2 * NB) * C::kGroupBytes + C::kKeyPart + kv_code_bytes(NB, VQ8) + look % (2 * NB) * 16;
    int up_exp = 13;  // acc and sum are 2^up_exp and 2^13 times the outputs' and weights' sums

    for (int grp = use.first + use.a; grp < grp_end && !dead; grp += TG) {
      const int st = used % S;
      if (!__all_sync(0xffffffffu, mbar_wait(bar + st, (used / S) & 1, p.a.wait_ns))) {
        // Nothing more is copied; what is in flight is waited for once more. The
        // warp's items end with what they have, so that no block waits in vain.
        bool drained = true;
        for (uint32_t i = used; i != filled; ++i) drained = mbar_wait(bar + i % S, (i / S) & 1, p.a.wait_ns) && drained;
        if (lane == 0) atomicOr(status, kDevTimeoutFull | (drained ? 0u : kDevTimeoutDrain));
        dead = true;
        break;
      }
      ++used;
      const uint32_t stage = ring_s + st * C::kStageBytes;
      const uint32_t ok = ok_bits >> (st * TG) & ((1u << TG) - 1);
      const int key0 = grp * kKvGroup;
      const bool full = ok == (1u << TG) - 1 && key0 + TG * kKvGroup <= use.len - p.a.m + 1 &&
                        (p.a.window == 0 || key0 >= use.len - p.a.window);

      // ---- scales of the values ----
      uint32_t vs[TG][NB][2];
#pragma unroll
      for (int gi = 0; gi < TG; ++gi) {
        const uint32_t at = stage + gi * C::kGroupBytes + C::kKeyPart + kv_code_bytes(NB, VQ8) + t * NB * 8;
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
          if (NB % 2 == 0) {
            const uint4 v = lds_u4(at + b * 8);
            vs[gi][b][0] = v.x, vs[gi][b][1] = v.y, vs[gi][min(b + 1, NB - 1)][0] = v.z, vs[gi][min(b + 1, NB - 1)][1] = v.w;
          } else {
            const uint2 v = lds_u2(at + b * 8);
            vs[gi][b][0] = v.x, vs[gi][b][1] = v.y;
            if (b + 1 < NB) {
              const uint2 u = lds_u2(at + b * 8 + 8);
              vs[gi][min(b + 1, NB - 1)][0] = u.x, vs[gi][min(b + 1, NB - 1)][1] = u.y;
            }
          }
        }
      }
      if (!full) {  // what no row sees may be anything, NaN among it: its scale is 0
#pragma unroll
        for (int gi = 0; gi < TG; ++gi)
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // e = tok / 4: column e & 1 of half e >> 1
            const int key = key0 + gi * kKvGroup + t + 4 * e;
            if (!(ok >> gi & 1) || key >= use.len || key < low_all)
#pragma unroll
              for (int b = 0; b < NB; ++b) vs[gi][b][e >> 1] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
          }
      }
      // The weights are p 2^13 and so p d_v 2^13: inside fp16 with room for both
      // terms while every scale is in [2^-7, 2), or 0. Scales that lie within 8
      // binades of each other are brought there by a power of two, exactly, which the
      // sums keep (up_exp). Others, and scales that are not finite, would lose bits
      // to the largest of them, or reach rows that must not see them: see `apart`.
      // To look at them all, a lane takes 16 bytes: of two blocks' (of one or two of
      // the four token columns t), tokens t, t + 4, t + 8 and t + 12.
      uint4 d = *reinterpret_cast<const uint4 *>(ring + st * C::kStageBytes + look_off);
      int e_new = 13;
      bool apart = false, odd = false;  // scales far apart, or not finite
      if (__any_sync(0xffffffffu, !full || ((d.x | d.y | d.z | d.w) & 0x40004000u) | (~(d.x & d.y & d.z & d.w) & 0x20002000u))) {
        if (!full) {  // (as above)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int unit = look % (2 * NB) * 2 + i, grp_i = look / (2 * NB);
            uint32_t *w = i ? &d.z : &d.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + grp_i * kKvGroup + unit / NB + 4 * e;
              if (!(ok >> grp_i & 1) || key >= use.len || key < low_all) w[e >> 1] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
            }
          }
        }
        uint32_t big = 0, small = ~0u;  // small: less 1, so that 0 is the largest
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = (&d.x)[i] & 0x7fff7fffu;
          big = __vmaxu2(big, x), small = __vminu2(small, __vsub2(x, 0x00010001u));
        }
        big = __reduce_max_sync(0xffffffffu, max(big & 0xffffu, big >> 16));
        small = __reduce_min_sync(0xffffffffu, min(small & 0xffffu, small >> 16)) + 1;
        // exponents -24 .. 15, of subnormal numbers too; 128 of infinities and NaN
        const int most = static_cast<int>(__float_as_uint(half_bits_to_float(big)) >> 23) - 127;
        const int least = static_cast<int>(__float_as_uint(half_bits_to_float(small)) >> 23) - 127;
        odd = most > 15;
        apart = odd || (big != 0 && most - least > 7);
        if (big == 0 || apart) {
          e_new = up_exp;
        } else if (most > 1 || least < -7) {  // (p d_v 2^13 is below 2^15 up to here)
          const auto times = [&](int by) {
            const uint32_t f = static_cast<uint32_t>(by + 15) << 10;
#pragma unroll
            for (int gi = 0; gi < TG; ++gi)
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) vs[gi][b][h] = h2_bits(__hmul2(bits_h2(vs[gi][b][h]), bits_h2(f | f << 16)));
          };
          e_new = 13 - most;
          const int by = max(-14, min(15, -most));  // (2^by is a normal fp16 number)
          times(by);
          if (by != -most) times(-most - by);
        }
      }

      // ---- scores ----
      float2 z[OCT][TG][2];
#pragma unroll
      for (int o = 0; o < OCT; ++o)
#pragma unroll
        for (int gi = 0; gi < TG; ++gi) z[o][gi][0] = z[o][gi][1] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int run = 0; run < kv_runs(NB, KQ8); ++run) {
        const int first = kv_run_first(NB, KQ8, run), n = kv_run_blocks(NB, KQ8, run), bytes = n * (KQ8 ? 8 : 4);
        uint32_t kw[TG][2][4];
#pragma unroll
        for (int gi = 0; gi < TG; ++gi)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t at = stage + gi * C::kGroupBytes + first * (KQ8 ? 512 : 256) + (j * 32 + lane) * bytes;
            if (bytes == 16) {
              const uint4 v = lds_u4(at);
              kw[gi][j][0] = v.x, kw[gi][j][1] = v.y, kw[gi][j][2] = v.z, kw[gi][j][3] = v.w;
            } else if (bytes == 8) {
              const uint2 v = lds_u2(at);
              kw[gi][j][0] = v.x, kw[gi][j][1] = v.y;
            } else {
              kw[gi][j][0] = lds_u32(at);
            }
          }
#pragma unroll
        for (int r = 0; r < (KQ8 ? 2 : 4); ++r) {
          if (r >= n) continue;
          const int b = first + r;
          uint4 q[OCT][TERMS];
#pragma unroll
          for (int o = 0; o < OCT; ++o)
#pragma unroll
            for (int i = 0; i < TERMS; ++i) q[o][i] = lds_u4(qfrag_s + ((o * NB + b) * TERMS + i) * 512);
#pragma unroll
          for (int gi = 0; gi < TG; ++gi) {
            // keys (g >> 1) + 4 (g & 1) and 8 more are rows g and g + 8
            uint4 k0, k1;
            uint32_t *a0 = &k0.x, *a1 = &k1.x;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (KQ8) {
                const uint32_t w0 = kw[gi][j][(2 * r) & 3] ^ 0x80808080u, w1 = kw[gi][j][(2 * r + 1) & 3] ^ 0x80808080u;
                a0[j] = q8_pair<0x5250>(w0, magic), a0[j + 2] = q8_pair<0x5351>(w0, magic);
                a1[j] = q8_pair<0x5250>(w1, magic), a1[j + 2] = q8_pair<0x5351>(w1, magic);
              } else {
                const uint32_t w = kw[gi][j][r], w8 = w >> 8;
                a0[j] = q4_low(w, magic), a0[j + 2] = q4_low(w8, magic);
                a1[j] = q4_high(w, magic), a1[j + 2] = q4_high(w8, magic);
              }
            }
            const uint2 ks = lds_u2(stage + gi * C::kGroupBytes + kv_code_bytes(NB, KQ8) + ((g >> 1) * NB + b) * 8);
            const float2 d = __half22float2(bits_h2(__byte_perm(ks.x, ks.y, g & 1 ? 0x7632 : 0x5410)));
#pragma unroll
            for (int o = 0; o < OCT; ++o) {
              float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int i = TERMS - 1; i >= 0; --i)
                c = mma_f16(k1, q[o][i].z, q[o][i].w, mma_f16(k0, q[o][i].x, q[o][i].y, c));
              z[o][gi][0] = __ffma2_rn(make_float2(d.x, d.x), make_float2(c.x, c.y), z[o][gi][0]);
              z[o][gi][1] = __ffma2_rn(make_float2(d.y, d.y), make_float2(c.z, c.w), z[o][gi][1]);
            }
          }
        }
      }

      if (!full) {
#pragma unroll
        for (int gi = 0; gi < TG; ++gi)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int key = key0 + gi * kKvGroup + (g >> 1) + 4 * (g & 1) + 8 * j;
#pragma unroll
            for (int o = 0; o < OCT; ++o) {
              if (!(ok >> gi & 1) || key > last[o].x || key < low[o].x) z[o][gi][j].x = -INFINITY;
              if (!(ok >> gi & 1) || key > last[o].y || key < low[o].y) z[o][gi][j].y = -INFINITY;
            }
          }
      }

      // ---- running maximum and sum ----
      float2 keep[OCT];
      __half2 ph[OCT][TG][2], pl[FINE ? OCT : 1][TG][2];  // weights, transposed: row g, keys t and t + 4 (and 8 more)
      const float turn = __uint_as_float(static_cast<uint32_t>(e_new - up_exp + 127) << 23);
      up_exp = e_new;
#pragma unroll
      for (int o = 0; o < OCT; ++o) {
        float2 m = make_float2(-INFINITY, -INFINITY);
#pragma unroll
        for (int gi = 0; gi < TG; ++gi) {
          m.x = fmaxf(m.x, fmaxf(z[o][gi][0].x, z[o][gi][1].x));
          m.y = fmaxf(m.y, fmaxf(z[o][gi][0].y, z[o][gi][1].y));
        }
#pragma unroll
        for (int by = 4; by < 32; by <<= 1) {
          m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, by));
          m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, by));
        }
        m = make_float2(fmaxf(m.x * factor[o].x, top[o].x), fmaxf(m.y * factor[o].y, top[o].y));
        const float2 ref = make_float2(m.x == -INFINITY ? 0.0f : m.x, m.y == -INFINITY ? 0.0f : m.y);
        // Products are rounded as the maximum's was, and 13 less the maximum downwards:
        // no weight is above 2^13, nor the largest lost, however large the scores.
        const float2 from13 = make_float2(__fsub_rd(13.0f, ref.x), __fsub_rd(13.0f, ref.y));
        const float2 k = make_float2(exp2_approx(top[o].x - ref.x), exp2_approx(top[o].y - ref.y));
        top[o] = m;
        float2 add = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int gi = 0; gi < TG; ++gi)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // (__fmul_rn one by one: a packed product before a packed sum became one operation)
            float2 w = make_float2(__fmul_rn(z[o][gi][j].x, factor[o].x), __fmul_rn(z[o][gi][j].y, factor[o].y));
            w = __fadd2_rn(w, from13);
            w = make_float2(exp2_approx(w.x), exp2_approx(w.y));
            add = __fadd2_rn(add, w);
            z[o][gi][j] = w;
            if (FINE) {
              __half2 h, l;
              split_f16(w, h, l);
              ph[o][gi][j] = transpose8(h), pl[FINE ? o : 0][gi][j] = transpose8(l);
            } else {
              ph[o][gi][j] = transpose8(__float22half2_rn(w));
            }
          }
        sum[o] = __ffma2_rn(sum[o], k, add);
        keep[o] = make_float2(k.x * turn, k.y * turn);
      }

      // ---- outputs ----
      // Scales of sizes far apart: in fp16 the small ones' weights would keep few bits,
      // whichever rows and dims the large ones belong to. And a value that is not
      // finite belongs to the rows that see it and to no other, but 0 times it in a
      // matrix product is not 0. (16 x 8192 keys of 8 heads of 128, Q4_0, fp32: 86 us
      // where every step is like that, 55 us where none is.)
      if (apart) {
#pragma unroll
        for (int o = 0; o < OCT; ++o)
#pragma unroll
          for (int n = 0; n < NB * 4; ++n) acc[o][n] = make_float2(acc[o][n].x * keep[o].x, acc[o][n].y * keep[o].y);
        if constexpr (NB > 4 && OCT > 1) {
          KvApart<NB, OCT, TG> s;
#pragma unroll
          for (int o = 0; o < OCT; ++o) {
            s.last[o] = last[o], s.low[o] = low[o];
#pragma unroll
            for (int n = 0; n < NB * 4; ++n) s.acc[o][n] = acc[o][n];
#pragma unroll
            for (int gi = 0; gi < TG; ++gi) s.z[o][gi][0] = z[o][gi][0], s.z[o][gi][1] = z[o][gi][1];
          }
          kv_add_apart_call<NB, VQ8, C::kGroupBytes>(s, stage + C::kKeyPart, ok, key0, e_new, odd, magic);
#pragma unroll
          for (int o = 0; o < OCT; ++o)
#pragma unroll
            for (int n = 0; n < NB * 4; ++n) acc[o][n] = s.acc[o][n];
        } else {
          kv_add_apart<NB, VQ8, C::kGroupBytes>(acc, z, stage + C::kKeyPart, ok, key0, e_new, odd, last, low, magic);
        }
      } else {
#pragma unroll
        for (int run = 0; run < kv_runs(NB, VQ8); ++run) {
          const int first = kv_run_first(NB, VQ8, run), n = kv_run_blocks(NB, VQ8, run);
          uint32_t vw[TG][4][2];
#pragma unroll
          for (int gi = 0; gi < TG; ++gi)
            kv_value_words<NB, VQ8>(vw[gi], stage + gi * C::kGroupBytes + C::kKeyPart, run);
#pragma unroll
          for (int r = 0; r < (VQ8 ? 2 : 4); ++r) {
            if (r >= n) continue;
            const int b = first + r;
            // value codes of the block: columns of 4 tiles, tokens in pairs
            uint32_t vb[TG][4][2];
#pragma unroll
            for (int gi = 0; gi < TG; ++gi)
              kv_value_tiles<VQ8>(vb[gi], vw[gi], r, magic);
#pragma unroll
            for (int o = 0; o < OCT; ++o) {
              float4 c[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
              uint32_t w[TG][TERMS][2];
#pragma unroll
              for (int gi = 0; gi < TG; ++gi)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const __half2 d = bits_h2(vs[gi][b][j]), hi = __hmul2(ph[o][gi][j], d);
                  w[gi][0][j] = h2_bits(hi);
                  if (FINE)  // p d_v = hi + what hi leaves of ph d_v + pl d_v
                    w[gi][TERMS - 1][j] = h2_bits(__hfma2(pl[FINE ? o : 0][gi][j], d, __hfma2(ph[o][gi][j], d, __hneg2(hi))));
                }
#pragma unroll
              for (int i = TERMS - 1; i >= 0; --i)
#pragma unroll
                for (int gi = 0; gi < TG; ++gi)
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    c[h] = mma_f16(make_uint4(vb[gi][2 * h][0], vb[gi][2 * h + 1][0], vb[gi][2 * h][1], vb[gi][2 * h + 1][1]),
                                   w[gi][i][0], w[gi][i][1], c[h]);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                acc[o][b * 4 + 2 * h] = __ffma2_rn(acc[o][b * 4 + 2 * h], keep[o], make_float2(c[h].x, c[h].y));
                acc[o][b * 4 + 2 * h + 1] = __ffma2_rn(acc[o][b * 4 + 2 * h + 1], keep[o], make_float2(c[h].z, c[h].w));
              }
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      fill();
    }

    // ---- the item's end for this warp ----
    const bool whole = use.a == 0 && use.b == use.n;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - up_exp) << 23);
    const int piece = 2 * warp + (use.a == 0 ? 1 : 0);
    float *kept = use.left <= 0 ? reinterpret_cast<float *>(own) : warp_slots + piece * C::kPiece;
    if (!whole && lane == 0) pieces[piece] = Piece{use.seq, use.head, use.tile, use.a, use.b, use.n, kept};
    __syncwarp();
#pragma unroll
    for (int o = 0; o < OCT; ++o) {
      float2 l = make_float2(sum[o].x * 0x1p-13f, sum[o].y * 0x1p-13f);
#pragma unroll
      for (int by = 4; by < 32; by <<= 1) {
        l.x += __shfl_xor_sync(0xffffffffu, l.x, by);
        l.y += __shfl_xor_sync(0xffffffffu, l.y, by);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = o * 8 + 2 * t + i, row = use.tile * C::kRows + r;
        if (row >= p.rows) continue;
        const float li = i ? l.y : l.x;
        if (!whole && g == 0) piece_ml[piece][r] = make_float2(i ? top[o].y : top[o].x, li);
        const float by = whole ? (li > 0.0f ? down / li : 0.0f) : down;
        const int64_t out = kv_out_at(p, use.seq, use.head, row, D) + 2 * g;
        float *part = kept + r * (D + 8) + 2 * g;
#pragma unroll
        for (int n = 0; n < NB * 2; ++n) {  // half blocks
          const float2 x = acc[o][n / 2 * 4 + n % 2], y = acc[o][n / 2 * 4 + n % 2 + 2];
          const float2 v = make_float2((i ? x.y : x.x) * by, (i ? y.y : y.x) * by);
          if (whole)
            kv_store(p, out + n * 16, v);
          else
            *reinterpret_cast<float2 *>(part + n * 16) = v;
        }
      }
    }
    use.a = use.b;
  }

  // ---- partial results ----
  // In the line's order a warp's piece that begins its item (odd) begins a group
  // of pieces of one item, the others go on with the one before. A group is
  // added up by warps, 32 quads of outputs each, to the result if it is the whole
  // item, else to one of the block's two slots (only its first and its last item
  // can lie in other blocks too). Then those two, if this block is the last of
  // theirs to be done, from all their blocks' slots.
  __syncthreads();
  const uint32_t valid = __ballot_sync(0xffffffffu, lane < 2 * NW && pieces[min(lane, 2 * NW - 1)].seq >= 0);
  const uint32_t begins = (valid & 0xaaaaaaaau) | (valid & (0u - valid));
  const int groups = __popc(begins);
  constexpr int kChunks = (C::kRows * (D / 4) + 31) / 32;
  if (tid < groups) {
    const int e = __fns(begins, 0, tid + 1);
    const uint32_t after = begins & ~((2u << e) - 1), mine = valid & (after ? (after & (0u - after)) - 1 : ~0u) & ~((1u << e) - 1);
    const Piece first = pieces[e];
    jobs[tid] = Job{first.seq, first.head, first.tile, first.a, mine, __popc(mine),
                    first.a == 0 && pieces[31 - __clz(mine)].b == first.n};
  }
  __syncthreads();
  if (groups == 0) return;
  int njobs = groups;
#pragma unroll 1
  for (int phase = 0; phase < 2; ++phase) {
#pragma unroll 1
    for (int it = warp; it < njobs * kChunks; it += NW) {
      const int job = it / kChunks, i = (it - job * kChunks) * 32 + lane, r = i / (D / 4), d = (i - r * (D / 4)) * 4;
      const Job w = jobs[job];
      const int row = w.tile * C::kRows + r;
      if (r >= C::kRows || row >= p.rows) continue;
      KvSum x;
      uint32_t left = w.pieces;  // phase 0: the group's pieces; phase 1: its first block
#pragma unroll 1
      for (int k = 0; k < w.n; k += 8) {
        float2 ml[8];
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ml[j] = make_float2(-INFINITY, 0.0f), v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k + j >= w.n) continue;  // (nothing in its place: results may be infinite)
          if (phase == 0) {
            const int e = __ffs(left) - 1;
            left &= left - 1;
            ml[j] = piece_ml[e][r];
            v[j] = *reinterpret_cast<const float4 *>(pieces[e].out + r * (D + 8) + d);
          } else {  // slot 1 of the first block, slot 0 of the others
            const int part = k + j;
            const float *o = p.a.ws + kKvMaxBlocks * 4 + (2 * (static_cast<int>(w.pieces) + part) + (part == 0 ? 1 : 0)) * kSlot;
            ml[j] = kv_load2(o + C::kRows * D + r * 2);
            v[j] = kv_load4(o + r * D + d);
          }
        }
        x.add(ml, v);
      }
      if (w.whole) {
        const float inv = x.l > 0.0f ? 1.0f / x.l : 0.0f;
        kv_store(p, kv_out_at(p, w.seq, w.head, row, D) + d,
                 make_float4(x.o.x * inv, x.o.y * inv, x.o.z * inv, x.o.w * inv));
      } else {
        float *slot = block_slots + (w.a == 0 ? kSlot : 0);
        *reinterpret_cast<float4 *>(slot + r * D + d) = x.o;
        if (d == 0) *reinterpret_cast<float2 *>(slot + C::kRows * D + r * 2) = make_float2(x.m, x.l);
      }
    }
    if (phase) break;
    const int split0 = !jobs[0].whole, split1 = groups > 1 && !jobs[groups - 1].whole;
    if (!split0 && !split1) break;
    __syncthreads();
    if (warp < 2 && (warp ? split1 : split0)) {
      const Job w = jobs[warp ? groups - 1 : 0];
      const KvShare share = kept_share;
      // The item's blocks: those of its first group and of its last unit.
      int64_t at = scan[w.seq / chunk];
      for (int s = w.seq / chunk * chunk; s < w.seq; ++s) at += kv_units(kv_seq(p, s, status).n) * per_seq;
      const int64_t units = kv_units(kv_seq(p, w.seq, status).n);
      at += (static_cast<int64_t>(w.head) * p.tiles + w.tile) * units;
      const int b0 = share.block_of(at + kKvItemCost), n = share.block_of(at + units - 1) - b0 + 1;
      // Marks need no first value: one that another call left is not this call's.
      // Of two blocks that end at once each may find all marks and join: the
      // results are the same. The joining block takes the marks off, for a replay.
      const auto mark_of = [&](int k) { return marks + 2 * (b0 + k) + (k == 0 ? 1 : 0); };
      __threadfence();  // (the block's results, written before the barrier)
      if (lane == 0) *mark_of(blockIdx.x - b0) = p.epoch;
      __syncwarp();
      __threadfence();
      bool all = true;
      for (int k = lane; k < n; k += 32) all = all && *mark_of(k) == p.epoch;
      all = __all_sync(0xffffffffu, all);
      __threadfence();
      if (all)
        for (int k = lane; k < n; k += 32) *mark_of(k) = 0;
      if (lane == 0) joins[warp] = Job{w.seq, w.head, w.tile, 0, static_cast<uint32_t>(b0), all ? n : 0, true};
    }
    __syncthreads();
    const int join0 = split0 && joins[0].n, join1 = split1 && joins[1].n;
    njobs = join0 + join1;
    if (tid < njobs) jobs[tid] = joins[tid == 0 && join0 ? 0 : 1];
    __syncthreads();
  }
}

template <int NB, bool KQ8, bool VQ8, int OCT, bool FINE>
__global__ void __launch_bounds__(KvCfg<NB, KQ8, VQ8, OCT, FINE>::kNW * 32, 1)
    kv_attn_kernel(const __grid_constant__ KvLaunch p, uint32_t *status) {
  kv_attn_body<NB, KQ8, VQ8, OCT, FINE>(p, status);
}

// Launch of one instance; the attribute is set once per device.
template <int NB, bool KQ8, bool VQ8, int OCT, bool FINE>
cudaError_t kv_attn_launch(const DevInfo &dev, KvLaunch &p, uint32_t *status, cudaLaunchConfig_t cfg) {
  using C = KvCfg<NB, KQ8, VQ8, OCT, FINE>;
  const auto kernel = kv_attn_kernel<NB, KQ8, VQ8, OCT, FINE>;
  static DeviceFlags ready;
  if (!ready.done(dev.device)) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    ready.set(dev.device);
  }
  cfg.blockDim = dim3(C::kNW * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  p.tiles = (p.rows + C::kRows - 1) / C::kRows;
  return cudaLaunchKernelEx(&cfg, kernel, p, status);
}

// Octets of rows that a warp takes at a time: all of them while most of their sums
// stay in registers (three of 128 with fp32 queries spill 76 bytes, four with bf16
// ones 112, two of 256 up to 236), else two. 16 x 8192 keys of 8 heads of 128, Q4_0,
// take for 1, 2, 3, 4 octets at a time 55, 88, 141, 195 us with fp32 queries (four as
// two and two 160) and 47, 68, 107, 143 us with bf16.
constexpr int kv_attn_octets(int nb, int rows, bool fine) {
  const int need = (rows + 7) / 8, most = nb > 4 ? 2 : fine ? 3 : 4;
  return need <= most ? need : 2;
}

template <int NB, bool KQ8, bool VQ8, bool FINE>
cudaError_t kv_attn_rows(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg) {
  switch (kv_attn_octets(NB, p.rows, FINE)) {
    case 1: return kv_attn_launch<NB, KQ8, VQ8, 1, FINE>(dev, p, status, cfg);
    case 2: return kv_attn_launch<NB, KQ8, VQ8, 2, FINE>(dev, p, status, cfg);
    case 3:
      if constexpr (NB <= 4) return kv_attn_launch<NB, KQ8, VQ8, 3, FINE>(dev, p, status, cfg);
      return cudaErrorInvalidValue;
    default:
      if constexpr (NB <= 4 && !FINE) return kv_attn_launch<NB, KQ8, VQ8, 4, FINE>(dev, p, status, cfg);
      return cudaErrorInvalidValue;
  }
}

// fp32 queries in two fp16 terms, bf16 ones (whose outputs keep 8 bits) in one, and
// the weights with them.
template <int NB, bool KQ8, bool VQ8>
cudaError_t kv_attn_dtype(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg) {
  return p.bf16 ? kv_attn_rows<NB, KQ8, VQ8, false>(dev, p, status, cfg)
                : kv_attn_rows<NB, KQ8, VQ8, true>(dev, p, status, cfg);
}

template <int NB>
cudaError_t kv_attn_types(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg) {
  if (p.f.kq8)
    return p.f.vq8 ? kv_attn_dtype<NB, true, true>(dev, p, status, cfg) : kv_attn_dtype<NB, true, false>(dev, p, status, cfg);
  return p.f.vq8 ? kv_attn_dtype<NB, false, true>(dev, p, status, cfg) : kv_attn_dtype<NB, false, false>(dev, p, status, cfg);
}

// kv_attn_d*.cu
cudaError_t kv_attn_d64(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg);
cudaError_t kv_attn_d96(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg);
cudaError_t kv_attn_d128(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg);
cudaError_t kv_attn_d192(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg);
cudaError_t kv_attn_d256(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg);

}  // namespace qmm
