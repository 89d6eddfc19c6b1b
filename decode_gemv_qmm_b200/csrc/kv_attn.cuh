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

// C += A . B, 16 x 8 x 16, fp16 operands, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Two fp32 values as fp16 pairs hi + lo: 22 bits of each, when they are neither
// above 65504 nor so small that lo falls below fp16's 2^-24.
__device__ __forceinline__ void split_f16(float x, float y, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = h2_bits(h);
  lo = h2_bits(__floats2half2_rn(x - f.x, y - f.y));
}

// Codes as fp16 pairs, exact: 0x6400 | c is 1024 + c.
//  low nibbles of bytes 0 and 2 of w
__device__ __forceinline__ uint32_t q4_low(uint32_t w) {
  return h2_bits(__hsub2(bits_h2((w & 0x000f000fu) | 0x64006400u), bits_h2(0x64086408u)));  // - 1032
}
//  high nibbles of bytes 0 and 2 of w: (1024 + 16 c) / 16 - 72
__device__ __forceinline__ uint32_t q4_high(uint32_t w) {
  return h2_bits(__hfma2(bits_h2((w & 0x00f000f0u) | 0x64006400u), bits_h2(0x2c002c00u), bits_h2(0xd480d480u)));
}
//  two bytes of w (already xor 0x80808080) chosen by sel, as codes
template <uint32_t kSel>
__device__ __forceinline__ uint32_t q8_pair(uint32_t w) {
  return h2_bits(__hsub2(bits_h2(__byte_perm(w, 0x64646464u, kSel)), bits_h2(0x64806480u)));  // - 1152
}

__device__ __forceinline__ uint2 lds_u2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// ---- configuration ----------------------------------------------------------

// Floats of one partial result: rows x (D + maximum and sum).
__host__ __device__ constexpr int64_t kv_attn_slot_floats(int rows, int d) { return static_cast<int64_t>(rows) * (d + 2); }

// What the main kernel tells the joining kernel about block c's last item.
struct KvSplit {
  int seq, head, tile, last;  // seq < 0: nothing to join; last: the block that holds the item's end
};

constexpr int kKvMaxBlocks = 1184;   // most blocks of a launch
constexpr int kKvRowsMax = 32;       // most rows of a partial result

template <int NB, bool KQ8, bool VQ8, int MT>
struct KvCfg {
  static constexpr int kD = NB * 32;
  static constexpr int kKeyPart = kv_part_bytes(NB, KQ8);
  static constexpr int kGroupBytes = kKeyPart + kv_part_bytes(NB, VQ8);
  static constexpr int kTG = kGroupBytes <= 4608 ? 2 : 1;  // groups of a step
  static constexpr int kStageBytes = kTG * kGroupBytes;
  static constexpr int kRowPad = kD + 16;                  // floats of a row in the joining buffer
  static constexpr int kRows = 8 * MT;
  static constexpr int kQBytes = MT * NB * 1024;
  static constexpr int kFixed = kQBytes + 1024;            // query fragments, barriers, statistics
  static constexpr int warp_bytes(int stages) { return stages * kStageBytes + 8 * kRowPad * 4; }
  static constexpr int kBudget = 220 * 1024 - kFixed;
  static constexpr int kNW = 8 * warp_bytes(2) <= kBudget ? 8 : 4;
  static constexpr int kStages = kNW * warp_bytes(4) <= kBudget ? 4 : kNW * warp_bytes(3) <= kBudget ? 3 : 2;
  static constexpr int kSmem = kFixed + kNW * warp_bytes(kStages);
  static_assert(kNW * warp_bytes(kStages) <= kBudget, "stages do not fit");
};

// A launch's constants.
struct KvLaunch {
  KvForm f;
  KvAttnArgs a;
  int ratio, rows, tiles;  // query heads of a key/value head; rows M ratio of one; tiles of kRows rows
  int min_groups;          // least groups of a block
  int bf16;
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

__device__ __forceinline__ void kv_store(const KvLaunch &p, int64_t at, float4 v) {
  if (p.bf16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.a.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
  } else {
    *reinterpret_cast<float4 *>(static_cast<float *>(p.a.out) + at) = v;
  }
}

// Output offset of row r (of one key/value head's M x ratio rows).
__device__ __forceinline__ int64_t kv_out_at(const KvLaunch &p, int s, int head, int r, int d) {
  const int i = r / p.ratio, h = r - i * p.ratio;
  return ((static_cast<int64_t>(s) * p.a.m + i) * p.a.hq + head * p.ratio + h) * d;
}

// ---- the kernel -------------------------------------------------------------
//
// Work is the line of all groups of all items, an item being (sequence, head,
// tile of query rows); each block takes an equal run of it, whatever the
// sequences' lengths, and its warps equal parts of each item's run. A warp
// brings its groups by bulk copies into a ring of its own and holds the running
// maximum, sum and outputs of its keys; at an item's end the warps are joined
// in shared memory. An item that lies in one block is finished there; the
// others leave partial results, which a second launch joins.
//
// Products run on the tensor cores with the cached codes as exact fp16
// integers. Eight query rows fill a 16-row tile: rows 0..7 hold the leading
// fp16 term and rows 8..15 the remainder (22 bits together), so fp32 accuracy
// costs no more products than the tile has. A key's block scale multiplies the
// finished 32-dim dot in fp32; a value's block scale goes into the weight,
// p d_v, before it is split. Each step's sums are added to fp32 registers
// outside the tensor core, which does not round its sums to nearest.
template <int NB, bool KQ8, bool VQ8, int MT>
__device__ __forceinline__ void kv_attn_body(const KvLaunch &p, uint32_t *status) {
  using C = KvCfg<NB, KQ8, VQ8, MT>;
  constexpr int NW = C::kNW, TG = C::kTG, S = C::kStages, D = C::kD;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[NW * S];
  __shared__ float w_max[NW][8], w_sum[NW][8];
  __shared__ int64_t scan[NW];
  __shared__ int start_seq;
  __shared__ int64_t start_base;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  __shared__ float q_factor[C::kRows];
  uint4 *qfrag = reinterpret_cast<uint4 *>(smem);  // [MT][NB][2][32]
  const uint32_t qfrag_s = smem_u32(qfrag);
  float *joins = reinterpret_cast<float *>(smem + C::kQBytes);
  float *join = joins + warp * 8 * C::kRowPad;
  uint8_t *ring = smem + C::kQBytes + NW * 8 * C::kRowPad * 4 + warp * S * C::kStageBytes;
  uint64_t *bar = bars + warp * S;

  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(bar + i, 1);
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  // The line's length and this block's run of it.
  const int64_t per_seq = static_cast<int64_t>(p.f.heads) * p.tiles;
  const int chunk = (p.a.batch + NW * 32 - 1) / (NW * 32);
  const int s0 = min(p.a.batch, tid * chunk), s1 = min(p.a.batch, s0 + chunk);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) mine += kv_seq(p, s, status).n * per_seq;
  int64_t incl = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < NW; ++w) {
    if (w < warp) incl += scan[w];
    total += scan[w];
  }
  // Rows of sequences without keys.
  for (int s = blockIdx.x; s < p.a.batch; s += gridDim.x) {
    if (kv_seq(p, s, status).n) continue;
    const int64_t n = static_cast<int64_t>(p.a.m) * p.a.hq * D;
    for (int64_t e = tid * 4; e < n; e += NW * 128) kv_store(p, s * n + e, make_float4(0.f, 0.f, 0.f, 0.f));
  }
  const int64_t blocks = min(static_cast<int64_t>(gridDim.x), (total + p.min_groups - 1) / p.min_groups);
  KvSplit *splits = reinterpret_cast<KvSplit *>(p.a.ws);
  float *slots = p.a.ws + kKvMaxBlocks * 4;
  if (blockIdx.x >= blocks) {
    if (tid == 0) splits[blockIdx.x].seq = -1;
    return;
  }
  int64_t pos = blockIdx.x * total / blocks;
  const int64_t end = (blockIdx.x + 1) * total / blocks;
  if (incl - mine <= pos && pos < incl) {
    int64_t base = incl - mine;
    int s = s0;
    for (;; ++s) {
      const int64_t n = kv_seq(p, s, status).n * per_seq;
      if (pos < base + n) break;
      base += n;
    }
    start_seq = s;
    start_base = base;
  }
  __syncthreads();
  int seq = start_seq;
  int64_t base = start_base;

  // The item at `pos`, and this warp's groups of it.
  struct Run {
    int seq, head, tile, len, n, a, b;  // item's groups [a, b) of n; a group's number counts from the sequence's first
    int lo, hi;                         // this warp's groups, numbered in the sequence
  } run, next;
  auto locate = [&](Run &r) {
    KvSeq q = kv_seq(p, seq, status);
    while (pos >= base + q.n * per_seq) {
      base += q.n * per_seq;
      q = kv_seq(p, ++seq, status);
    }
    const int64_t in = pos - base;
    const int item = static_cast<int>(in / q.n);
    r.seq = seq;
    r.head = item / p.tiles;
    r.tile = item - r.head * p.tiles;
    r.len = q.len;
    r.n = q.n;
    r.a = static_cast<int>(in - static_cast<int64_t>(item) * q.n);
    r.b = static_cast<int>(min(static_cast<int64_t>(q.n), r.a + (end - pos)));
    const int ng = r.b - r.a;
    r.lo = q.first + r.a + static_cast<int>(static_cast<int64_t>(ng) * warp / NW);
    r.hi = q.first + r.a + static_cast<int>(static_cast<int64_t>(ng) * (warp + 1) / NW);
  };

  const int per_page = p.f.page / kKvGroup;
  const int page_shift = 31 - __clz(per_page);
  const uint64_t policy = l2_evict_first_policy();
  const uint32_t ring_s = smem_u32(ring);
  uint32_t put = 0, got = 0;  // stages filled and used so far (ring positions)
  uint32_t ok_bits = 0;       // groups of the ring whose page exists
  bool dead = false;          // a wait ran out

  // Fill the ring's next stage with the step of groups [grp, grp + TG) of `r`.
  auto fill = [&](const Run &r, int grp) {
    const int st = put % S;
    uint32_t ok = 0;
    const int32_t *table = p.a.table + r.seq * p.a.table_stride;
    int64_t page[TG];
#pragma unroll
    for (int i = 0; i < TG; ++i) {
      page[i] = -1;
      if (grp + i < r.hi) {
        page[i] = __ldg(table + ((grp + i) >> page_shift));
        if (page[i] < 0 || page[i] >= p.f.pages) {
          page[i] = -1;
          if (lane == 0) atomicOr(status, kDevBadIndex);
        }
      }
      if (page[i] >= 0) ok |= 1u << i;
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(bar + st, __popc(ok) * C::kGroupBytes);
#pragma unroll
      for (int i = 0; i < TG; ++i)
        if (page[i] >= 0)
          bulk_g2s(ring + st * C::kStageBytes + i * C::kGroupBytes,
                   p.a.cache + ((page[i] * p.f.heads + r.head) * per_page + ((grp + i) & (per_page - 1))) *
                                   static_cast<int64_t>(C::kGroupBytes),
                   C::kGroupBytes, bar + st, policy);
    }
    ok_bits = (ok_bits & ~(((1u << TG) - 1) << (st * TG))) | ok << (st * TG);
    ++put;
  };

  // Query rows of `r` as fragments, each row brought to [2^14, 2^15) by a power
  // of two so that both terms stay in fp16's range; its inverse, with the
  // softmax's scale and log2(e), is the factor of the row's scores. Warp w
  // makes the fragments of units (tile, block) w, w + NW, ...
  auto load_q = [&](const Run &r) {
    for (int u = warp; u < MT * NB; u += NW) {
      const int mt = u / NB, mine_b = u - mt * NB;
      const int row = r.tile * C::kRows + mt * 8 + g;
      const bool there = row < p.rows;
      const int i = there ? row / p.ratio : 0, h = there ? row - i * p.ratio : 0;
      const int64_t at = r.seq * p.a.q_seq + i * p.a.q_tok +
                         (static_cast<int64_t>(r.head) * p.ratio + h) * p.a.q_head + 4 * t;
      float x[8], top = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int64_t e = at + b * 32 + half * 16;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (there) {
            if (p.bf16) {
              const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.a.q) + e);
              v = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                              __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
            } else {
              v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.a.q) + e);
            }
          }
          top = fmaxf(top, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
          if (b == mine_b) x[half * 4] = v.x, x[half * 4 + 1] = v.y, x[half * 4 + 2] = v.z, x[half * 4 + 3] = v.w;
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // exponent of top, at least -100 (smaller rows keep fewer bits of scores that are 0 anyway)
      const int ex = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
      const float up = __uint_as_float(static_cast<uint32_t>(14 - ex + 127) << 23);
      if (mine_b == 0 && t == 0)
        q_factor[mt * 8 + g] = p.a.scale * 1.44269504088896f * __uint_as_float(static_cast<uint32_t>(ex - 14 + 127) << 23);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint4 f;
        split_f16(x[half * 4] * up, x[half * 4 + 2] * up, f.x, f.y);
        split_f16(x[half * 4 + 1] * up, x[half * 4 + 3] * up, f.z, f.w);
        qfrag[(u * 2 + half) * 32 + lane] = f;
      }
    }
  };

  locate(run);
  for (int i = 0; i < S; ++i)
    if (run.lo + i * TG < run.hi) fill(run, run.lo + i * TG);
  load_q(run);
  __syncthreads();

  while (true) {
    // ---- this warp's groups of the item ----
    float top[MT], sum[MT], acc[MT][NB * 4][2];
    int last[MT], low[MT];
    float factor[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      top[mt] = -INFINITY;
      sum[mt] = 0.0f;
#pragma unroll
      for (int n = 0; n < NB * 4; ++n) acc[mt][n][0] = acc[mt][n][1] = 0.0f;
      const int i = min((run.tile * C::kRows + mt * 8 + g) / p.ratio, p.a.m - 1);
      last[mt] = run.len - p.a.m + i;
      low[mt] = p.a.window > 0 ? max(0, last[mt] - p.a.window + 1) : 0;
      factor[mt] = q_factor[mt * 8 + g];
    }
    const int low_all = p.a.window > 0 ? max(0, run.len - p.a.m - p.a.window + 1) : 0;
    int up_exp = 0;  // acc is 2^up_exp times the outputs' sums

    for (int grp = run.lo; grp < run.hi; grp += TG) {
      const int st = got % S;
      if (!dead && !mbar_wait(bar + st, (got / S) & 1)) {
        // Nothing more is copied; what is in flight is waited for once more.
        bool drained = true;
        for (uint32_t i = got; i != put; ++i) drained = mbar_wait(bar + i % S, (i / S) & 1) && drained;
        if (lane == 0) atomicOr(status, kDevTimeoutFull | (drained ? 0u : kDevTimeoutDrain));
        dead = true;
      }
      ++got;
      if (dead) continue;
      const uint32_t stage = ring_s + st * C::kStageBytes;
      const uint32_t ok = ok_bits >> (st * TG) & ((1u << TG) - 1);
      const int key0 = grp * kKvGroup;
      const bool full = ok == (1u << TG) - 1 && key0 + TG * kKvGroup <= run.len - p.a.m + 1 &&
                        (p.a.window == 0 || key0 >= run.len - p.a.window);

      // ---- scores ----
      float z[MT][TG][2][2];
      {
        constexpr int KW = KQ8 ? 2 * NB : NB;
        uint32_t kw[TG][2][KW];
        uint32_t ks[TG][NB][2];
#pragma unroll
        for (int gi = 0; gi < TG; ++gi) {
          const uint32_t part = stage + gi * C::kGroupBytes;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int first = 0; first < NB;) {
              const int n = kv_run(NB, KQ8, first).n, bytes = n * (KQ8 ? 8 : 4), w0 = first * (KQ8 ? 2 : 1);
              const uint32_t at = part + first * (KQ8 ? 512 : 256) + (j * 32 + lane) * bytes;
              if (bytes == 16) {
                const uint4 v = lds_u4(at);
                kw[gi][j][w0] = v.x, kw[gi][j][w0 + 1] = v.y, kw[gi][j][w0 + 2] = v.z, kw[gi][j][w0 + 3] = v.w;
              } else if (bytes == 8) {
                const uint2 v = lds_u2(at);
                kw[gi][j][w0] = v.x, kw[gi][j][w0 + 1] = v.y;
              } else {
                kw[gi][j][w0] = lds_u32(at);
              }
              first += n;
            }
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint2 v = lds_u2(part + kv_code_bytes(NB, KQ8) + (t * NB + b) * 8);
            ks[gi][b][0] = v.x, ks[gi][b][1] = v.y;
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int gi = 0; gi < TG; ++gi) z[mt][gi][0][0] = z[mt][gi][0][1] = z[mt][gi][1][0] = z[mt][gi][1][1] = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint4 qa[MT][2];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            qa[mt][0] = lds_u4(qfrag_s + (((mt * NB + b) * 2) * 32 + lane) * 16);
            qa[mt][1] = lds_u4(qfrag_s + (((mt * NB + b) * 2 + 1) * 32 + lane) * 16);
          }
#pragma unroll
          for (int gi = 0; gi < TG; ++gi)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t k00, k01, k10, k11;
              if (KQ8) {
                const uint32_t w0 = kw[gi][j][KQ8 ? 2 * b : b] ^ 0x80808080u;
                const uint32_t w1 = kw[gi][j][KQ8 ? 2 * b + 1 : b] ^ 0x80808080u;
                k00 = q8_pair<0x4240>(w0), k01 = q8_pair<0x4341>(w0);
                k10 = q8_pair<0x4240>(w1), k11 = q8_pair<0x4341>(w1);
              } else {
                const uint32_t w = kw[gi][j][b], w8 = w >> 8;
                k00 = q4_low(w), k01 = q4_low(w8), k10 = q4_high(w), k11 = q4_high(w8);
              }
              const float2 d = __half22float2(bits_h2(ks[gi][b][j]));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(c, qa[mt][0], k00, k01);
                mma_f16(c, qa[mt][1], k10, k11);
                z[mt][gi][j][0] = fmaf(d.x, c[0] + c[2], z[mt][gi][j][0]);
                z[mt][gi][j][1] = fmaf(d.y, c[1] + c[3], z[mt][gi][j][1]);
              }
            }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int gi = 0; gi < TG; ++gi)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[mt][gi][e >> 1][e & 1] *= factor[mt];

      // ---- scales of the values, and what the masks leave ----
      uint32_t vs[TG][NB][2];
#pragma unroll
      for (int gi = 0; gi < TG; ++gi)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint2 v = lds_u2(stage + gi * C::kGroupBytes + C::kKeyPart + kv_code_bytes(NB, VQ8) + (t * NB + b) * 8);
          vs[gi][b][0] = v.x, vs[gi][b][1] = v.y;
        }
      if (!full) {
#pragma unroll
        for (int gi = 0; gi < TG; ++gi) {
          const bool there = ok >> gi & 1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // e = tok / 4: column e & 1 of half e >> 1
            const int key = key0 + gi * kKvGroup + t + 4 * e;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              if (!there || key > last[mt] || key < low[mt]) z[mt][gi][e >> 1][e & 1] = -INFINITY;
            // what no row sees may be anything, NaN among it: its scale is 0
            if (!there || key >= run.len || key < low_all)
#pragma unroll
              for (int b = 0; b < NB; ++b) vs[gi][b][e >> 1] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
          }
        }
      }

      // ---- running maximum and sum ----
      float keep[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float m = -INFINITY;
#pragma unroll
        for (int gi = 0; gi < TG; ++gi)
          m = fmaxf(m, fmaxf(fmaxf(z[mt][gi][0][0], z[mt][gi][0][1]), fmaxf(z[mt][gi][1][0], z[mt][gi][1][1])));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = fmaxf(m, top[mt]);
        const float ref = m == -INFINITY ? 0.0f : m;
        keep[mt] = exp2_approx(top[mt] - ref);
        top[mt] = m;
        float add = 0.0f;
#pragma unroll
        for (int gi = 0; gi < TG; ++gi)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = exp2_approx(z[mt][gi][e >> 1][e & 1] - ref);
            z[mt][gi][e >> 1][e & 1] = w;
            add += w;
          }
        sum[mt] = fmaf(sum[mt], keep[mt], add);
      }

      // ---- outputs ----
      // A power of two brings the largest weight p d_v of the step below 2^15,
      // so that the split keeps its 22 bits however small the values are.
      uint32_t big = 0;
#pragma unroll
      for (int gi = 0; gi < TG; ++gi)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          big = __vmaxu2(big, __vmaxu2(vs[gi][b][0] & 0x7fff7fffu, vs[gi][b][1] & 0x7fff7fffu));
      big = __reduce_max_sync(0xffffffffu, max(big & 0xffffu, big >> 16));
      const int e_new = 29 - static_cast<int>(max(big >> 10, 1u));
      const float up = __uint_as_float(static_cast<uint32_t>(e_new + 127) << 23);
      const float turn = __uint_as_float(static_cast<uint32_t>(e_new - up_exp + 127) << 23);
      up_exp = e_new;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        keep[mt] *= turn;
#pragma unroll
        for (int gi = 0; gi < TG; ++gi)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[mt][gi][e >> 1][e & 1] *= up;
      }
#pragma unroll
      for (int first = 0; first < NB;) {
        const int n = kv_run(NB, VQ8, first).n, unit = VQ8 ? 4 : 2, bytes = n * unit;
        uint32_t vw[TG][4][2];
#pragma unroll
        for (int gi = 0; gi < TG; ++gi)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok4 = e * 4;
            const uint32_t part = stage + gi * C::kGroupBytes + C::kKeyPart + first * 64 * unit * 2;
            if (bytes == 8) {
              const uint2 v = lds_u2(part + ((g >> 2) * 64 + (t + tok4) * 4 + (g & 3)) * 8);
              vw[gi][e][0] = v.x, vw[gi][e][1] = v.y;
            } else if (bytes == 4) {
              vw[gi][e][0] = lds_u32(part + ((t + tok4) * 8 + g) * 4);
            } else {
              vw[gi][e][0] = lds_u16(part + ((t + tok4) * 8 + g) * 2);
            }
          }
#pragma unroll
        for (int r = 0; r < n; ++r) {
          const int b = first + r;
          // value codes of the block: columns of 4 tiles, tokens in pairs
          uint32_t vb[TG][4][2];
#pragma unroll
          for (int gi = 0; gi < TG; ++gi)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (VQ8) {
                const uint32_t w0 = vw[gi][2 * h][r] ^ 0x80808080u, w1 = vw[gi][2 * h + 1][r] ^ 0x80808080u;
                const uint32_t x = __byte_perm(w0, w1, 0x5140), y = __byte_perm(w0, w1, 0x7362);
                vb[gi][0][h] = q8_pair<0x4140>(x), vb[gi][2][h] = q8_pair<0x4342>(x);
                vb[gi][1][h] = q8_pair<0x4140>(y), vb[gi][3][h] = q8_pair<0x4342>(y);
              } else {
                const uint32_t x = __byte_perm(vw[gi][2 * h][r >> 1], vw[gi][2 * h + 1][r >> 1], r & 1 ? 0x7632 : 0x5410);
                const uint32_t x8 = x >> 8;
                vb[gi][0][h] = q4_low(x), vb[gi][1][h] = q4_high(x);
                vb[gi][2][h] = q4_low(x8), vb[gi][3][h] = q4_high(x8);
              }
            }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float c[4][4];
#pragma unroll
            for (int n4 = 0; n4 < 4; ++n4) c[n4][0] = c[n4][1] = c[n4][2] = c[n4][3] = 0.0f;
#pragma unroll
            for (int gi = 0; gi < TG; ++gi) {
              const float2 d0 = __half22float2(bits_h2(vs[gi][b][0])), d1 = __half22float2(bits_h2(vs[gi][b][1]));
              uint4 w;
              split_f16(z[mt][gi][0][0] * d0.x, z[mt][gi][0][1] * d0.y, w.x, w.y);
              split_f16(z[mt][gi][1][0] * d1.x, z[mt][gi][1][1] * d1.y, w.z, w.w);
#pragma unroll
              for (int n4 = 0; n4 < 4; ++n4) mma_f16(c[n4], w, vb[gi][n4][0], vb[gi][n4][1]);
            }
#pragma unroll
            for (int n4 = 0; n4 < 4; ++n4) {
              acc[mt][b * 4 + n4][0] = fmaf(acc[mt][b * 4 + n4][0], keep[mt], c[n4][0] + c[n4][2]);
              acc[mt][b * 4 + n4][1] = fmaf(acc[mt][b * 4 + n4][1], keep[mt], c[n4][1] + c[n4][3]);
            }
          }
        }
        first += n;
      }
      __syncwarp();  // every lane has read the stage
      if (grp + S * TG < run.hi) fill(run, grp + S * TG);
    }

    // ---- the next item's groups are on their way while this one is joined ----
    pos += run.b - run.a;
    const bool more = pos < end;
    if (more) {
      locate(next);
      if (!dead)
        for (int i = 0; i < S; ++i)
          if (next.lo + i * TG < next.hi) fill(next, next.lo + i * TG);
    }

    // ---- join the warps ----
    const float down = __uint_as_float(static_cast<uint32_t>(127 - up_exp) << 23);
    const bool whole = run.a == 0 && run.b == run.n;
    float *slot = slots + (2 * blockIdx.x + (run.a == 0 ? 1 : 0)) * kv_attn_slot_floats(C::kRows, D);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt) __syncthreads();  // the previous tile's join has been read
      sum[mt] += __shfl_xor_sync(0xffffffffu, sum[mt], 1);
      sum[mt] += __shfl_xor_sync(0xffffffffu, sum[mt], 2);
      if (t == 0) w_max[warp][g] = top[mt], w_sum[warp][g] = sum[mt];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float(*c)[2] = &acc[mt][b * 4];
        float *row = join + g * C::kRowPad + b * 32 + 4 * t;
        *reinterpret_cast<float4 *>(row) = make_float4(c[0][0] * down, c[2][0] * down, c[0][1] * down, c[2][1] * down);
        *reinterpret_cast<float4 *>(row + 16) = make_float4(c[1][0] * down, c[3][0] * down, c[1][1] * down, c[3][1] * down);
      }
      __syncthreads();
      for (int e = tid; e < 8 * (D / 4); e += NW * 32) {
        const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
        const int row = run.tile * C::kRows + mt * 8 + r;
        if (row >= p.rows) continue;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) m = fmaxf(m, w_max[w][r]);
        const float ref = m == -INFINITY ? 0.0f : m;
        float l = 0.0f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float k = exp2_approx(w_max[w][r] - ref);
          l = fmaf(k, w_sum[w][r], l);
          const float4 v = *reinterpret_cast<const float4 *>(joins + (w * 8 + r) * C::kRowPad + d);
          o.x = fmaf(k, v.x, o.x), o.y = fmaf(k, v.y, o.y), o.z = fmaf(k, v.z, o.z), o.w = fmaf(k, v.w, o.w);
        }
        if (whole) {
          const float inv = l > 0.0f ? 1.0f / l : 0.0f;
          kv_store(p, kv_out_at(p, run.seq, run.head, row, D) + d,
                   make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        } else {
          *reinterpret_cast<float4 *>(slot + (mt * 8 + r) * D + d) = o;
          if (d == 0) *reinterpret_cast<float2 *>(slot + C::kRows * D + (mt * 8 + r) * 2) = make_float2(m, l);
        }
      }
    }
    if (!more) {
      // What is left to join: an item that begins here and ends in a later block.
      if (tid == 0) {
        KvSplit sp{-1, 0, 0, 0};
        if (run.a == 0 && run.b < run.n) {
          const int64_t tail = end - (run.b - run.a) + run.n - 1;  // the item's last group on the line
          sp = KvSplit{run.seq, run.head, run.tile, static_cast<int>(((tail + 1) * blocks - 1) / total)};
        }
        splits[blockIdx.x] = sp;
      }
      break;
    }
    __syncthreads();  // the join and the fragments have been read
    run = next;
    load_q(run);
    __syncthreads();
  }
}

template <int NB, bool KQ8, bool VQ8, int MT>
__global__ void __launch_bounds__(KvCfg<NB, KQ8, VQ8, MT>::kNW * 32, 1)
    kv_attn_kernel(const __grid_constant__ KvLaunch p, uint32_t *status) {
  kv_attn_body<NB, KQ8, VQ8, MT>(p, status);
}

// Launch of one instance; the attribute is set once per device.
template <int NB, bool KQ8, bool VQ8, int MT>
cudaError_t kv_attn_launch(const DevInfo &dev, KvLaunch &p, uint32_t *status, cudaLaunchConfig_t cfg) {
  using C = KvCfg<NB, KQ8, VQ8, MT>;
  static DeviceFlags ready;
  if (!ready.done(dev.device)) {
    cudaError_t e = cudaFuncSetAttribute(kv_attn_kernel<NB, KQ8, VQ8, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmem);
    if (e != cudaSuccess) return e;
    ready.set(dev.device);
  }
  cfg.blockDim = dim3(C::kNW * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  p.tiles = (p.rows + C::kRows - 1) / C::kRows;
  return cudaLaunchKernelEx(&cfg, kv_attn_kernel<NB, KQ8, VQ8, MT>, p, status);
}

// Row tiles of a block: the fewest that hold the rows, 16 (block, tile) pairs at
// most (their sums stay in registers).
template <int NB>
constexpr int kv_attn_tiles(int rows) {
  const int most = NB * 4 <= 16 ? 4 : 2;
  return rows <= 8 ? 1 : rows <= 16 || most == 2 ? 2 : 4;
}

template <int NB, bool KQ8, bool VQ8>
cudaError_t kv_attn_rows(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg) {
  switch (kv_attn_tiles<NB>(p.rows)) {
    case 1: return kv_attn_launch<NB, KQ8, VQ8, 1>(dev, p, status, cfg);
    case 2: return kv_attn_launch<NB, KQ8, VQ8, 2>(dev, p, status, cfg);
    default:
      if constexpr (NB <= 4) return kv_attn_launch<NB, KQ8, VQ8, 4>(dev, p, status, cfg);
      return cudaErrorInvalidValue;
  }
}

template <int NB>
cudaError_t kv_attn_types(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg) {
  if (p.f.kq8) return p.f.vq8 ? kv_attn_rows<NB, true, true>(dev, p, status, cfg) : kv_attn_rows<NB, true, false>(dev, p, status, cfg);
  return p.f.vq8 ? kv_attn_rows<NB, false, true>(dev, p, status, cfg) : kv_attn_rows<NB, false, false>(dev, p, status, cfg);
}

// kv_attn_d*.cu
cudaError_t kv_attn_d64(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg);
cudaError_t kv_attn_d96(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg);
cudaError_t kv_attn_d128(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg);
cudaError_t kv_attn_d192(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg);
cudaError_t kv_attn_d256(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg);

}  // namespace qmm
