// kv_attn.cu -- decode attention over the quantised key/value cache: launch and
// the joining of partial results (include/qmm.h, qmm_kv_attn; the kernel:
// kv_attn.cuh).
#include "kv_attn.cuh"

namespace qmm {
namespace {

__device__ uint32_t g_attn_status;

// Joins the items that more than one block worked on: block (j, r) takes row r
// of the item that begins in block j of the main launch and ends in a later
// one. The partial results are added in block order: the same sums every time.
template <int D, int ROWS>
__global__ void __launch_bounds__(128) kv_attn_join_kernel(const __grid_constant__ KvLaunch p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kQuads = D / 4, kParts = 128 / kQuads;  // threads of a partial result; partial results at a time
  const KvSplit sp = reinterpret_cast<const KvSplit *>(p.a.ws)[blockIdx.x];
  const int r = blockIdx.y, row = sp.tile * ROWS + r;
  if (sp.seq < 0 || row >= p.rows) return;
  const float *slots = p.a.ws + kKvMaxBlocks * 4;
  const int64_t size = kv_attn_slot_floats(ROWS, D);
  const int n = sp.last - blockIdx.x + 1;  // partial results: slot 1 of block j, slot 0 of the others
  const auto slot = [&](int i) { return slots + (2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * size; };
  __shared__ float4 part_o[kParts][kQuads];
  __shared__ float part_m[kParts], part_l[kParts];
  const int part = threadIdx.x / kQuads, d = (threadIdx.x - part * kQuads) * 4;
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (part < kParts)
    for (int i = part; i < n; i += kParts) {
      const float *s = slot(i);
      const float2 ml = *reinterpret_cast<const float2 *>(s + ROWS * D + r * 2);
      const float4 v = *reinterpret_cast<const float4 *>(s + r * D + d);
      const float next = fmaxf(m, ml.x), ref = next == -INFINITY ? 0.0f : next;
      const float keep = exp2_approx(m - ref), k = exp2_approx(ml.x - ref);
      m = next;
      l = fmaf(l, keep, k * ml.y);
      o.x = fmaf(o.x, keep, k * v.x), o.y = fmaf(o.y, keep, k * v.y);
      o.z = fmaf(o.z, keep, k * v.z), o.w = fmaf(o.w, keep, k * v.w);
    }
  if (part < kParts) {
    part_o[part][d / 4] = o;
    if (d == 0) part_m[part] = m, part_l[part] = l;
  }
  __syncthreads();
  if (part) return;
  m = -INFINITY;
  for (int i = 0; i < kParts; ++i) m = fmaxf(m, part_m[i]);
  const float ref = m == -INFINITY ? 0.0f : m;
  l = 0.0f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < kParts; ++i) {
    const float k = exp2_approx(part_m[i] - ref);
    const float4 v = part_o[i][d / 4];
    l = fmaf(k, part_l[i], l);
    o.x = fmaf(k, v.x, o.x), o.y = fmaf(k, v.y, o.y), o.z = fmaf(k, v.z, o.z), o.w = fmaf(k, v.w, o.w);
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  kv_store(p, kv_out_at(p, sp.seq, sp.head, row, D) + d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

template <int D>
cudaError_t join_rows(int rows, const cudaLaunchConfig_t &cfg, const KvLaunch &p) {
  switch (rows) {
    case 8: return cudaLaunchKernelEx(&cfg, kv_attn_join_kernel<D, 8>, p);
    case 16: return cudaLaunchKernelEx(&cfg, kv_attn_join_kernel<D, 16>, p);
    default: return cudaLaunchKernelEx(&cfg, kv_attn_join_kernel<D, 32>, p);
  }
}

}  // namespace

qmm_status launch_kv_attn(const DevInfo &dev, const KvForm &f, int dtype, const KvAttnArgs &a, cudaStream_t stream) {
  KvLaunch p{};
  p.f = f;
  p.a = a;
  p.ratio = a.hq / f.heads;
  p.rows = a.m * p.ratio;
  p.min_groups = 16;
  p.bf16 = dtype == QMM_BF16;
  void *status = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&status, g_attn_status);
  if (e != cudaSuccess) return cuda_check(e, "kv_attn status");
  uint32_t *st = static_cast<uint32_t *>(status);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(std::min(dev.sms, kKvMaxBlocks));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (f.nb) {
    case 2: e = kv_attn_d64(dev, p, st, cfg); break;
    case 3: e = kv_attn_d96(dev, p, st, cfg); break;
    case 4: e = kv_attn_d128(dev, p, st, cfg); break;
    case 6: e = kv_attn_d192(dev, p, st, cfg); break;
    default: e = kv_attn_d256(dev, p, st, cfg); break;
  }
  if (e != cudaSuccess) return cuda_check(e, "kv_attn launch");
  const int rows = 8 * (f.nb <= 4 ? kv_attn_tiles<4>(p.rows) : kv_attn_tiles<8>(p.rows));
  p.tiles = (p.rows + rows - 1) / rows;
  cfg.gridDim.y = std::min(rows, p.rows);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  switch (f.nb) {
    case 2: e = join_rows<64>(rows, cfg, p); break;
    case 3: e = join_rows<96>(rows, cfg, p); break;
    case 4: e = join_rows<128>(rows, cfg, p); break;
    case 6: e = join_rows<192>(rows, cfg, p); break;
    default: e = join_rows<256>(rows, cfg, p); break;
  }
  return cuda_check(e, "kv_attn join launch");
}

int64_t kv_attn_workspace_floats(int64_t batch, int m, int hq, int hkv, int d) {
  (void)batch;
  const int rows = 8 * (d <= 128 ? kv_attn_tiles<4>(m * (hq / hkv)) : kv_attn_tiles<8>(m * (hq / hkv)));
  return kKvMaxBlocks * 4 + 2 * static_cast<int64_t>(kKvMaxBlocks) * kv_attn_slot_floats(rows, d);
}

cudaError_t kv_attn_status(uint32_t *bits) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_attn_status, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(uint32_t));
  return e;
}

}  // namespace qmm
