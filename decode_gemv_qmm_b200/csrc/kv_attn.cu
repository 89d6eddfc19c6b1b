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
__global__ void __launch_bounds__(256) kv_attn_join_kernel(const __grid_constant__ KvLaunch p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kQuads = D / 4, kParts = 256 / kQuads;  // threads of a partial result; partial results at a time
  const KvSplit sp = reinterpret_cast<const KvSplit *>(p.a.ws)[blockIdx.x];
  const int r = blockIdx.y, row = sp.tile * ROWS + r;
  if (sp.seq < 0 || row >= p.rows) return;
  const float *slots = p.a.ws + kKvMaxBlocks * 4;
  constexpr int64_t kSlot = kv_attn_slot_floats(ROWS, D);
  const int n = sp.last - blockIdx.x + 1;  // partial results: slot 1 of block j, slot 0 of the others
  __shared__ float4 part_o[kParts][kQuads];
  __shared__ float part_m[kParts], part_l[kParts];
  const int part = threadIdx.x / kQuads, d = (threadIdx.x - part * kQuads) * 4;
  if (part < kParts) {
    KvSum x;
    for (int i = part; i < n; i += kParts) {
      const float *s = slots + (2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * kSlot;
      const float2 ml = *reinterpret_cast<const float2 *>(s + ROWS * D + r * 2);
      x.add(ml.x, ml.y, *reinterpret_cast<const float4 *>(s + r * D + d));
    }
    part_o[part][d / 4] = x.o;
    if (d == 0) part_m[part] = x.m, part_l[part] = x.l;
  }
  __syncthreads();
  if (part) return;
  KvSum x;
  for (int i = 0; i < kParts; ++i) x.add(part_m[i], part_l[i], part_o[i][d / 4]);
  kv_store(p, kv_out_at(p, sp.seq, sp.head, row, D) + d, x.result());
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
  p.min_units = kKvItemCost + 2;
  p.bf16 = dtype == QMM_BF16;
  p.magic = KvMagic{0x64006400u, 0x2c002c00u, 0xd480d480u};
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
  const int rows = 8 * kv_attn_octets(f.nb, p.rows, !p.bf16);
  p.tiles = (p.rows + rows - 1) / rows;
  cfg.gridDim.y = std::min(rows, p.rows);
  cfg.blockDim = dim3(256);
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
  return kv_attn_scratch_floats(8 * kv_attn_octets(d / 32, m * (hq / hkv), false), d);
}

cudaError_t kv_attn_status(uint32_t *bits) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_attn_status, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(uint32_t));
  return e;
}

}  // namespace qmm
