// kv_attn.cu -- decode attention over the quantised key/value cache: launch
// (include/qmm.h, qmm_kv_attn; the kernel: kv_attn.cuh).
#include "kv_attn.cuh"

#include <atomic>
#include <chrono>

namespace qmm {
namespace {

__device__ uint32_t g_attn_status;

}  // namespace

qmm_status launch_kv_attn(const DevInfo &dev, const KvForm &f, int dtype, const KvAttnArgs &a, cudaStream_t stream) {
  KvLaunch p{};
  p.f = f;
  p.a = a;
  p.ratio = a.hq / f.heads;
  p.rows = a.m * p.ratio;
  p.min_units = 4;
  p.bf16 = dtype == QMM_BF16;
  // A number that no other call has; the start keeps it from what scratch memory may hold.
  static std::atomic<uint64_t> calls{static_cast<uint64_t>(std::chrono::steady_clock::now().time_since_epoch().count()) *
                                     0x9e3779b97f4a7c15ull};
  p.epoch = calls.fetch_add(1, std::memory_order_relaxed) | 1ull << 63;
  p.magic = KvMagic{0x64006400u, 0x2c002c00u, 0xd480d480u};
  // The status word's address on this device, looked up once.
  static std::atomic<uint32_t *> words[64];
  uint32_t *st = words[dev.device & 63].load(std::memory_order_acquire);
  cudaError_t e;
  if (st == nullptr) {
    void *word = nullptr;
    e = cudaGetSymbolAddress(&word, g_attn_status);
    if (e != cudaSuccess) return cuda_check(e, "kv_attn status");
    st = static_cast<uint32_t *>(word);
    words[dev.device & 63].store(st, std::memory_order_release);
  }
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
  return cuda_check(e, "kv_attn launch");
}

int64_t kv_attn_workspace_floats(int64_t batch, int m, int hq, int hkv, int d) {
  (void)batch;
  const int rows = m * (hq / hkv), nb = d / 32;
  return kv_attn_scratch_floats(8 * std::max(kv_attn_octets(nb, rows, false), kv_attn_octets(nb, rows, true)), d);
}

cudaError_t kv_attn_status(uint32_t *bits) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_attn_status, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(uint32_t));
  return e;
}

}  // namespace qmm
