// kv_attn_d128.cu -- instances of the decode attention kernel for head size 128.
#include "kv_attn.cuh"

namespace qmm {

cudaError_t kv_attn_d128(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg) {
  return kv_attn_types<4>(dev, p, status, cfg);
}

}  // namespace qmm
