// kv_attn_d256.cu -- instances of the decode attention kernel for head size 256.
#include "kv_attn.cuh"

namespace qmm {

cudaError_t kv_attn_d256(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg) {
  return kv_attn_types<8>(dev, p, status, cfg);
}

}  // namespace qmm
