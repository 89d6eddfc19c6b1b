// kv_attn_d192.cu -- instances of the decode attention kernel for head size 192.
#include "kv_attn.cuh"

namespace qmm {

cudaError_t kv_attn_d192(const DevInfo &dev, KvLaunch &p, uint32_t *status, const cudaLaunchConfig_t &cfg) {
  return kv_attn_types<6>(dev, p, status, cfg);
}

}  // namespace qmm
