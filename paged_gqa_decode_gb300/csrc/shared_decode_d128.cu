// Decode over shared pages at head_dim 128 (shared_decode.cuh).
#include "shared_decode.cuh"

namespace pgd {

cudaError_t launch_shared_d128(const SharedParams& p, const CUtensorMap& k_map,
                             const CUtensorMap& v_map, const CUtensorMap& q_map,
                             int ctas, cudaStream_t stream) {
  return launch_shared<128, 5>(p, k_map, v_map, q_map, ctas, stream);
}

}  // namespace pgd
