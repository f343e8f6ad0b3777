// Decode with modified scores at head_dim 64.
#include "mod_decode.cuh"

namespace pgd {

cudaError_t launch_mod_decode_d64(const ModParams& p, const CUtensorMap& k_map,
                                  const CUtensorMap& v_map, int grid_splits, int pages_per_cta,
                                  cudaStream_t stream) {
  return launch_mod_decode<64>(p, k_map, v_map, grid_splits, pages_per_cta, stream);
}

}  // namespace pgd
