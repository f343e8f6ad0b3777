// tcgen05 prefill with modified scores (paged_score.cuh) at head_dim 64.
#include "paged_prefill_umma.cuh"
#include "pgd_ext_internal.h"

namespace pgd {

cudaError_t launch_mod_prefill_d64(const ModParams& p, const CUtensorMap& k_map,
                                   const CUtensorMap& v_map, const CUtensorMap& q_map,
                                   int sm_count, bool prepared, int parts, cudaStream_t stream) {
  return launch_prefill_umma<64, 8, 8, ModScore>(p, k_map, v_map, q_map, sm_count, prepared, parts,
                                                 stream);
}

}  // namespace pgd
