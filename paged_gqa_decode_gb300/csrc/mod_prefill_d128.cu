// tcgen05 prefill with modified scores (paged_score.cuh) at head_dim 128, and
// the prefill step's write for both head dims.
#include "paged_prefill_umma.cuh"
#include "pgd_ext_internal.h"

namespace pgd {

cudaError_t launch_mod_prefill_d128(const ModParams& p, const CUtensorMap& k_map,
                                    const CUtensorMap& v_map, const CUtensorMap& q_map,
                                    int sm_count, bool prepared, int parts, cudaStream_t stream) {
  return launch_prefill_umma<128, 4, 4, ModScore>(p, k_map, v_map, q_map, sm_count, prepared,
                                                  parts, stream);
}

cudaError_t launch_mod_prefill_write(const ModParams& p, int head_dim, bool umma,
                                     cudaStream_t stream) {
  return head_dim == 64 ? launch_prefill_write_for<64, ModScore>(p, umma, stream)
                        : launch_prefill_write_for<128, ModScore>(p, umma, stream);
}

}  // namespace pgd
