// Prefill with modified scores: the choice of kernel by head_dim and kind (each
// compiled in a unit of its own), and the prefill step's write.
#include "paged_prefill_umma.cuh"
#include "pgd_ext_internal.h"

namespace pgd {

template <int D, int KIND>  // KIND: 1 capped, 2 biased (paged_prefill_mod.cuh)
cudaError_t launch_prefill_mod(const ModParams& p, const CUtensorMap& k_map,
                               const CUtensorMap& v_map, const CUtensorMap& q_map, int sm_count,
                               bool prepared, int parts, cudaStream_t stream);

template <int D>
static cudaError_t launch_kind(const ModParams& p, const CUtensorMap& k_map,
                               const CUtensorMap& v_map, const CUtensorMap& q_map, int sm_count,
                               bool prepared, int parts, cudaStream_t stream) {
  const int kind = (p.cap_in != 0.f ? 1 : 0) | (p.slopes ? 2 : 0);
  switch (kind) {
    case 0:
      return launch_prefill_mod<D, 0>(p, k_map, v_map, q_map, sm_count, prepared, parts, stream);
    case 1:
      return launch_prefill_mod<D, 1>(p, k_map, v_map, q_map, sm_count, prepared, parts, stream);
    case 2:
      return launch_prefill_mod<D, 2>(p, k_map, v_map, q_map, sm_count, prepared, parts, stream);
    default:
      return launch_prefill_mod<D, 3>(p, k_map, v_map, q_map, sm_count, prepared, parts, stream);
  }
}

cudaError_t launch_mod_prefill(const ModParams& p, const CUtensorMap& k_map,
                               const CUtensorMap& v_map, const CUtensorMap& q_map, int head_dim,
                               int sm_count, bool prepared, int parts, cudaStream_t stream) {
  return head_dim == 64
             ? launch_kind<64>(p, k_map, v_map, q_map, sm_count, prepared, parts, stream)
             : launch_kind<128>(p, k_map, v_map, q_map, sm_count, prepared, parts, stream);
}

cudaError_t launch_mod_prefill_write(const ModParams& p, int head_dim, bool umma,
                                     cudaStream_t stream) {
  return head_dim == 64 ? launch_prefill_write_for<64, ModScore>(p, umma, stream)
                        : launch_prefill_write_for<128, ModScore>(p, umma, stream);
}

}  // namespace pgd
