// Decode kernels for modified scores (paged_score.cuh) at one head_dim: the
// split kernel of paged_decode.cuh with the tensor-core consumer, its ring no
// deeper than the pages a split can stream.  As that bound by the copies of K and
// V: 64 rows of 512 to 4096 positions, 64 / 8 heads of 64, capped, 55.5-57 us (303 MB,
// 5.4 TB/s; 53.7 us uncapped), 64 rows of 1024 to 16384, 32 / 8 heads of 128, with a
// bias and documents, 189-193 us (1.25 GB, 6.5 TB/s).
#pragma once

#include "paged_decode.cuh"
#include "pgd_ext_internal.h"

namespace pgd {

template <int D>
cudaError_t launch_mod_decode(const ModParams& p, const CUtensorMap& k_map,
                              const CUtensorMap& v_map, int grid_splits, int pages_per_cta,
                              cudaStream_t stream) {
  using Consumer = MmaConsumer<D, ModScore>;
  if (pages_per_cta <= 1)
    return launch_decode<D, 1, Consumer, kShortWarps>(p, k_map, v_map, grid_splits, stream);
  if (pages_per_cta <= 2)
    return launch_decode<D, 2, Consumer, kShortWarps>(p, k_map, v_map, grid_splits, stream);
  if (D == 64 && pages_per_cta <= 3)
    return launch_decode<D, kShortStages3, Consumer, kShortWarps>(p, k_map, v_map, grid_splits,
                                                                  stream);
  return launch_decode<D, D == 128 ? 3 : 6, Consumer>(p, k_map, v_map, grid_splits, stream);
}

}  // namespace pgd
