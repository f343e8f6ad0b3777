// tcgen05 prefill with modified scores (paged_prefill_mod.cuh), head_dim 64: capped and biased scores.
#include "paged_prefill_mod.cuh"

namespace pgd {

template cudaError_t launch_prefill_mod<64, 3>(const ModParams&, const CUtensorMap&,
                                              const CUtensorMap&, const CUtensorMap&, int, bool,
                                              int, cudaStream_t);

}  // namespace pgd
