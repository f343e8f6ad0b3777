// tcgen05 prefill with modified scores (paged_prefill_mod.cuh), head_dim 128: masks only.
#include "paged_prefill_mod.cuh"

namespace pgd {

template cudaError_t launch_prefill_mod<128, 0>(const ModParams&, const CUtensorMap&,
                                              const CUtensorMap&, const CUtensorMap&, int, bool,
                                              int, cudaStream_t);

}  // namespace pgd
