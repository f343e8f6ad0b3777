// Launch parameters and launcher declarations of libpgd_ext's kernels, shared
// by its host API (pgd_ext_api.cu) and the kernel translation units.
#pragma once

#include "paged_score.cuh"
#include "pgd_ext.h"
#include "pgd_internal.h"

namespace pgd {

struct AssignParams {
  int32_t* table;  // [requests][maxp], read (pages in use) and written (new pages)
  const int32_t* cached;
  const int32_t* new_tokens;
  const int32_t* free_pages;
  const int32_t* free_head;  // nullptr: 0
  int32_t* rows;
  int32_t* positions;
  int32_t* slots;
  int32_t* starts;
  int32_t* lengths;
  int32_t* free_head_out;
  unsigned int* err;
  int requests, maxp, num_pages, tokens, num_free;
};
cudaError_t launch_assign_pages(const AssignParams& p, int sm_count, cudaStream_t stream);

struct RotaryParams {
  const uint16_t* q;  // rows of [Hq][D] at q_stride, or nullptr
  uint16_t* q_out;    // rows of [Hq][D] at q_out_stride (q itself: in place)
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t q_stride, q_out_stride, k_stride, v_stride;  // values from token to token
  const int32_t* table;
  const int32_t* row_of;
  const int32_t* positions;
  const int32_t* slots;
  uint16_t* k_pool;
  uint16_t* v_pool;
  unsigned int* err;
  int rows, table_rows, hq, hkv, maxp, num_pages, layout;
  pgdx_rotary rotary;
};
cudaError_t launch_rotary_append(const RotaryParams& p, int head_dim, cudaStream_t stream);

// Attention with the scores of ModParams: the split decode (and its combine),
// the tcgen05 prefill (and its block order or key-part combine), and the
// prefill step's write, as their namesakes in pgd_internal.h.
cudaError_t launch_mod_decode_d64(const ModParams& p, const CUtensorMap& k_map,
                                  const CUtensorMap& v_map, int grid_splits, int pages_per_cta,
                                  cudaStream_t stream);
cudaError_t launch_mod_decode_d128(const ModParams& p, const CUtensorMap& k_map,
                                   const CUtensorMap& v_map, int grid_splits, int pages_per_cta,
                                   cudaStream_t stream);
cudaError_t launch_mod_prefill(const ModParams& p, const CUtensorMap& k_map,
                               const CUtensorMap& v_map, const CUtensorMap& q_map, int head_dim,
                               int sm_count, bool prepared, int parts, cudaStream_t stream);
cudaError_t launch_mod_prefill_write(const ModParams& p, int head_dim, bool umma,
                                     cudaStream_t stream);

}  // namespace pgd
