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

struct ForkParams {
  int32_t* table;  // [rows][width], rewritten in place
  const int32_t* lengths;
  const int32_t* parents;
  const int32_t* keep;  // or nullptr
  int32_t* shares;      // [num_pages]
  int32_t* free_pages;
  const int32_t* free_head;  // nullptr: 0
  int32_t* new_lengths;
  int32_t* sources;
  int32_t* targets;
  int32_t* counts;
  int32_t* free_head_out;
  unsigned int* err;
  int rows, width, num_pages, num_free;
  int slab_shift;  // (the launcher's, as the next)
  int undo;        // fork_adjust_kernel: take its changes to the shares back
};
constexpr int kMaxForkRows = 8192;  // five words a row and a column of them in shared memory
cudaError_t launch_fork_rows(const ForkParams& p, int sm_count, cudaStream_t stream);

constexpr int kMaxCopyPools = 128;  // of one launch
struct CopyParams {
  const int32_t* sources;
  const int32_t* targets;
  const int32_t* counts;  // or nullptr: whole pages
  unsigned int* err;
  int copies, pools, hkv, num_pages, layout;
  void* pool[kMaxCopyPools];
};
cudaError_t launch_copy_pages(const CopyParams& p, int head_dim, int sm_count,
                              cudaStream_t stream);

struct CompactParams {
  const int32_t* table;  // [rows][width]
  const int32_t* lengths;
  const int32_t* shares;
  const int32_t* free_pages;
  const int32_t* free_head;  // nullptr: 0
  int32_t* new_table;        // each may be its input
  int32_t* new_shares;
  int32_t* new_free;
  int32_t* sources;  // [max_moves]
  int32_t* targets;
  int32_t* end;
  uint32_t* bits;  // workspace: two bitmaps over the pool, a flag, the barriers' count of arrivals
  unsigned int* err;
  int rows, width, num_pages, num_free, max_moves;
  int step;  // (the launcher's)
};
constexpr int kMaxCompactPrefixes = 24 * 1024;  // of a bitmap, in shared memory
size_t compact_workspace_bytes(int num_pages);
cudaError_t launch_compact_pages(const CompactParams& p, int sm_count, cudaStream_t stream);

constexpr int kMaxSharedGroups = 8192;  // two words a group in shared memory
constexpr int kMaxSharedCtas = 160;
// What the combine needs of a row: where its own pages and its group's begin in the cut
// (-1: it has none), its group's rows and pages, and its position.
struct SharedRecord {
  long long own, group;
  int start, end, shared, n;
};

struct SharedCut;  // what falls to which CTA (shared_decode.cuh)
constexpr int kSharedCutBytes = 48;

struct SharedParams {
  const uint16_t* q;
  const int32_t* table;
  const int32_t* positions;
  const int32_t* starts;  // [groups + 1]
  const int32_t* pages;   // [groups]
  const float* sinks;     // or nullptr
  uint16_t* out;
  float* part_acc;     // D values of each partial
  float* part_ml;      // (m, l) of each
  SharedRecord* records;  // [rows], for the combine, with
  SharedCut* cut;
  unsigned int* err;
  int rows, groups, hq, hkv, group, maxp, num_pages, layout;
  int tile;                // rows of a tile, 128 / group
  uint32_t block_inverse;  // 2^32 / (2 tile), rounded up
  float q_scale_log2;
  const uint16_t* k_new;  // or nullptr
  const uint16_t* v_new;
  uint16_t* k_pool;
  uint16_t* v_pool;
};
cudaError_t launch_shared_d64(const SharedParams& p, const CUtensorMap& k_map,
                              const CUtensorMap& v_map, const CUtensorMap& q_map, int ctas,
                              cudaStream_t stream);
cudaError_t launch_shared_d128(const SharedParams& p, const CUtensorMap& k_map,
                              const CUtensorMap& v_map, const CUtensorMap& q_map, int ctas,
                              cudaStream_t stream);

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
