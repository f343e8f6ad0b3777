// Host-side helpers of the C ABIs (pgd_api.cu and pgd_ext_api.cu): the device's
// properties and error word, argument checks, launch planning (pages per
// split, key parts) and TMA descriptor encoding.  Included by one translation
// unit of each library; everything here is that unit's own.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "pgd.h"
#include "pgd_internal.h"

namespace pgd {

namespace {

// The sticky device error word of each device that loads the library.
__device__ unsigned int g_device_error = 0;

constexpr int kMaxDevices = 64;
constexpr int kPageSize = 64;
constexpr int kMinPagesPerSplit = 24;
constexpr int kMaxPagesPerSplit = 64;

struct DeviceInfo {
  std::once_flag once;
  cudaError_t status = cudaSuccess;
  int sm_count = 0;
  unsigned int* err = nullptr;  // device address of g_device_error
};
DeviceInfo g_devices[kMaxDevices];

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

int current_device(DeviceInfo** info) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PGD_ECUDA;
  DeviceInfo& d = g_devices[dev];
  std::call_once(d.once, [&] {
    d.status = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (d.status == cudaSuccess)
      d.status = cudaGetSymbolAddress(reinterpret_cast<void**>(&d.err), g_device_error);
  });
  if (d.status != cudaSuccess) return PGD_ECUDA;
  *info = &d;
  return PGD_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_dims(const pgd_dims* d) {
  if (!d) return PGD_EINVAL;
  if (d->rows < 0 || d->num_q_heads <= 0 || d->num_kv_heads <= 0 || d->head_dim <= 0 ||
      d->num_pages <= 0 || d->max_pages_per_row <= 0)
    return PGD_EINVAL;
  if (d->num_q_heads % d->num_kv_heads != 0) return PGD_EINVAL;
  if (d->layout != PGD_PAGE_MAJOR && d->layout != PGD_HEAD_MAJOR && d->layout != PGD_ROW_MAJOR)
    return PGD_EINVAL;
  if (d->layout == PGD_ROW_MAJOR && d->num_pages % d->max_pages_per_row != 0) return PGD_EINVAL;
  if (d->page_size != kPageSize) return PGD_EUNSUPPORTED;
  if (d->head_dim != 64 && d->head_dim != 128) return PGD_EUNSUPPORTED;
  if (padded_group(d->num_q_heads / d->num_kv_heads) == 0) return PGD_EUNSUPPORTED;
  // Pool rows are addressed with 32-bit TMA coordinates; positions are int32.
  if ((int64_t)d->num_pages * d->num_kv_heads * kPageSize >= (int64_t)INT32_MAX)
    return PGD_EUNSUPPORTED;
  if ((int64_t)d->max_pages_per_row * kPageSize > (int64_t)INT32_MAX) return PGD_EUNSUPPORTED;
  return PGD_OK;
}

struct Plan {
  int pages_per_split;
  int max_splits;
};

// Key parts of the one-SM tcgen05 prefill (AUTO only) for a call of these
// dims: with at most half as many work items (blocks of 2 x 128 / group
// tokens, times the kv heads) as SMs, each item's pages are cut into parts,
// each a work unit of its own, so that the units fill the SMs.  At most 8,
// and at least 8 pages a part on the longest item the table allows (a
// window bounds it): parts of a few pages cost more in partials and the
// combine than they gain.  1: no parts.
constexpr int kMaxKeyParts = 8;
constexpr int kMinPartPages = 8;
int prefill_key_parts(const pgd_dims* d, int sm_count, int32_t window) {
  const int64_t block = 2 * (128 / (d->num_q_heads / d->num_kv_heads));
  const int64_t items = (d->rows + block - 1) / block * d->num_kv_heads;
  if (sm_count <= 0 || items <= 0 || items * 2 > sm_count) return 1;
  int64_t pages = d->max_pages_per_row;
  if (window > 0) {
    const int64_t span = ((int64_t)window + block - 2) / kPageSize + 2;  // window + block - 1 keys
    if (span < pages) pages = span;
  }
  int64_t parts = sm_count / items;
  if (parts > kMaxKeyParts) parts = kMaxKeyParts;
  if (parts > pages / kMinPartPages) parts = pages / kMinPartPages;
  return parts >= 2 ? (int)parts : 1;
}

// Pages per split: enough CTAs for several waves of 2 CTAs per SM when rows
// are about half full, but at least 24 pages (sweeps over 1..64 on GB300
// found every workload fastest at 24 or more: a split's fixed costs --
// setup, merge, partials and the combine -- outweigh the parallelism that
// shorter splits add) and at most 64.
Plan make_plan(const pgd_dims* d, const pgd_decode_options* opts, int sm_count) {
  Plan pl;
  int pps = opts ? opts->pages_per_split : 0;
  if (pps <= 0) {
    const int64_t target = 4ll * 2 * (sm_count > 0 ? sm_count : 1);
    const int64_t expected = (int64_t)d->rows * d->num_kv_heads *
                             (d->max_pages_per_row > 1 ? d->max_pages_per_row / 2 : 1);
    int64_t v = (expected + target - 1) / target;
    pps = (int)(v < kMinPagesPerSplit ? kMinPagesPerSplit
                                      : (v > kMaxPagesPerSplit ? kMaxPagesPerSplit : v));
  }
  if (pps > d->max_pages_per_row) pps = d->max_pages_per_row;
  pl.pages_per_split = pps;
  pl.max_splits = (d->max_pages_per_row + pps - 1) / pps;
  // the same workspace serves a prefill call of these dims: its key parts'
  // partials take one split's room each, beside the work counter
  const int parts = prefill_key_parts(d, sm_count, 0);  // the most any window allows
  if (parts > 1 && parts + 1 > pl.max_splits) pl.max_splits = parts + 1;
  return pl;
}

size_t workspace_bytes(const pgd_dims* d, const Plan& pl) {
  return (size_t)d->rows * d->num_q_heads * pl.max_splits * (d->head_dim + 2) * sizeof(float);
}

// Whether the per-token split kernel's grid, (splits, kv heads, rows), holds the
// call: the last two stop at 65535.
constexpr int kMaxGridYZ = 65535;
bool per_token_fits(const pgd_dims* d) {
  return d->rows <= kMaxGridYZ && d->num_kv_heads <= kMaxGridYZ;
}

// The kernel a call runs: opts->kernel, or for AUTO the per-token split
// kernel, except that prefill with tokens in runs goes to a tcgen05 kernel:
// the one-SM kernel, with key parts (`key_parts` > 1) when its work items
// are at most half the SMs (`sm_count`; 0 = unknown) and long enough to
// cut, else for such calls at head_dim 128 the paired one, which puts two
// SMs on each item.  `window` bounds the items' length.
int resolve_kernel(const pgd_dims* dims, int32_t table_rows, bool prefill,
                   const pgd_decode_options* opts, int* kernel, int sm_count = 0,
                   int* key_parts = nullptr, int32_t window = 0) {
  int k = opts ? opts->kernel : PGD_KERNEL_AUTO;
  if (k < PGD_KERNEL_AUTO || k > PGD_KERNEL_PREFILL_PAIR) return PGD_EINVAL;
  if ((k == PGD_KERNEL_PREFILL_TILED || k == PGD_KERNEL_PREFILL_UMMA ||
       k == PGD_KERNEL_PREFILL_PAIR) &&
      !prefill)
    return PGD_EINVAL;
  if (k == PGD_KERNEL_PREFILL_PAIR && dims->head_dim != 128) return PGD_EINVAL;
  // Prefill: the tcgen05 kernel shares each page load among the tokens of a
  // block, which pays when they come in runs (prompt chunks); tokens that are
  // mostly one per table row (decode steps) go to the per-token split kernel.
  // Calls with at most half as many work items as SMs: key parts on one SM
  // per unit when the items are long enough to cut, else at head_dim 128 a
  // pair of SMs per item (measured on GB300: key parts 41-99 us against
  // 43-109 us for pairs on one Mistral-shaped chunk of 256-512 tokens; with
  // 128 items, pairs 102 us against 96-98 us for one SM per item).
  // More tokens than the split kernel's grid holds go to blocks whatever they are.
  int parts = 1;
  const bool window_kernel = window > 0 && window <= kMaxWindowKernel;
  if (prefill && k == PGD_KERNEL_AUTO &&
      (dims->rows >= 8ll * table_rows || (!per_token_fits(dims) && !window_kernel))) {
    k = PGD_KERNEL_PREFILL_UMMA;
    const int group = dims->num_q_heads / dims->num_kv_heads;
    const int64_t block = 2 * (128 / group);  // tokens per work item
    const int64_t items = (dims->rows + block - 1) / block * dims->num_kv_heads;
    parts = prefill_key_parts(dims, sm_count, window);
    if (parts == 1 && dims->head_dim == 128 && sm_count > 0 && items * 2 <= sm_count)
      k = PGD_KERNEL_PREFILL_PAIR;
  }
  *kernel = k;
  if (key_parts) *key_parts = parts;
  return PGD_OK;
}

// AUTO decode with full attention over a table of a few pages runs the
// window kernel, the whole table its window (every row's rows copied at
// once, one warp per 32 positions, no splits), when the split size is the
// library's choice and the batch has between half as many and as many
// (row, kv head) units as SMs: one round of units, each on an SM of its own.
// Outside that range the split kernel measured faster (GB300, per step
// between L2 flushes: Qwen2.5 shapes, 64 rows (128 units) 12.4 against 13.0
// us with the window kernel, 4 rows (8 units) 10.8 against 10.3 us; 64
// dense gpt-oss rows of 640 positions (512 units) 35.3 against 24.3 us).
bool short_row_kernel(const pgd_dims* d, int32_t window, const pgd_decode_options* opts,
                      int kernel, int sm_count) {
  const int64_t units = (int64_t)d->rows * d->num_kv_heads;
  return kernel == PGD_KERNEL_AUTO && window <= 0 && !(opts && opts->pages_per_split > 0) &&
         sm_count > 0 && units * 2 >= sm_count && units <= sm_count &&
         short_row_tiles(d->head_dim, d->max_pages_per_row) > 0;
}

// Pages the split grid must cover per row: the table width, or with a
// window at most ceil((window - 1) / 64) + 1 pages.
int span_pages(const pgd_dims* dims, int32_t window) {
  int grid_pages = dims->max_pages_per_row;
  if (window > 0) {
    const int64_t wp = ((int64_t)window + kPageSize - 2) / kPageSize + 1;
    if (wp < grid_pages) grid_pages = (int)wp;
  }
  return grid_pages;
}

int encode_pool_map_uncached(CUtensorMap* map, const void* pool, const pgd_dims* d, int kind);

// Encoded pool descriptors are reused while the same pool is passed again: a
// small per-process cache keyed by (device, address, pages, kv heads, dim).
struct MapEntry {
  int dev;
  const void* pool;
  int32_t num_pages, kv_heads, head_dim;
  int kind;
  CUtensorMap map;
};
constexpr int kMapCache = 16;
MapEntry g_maps[kMapCache];
int g_map_count = 0, g_map_next = 0;
std::mutex g_map_mutex;

// Box shapes of a pool's tensor map.
enum MapKind {
  kMapBoxes = 0,      // 64 rows x 64 values: a page tile, or a 64-wide half of one
  kMapWholeTile = 1,  // head_dim 128: a page tile's two 64-wide boxes in one copy
};

int encode_pool_map(CUtensorMap* map, const void* pool, const pgd_dims* d,
                    int kind = kMapBoxes) {
  if (d->head_dim != 128) kind = kMapBoxes;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PGD_ECUDA;
  {
    std::lock_guard<std::mutex> lock(g_map_mutex);
    for (int i = 0; i < g_map_count; ++i) {
      const MapEntry& m = g_maps[i];
      if (m.dev == dev && m.pool == pool && m.num_pages == d->num_pages &&
          m.kv_heads == d->num_kv_heads && m.head_dim == d->head_dim && m.kind == kind) {
        *map = m.map;
        return PGD_OK;
      }
    }
  }
  const int rc = encode_pool_map_uncached(map, pool, d, kind);
  if (rc != PGD_OK) return rc;
  std::lock_guard<std::mutex> lock(g_map_mutex);
  MapEntry& slot = g_maps[g_map_next];
  slot = MapEntry{dev, pool, d->num_pages, d->num_kv_heads, d->head_dim, kind, *map};
  g_map_next = (g_map_next + 1) % kMapCache;
  if (g_map_count < kMapCache) ++g_map_count;
  return PGD_OK;
}

bool load_encode() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode != nullptr;
}

// q of a packed prefill, [tokens][Hq][D] bf16, as (64 values, heads,
// tokens) with boxes of 64 x group x (128 / group): one box is one half of a
// query tile's rows (token-major, head-minor), 128-byte swizzled -- the
// layout the tcgen05 prefill's S products read.  Tokens past the end read
// as zeros.
int encode_q_map(CUtensorMap* map, const void* q, const pgd_dims* d) {
  if (!load_encode()) return PGD_ECUDA;
  const int group = d->num_q_heads / d->num_kv_heads;
  const cuuint64_t dims3[3] = {(cuuint64_t)d->head_dim, (cuuint64_t)d->num_q_heads,
                               (cuuint64_t)d->rows};
  const cuuint64_t strides3[2] = {(cuuint64_t)d->head_dim * 2,
                                  (cuuint64_t)d->num_q_heads * d->head_dim * 2};
  const cuuint32_t box3[3] = {64, (cuuint32_t)group, (cuuint32_t)(128 / group)};
  const cuuint32_t elem3[3] = {1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims3,
                        strides3, box3, elem3, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PGD_OK : PGD_ECUDA;
}

int encode_pool_map_uncached(CUtensorMap* map, const void* pool, const pgd_dims* d, int kind) {
  if (!load_encode()) return PGD_ECUDA;
  // The pool as a 2-D tensor: rows of head_dim bf16 values, one row per
  // (page, kv head, position) in either layout.  A box is 64 rows x 64
  // values (128 bytes): one page tile, or half of one when head_dim is 128.
  const cuuint64_t rows = (cuuint64_t)d->num_pages * d->num_kv_heads * kPageSize;
  if (kind != kMapBoxes) {
    // head_dim 128 as (64 values, rows, 2 halves): strides 256 bytes (a row)
    // and 128 bytes (a half), box 64 x 64 x 2 -- one copy lands a page tile as
    // the two consecutive 128-byte-swizzled 64-wide boxes the 2-D map gives.
    const cuuint64_t dims3[3] = {64, rows, 2};
    const cuuint64_t strides3[2] = {256, 128};
    const cuuint32_t box3[3] = {64, (cuuint32_t)kPageSize, 2};
    const cuuint32_t elem3[3] = {1, 1, 1};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(pool),
                          dims3, strides3, box3, elem3, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PGD_OK : PGD_ECUDA;
  }
  const cuuint64_t dims[2] = {(cuuint64_t)d->head_dim, rows};
  const cuuint64_t strides[1] = {(cuuint64_t)d->head_dim * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)kPageSize};
  const cuuint32_t elem[2] = {1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims,
                        strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PGD_OK : PGD_ECUDA;
}

// The attention calls' common part, after check_dims and the check for no
// rows: the arguments' checks, the split plan against the workspace, and the
// launch parameters.
int prepare_attention(const pgd_dims* dims, int32_t table_rows, const int32_t* row_of,
                      const void* q, const void* k_pool, const void* v_pool, const int32_t* table,
                      const int32_t* positions, const float* sinks, int32_t window, float scale,
                      void* out, void* workspace, size_t workspace_size,
                      const pgd_decode_options* opts, const void* k_new, const void* v_new,
                      DeviceInfo** device, Plan* plan, DecodeParams* params) {
  if (!q || !k_pool || !v_pool || !positions || !out) return PGD_EINVAL;
  if (!table && dims->layout != PGD_ROW_MAJOR) return PGD_EINVAL;
  if (row_of != nullptr && table_rows <= 0) return PGD_EINVAL;
  if (!table && (int64_t)(row_of ? table_rows : dims->rows) * dims->max_pages_per_row >
                    dims->num_pages)
    return PGD_EINVAL;  // dense rows: every row needs its own P pages
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return PGD_EINVAL;
  if ((k_new == nullptr) != (v_new == nullptr) ||
      (k_new && (!aligned16(k_new) || !aligned16(v_new))))
    return PGD_EINVAL;
  if (!std::isfinite(scale)) return PGD_EINVAL;
  const int rc = current_device(device);
  if (rc != PGD_OK) return rc;
  const Plan pl = make_plan(dims, opts, (*device)->sm_count);
  const size_t need = workspace_bytes(dims, pl);
  if (workspace_size < need) return PGD_EWORKSPACE;
  if (!workspace || !aligned16(workspace)) return PGD_EINVAL;
  *plan = pl;

  DecodeParams& p = *params;
  p.q = static_cast<const uint16_t*>(q);
  p.table = table;
  p.positions = positions;
  p.row_of = row_of;
  p.table_rows = table_rows;
  p.sinks = sinks;
  p.out = static_cast<uint16_t*>(out);
  const size_t acc_floats =
      (size_t)dims->rows * dims->num_q_heads * pl.max_splits * dims->head_dim;
  p.ws_acc = static_cast<float*>(workspace);
  p.ws_ml = p.ws_acc + acc_floats;
  p.err = (*device)->err;
  p.rows = dims->rows;
  p.hq = dims->num_q_heads;
  p.hkv = dims->num_kv_heads;
  p.group = dims->num_q_heads / dims->num_kv_heads;
  p.maxp = dims->max_pages_per_row;
  p.num_pages = dims->num_pages;
  p.layout = dims->layout;
  p.window = window > 0 ? window : 0;
  p.pages_per_split = pl.pages_per_split;
  p.max_splits = pl.max_splits;
  p.q_scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  p.k_pool = k_new ? static_cast<uint16_t*>(const_cast<void*>(k_pool)) : nullptr;
  p.v_pool = k_new ? static_cast<uint16_t*>(const_cast<void*>(v_pool)) : nullptr;
  p.k_read = static_cast<const uint16_t*>(k_pool);
  p.v_read = static_cast<const uint16_t*>(v_pool);
  return PGD_OK;
}

}  // namespace

}  // namespace pgd
