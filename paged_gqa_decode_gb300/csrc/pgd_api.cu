// Host side of the C ABI declared in include/pgd.h: argument validation and
// launches (planning and TMA descriptors in pgd_host.h).
#include <cmath>

#include "pgd_host.h"

using namespace pgd;

extern "C" {

static int append_impl(const pgd_dims* dims, const void* k_new, const void* v_new,
                       const int32_t* table, const int32_t* positions, const int32_t* slots,
                       void* k_pool, void* v_pool, pgd_stream_t stream) {
  int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (dims->rows == 0) return PGD_OK;
  if (!k_new || !v_new || !k_pool || !v_pool) return PGD_EINVAL;
  if (slots == nullptr && (!positions || (!table && dims->layout != PGD_ROW_MAJOR)))
    return PGD_EINVAL;
  if (slots == nullptr && !table &&
      (int64_t)dims->rows * dims->max_pages_per_row > dims->num_pages)
    return PGD_EINVAL;  // dense rows: every row needs its own P pages
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool))
    return PGD_EINVAL;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev)) != PGD_OK) return rc;
  AppendParams p;
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  p.table = table;
  p.positions = positions;
  p.slots = slots;
  p.k_pool = static_cast<uint16_t*>(k_pool);
  p.v_pool = static_cast<uint16_t*>(v_pool);
  p.err = dev->err;
  p.rows = dims->rows;
  p.hkv = dims->num_kv_heads;
  p.head_dim = dims->head_dim;
  p.maxp = dims->max_pages_per_row;
  p.num_pages = dims->num_pages;
  p.layout = dims->layout;
  return launch_kv_append(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PGD_OK
                                                                                     : PGD_ECUDA;
}

int pgd_kv_append_paged(const pgd_dims* dims, const void* k_new, const void* v_new,
                        const int32_t* table, const int32_t* positions, void* k_pool,
                        void* v_pool, pgd_stream_t stream) {
  return append_impl(dims, k_new, v_new, table, positions, nullptr, k_pool, v_pool, stream);
}

int pgd_rope_append_paged(const pgd_dims* dims, float theta, void* q, const void* k_new,
                          const void* v_new, const int32_t* table, const int32_t* positions,
                          const int32_t* slots, void* k_pool, void* v_pool, pgd_stream_t stream) {
  int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (dims->rows == 0) return PGD_OK;
  if (!(theta > 0.f) || !std::isfinite(theta)) return PGD_EINVAL;
  if (!k_new || !v_new || !positions || !k_pool || !v_pool) return PGD_EINVAL;
  if (!slots && !table && dims->layout != PGD_ROW_MAJOR) return PGD_EINVAL;
  if (!slots && !table && (int64_t)dims->rows * dims->max_pages_per_row > dims->num_pages)
    return PGD_EINVAL;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool) ||
      (q && !aligned16(q)))
    return PGD_EINVAL;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev)) != PGD_OK) return rc;
  RopeAppendParams p;
  p.q = static_cast<uint16_t*>(q);
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  p.table = table;
  p.positions = positions;
  p.slots = slots;
  p.k_pool = static_cast<uint16_t*>(k_pool);
  p.v_pool = static_cast<uint16_t*>(v_pool);
  p.err = dev->err;
  p.rows = dims->rows;
  p.hq = dims->num_q_heads;
  p.hkv = dims->num_kv_heads;
  p.head_dim = dims->head_dim;
  p.maxp = dims->max_pages_per_row;
  p.num_pages = dims->num_pages;
  p.layout = dims->layout;
  if (dims->head_dim / 2 > 64) return PGD_EUNSUPPORTED;
  // inv_freq[i] = exp(-(i * 2 / D) * log(theta)), in f32 as the tables are written
  const float log_theta = logf(theta);
  for (int i = 0; i < dims->head_dim / 2; ++i) {
    const float scaled = ((float)i * 2.0f) / (float)dims->head_dim;
    p.inv_freq[i] = expf(-scaled * log_theta);
  }
  return launch_rope_append(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PGD_OK
             : PGD_ECUDA;
}

int pgd_page_slots(const pgd_dims* dims, int32_t table_rows, const int32_t* table,
                   const int32_t* rows, const int32_t* positions, int32_t* slots,
                   pgd_stream_t stream) {
  int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (dims->rows == 0) return PGD_OK;
  if (!table || !positions || !slots) return PGD_EINVAL;
  if (rows != nullptr && table_rows <= 0) return PGD_EINVAL;
  if ((int64_t)dims->num_pages * kPageSize > (int64_t)INT32_MAX) return PGD_EUNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev)) != PGD_OK) return rc;
  SlotParams p;
  p.table = table;
  p.row_of = rows;
  p.positions = positions;
  p.slots = slots;
  p.err = dev->err;
  p.tokens = dims->rows;
  p.table_rows = rows ? table_rows : dims->rows;
  p.maxp = dims->max_pages_per_row;
  p.num_pages = dims->num_pages;
  return launch_page_slots(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PGD_OK
                                                                                     : PGD_ECUDA;
}

int pgd_kv_write_slots(const pgd_dims* dims, const void* k_new, const void* v_new,
                       const int32_t* slots, void* k_pool, void* v_pool, pgd_stream_t stream) {
  const int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (dims->rows > 0 && !slots) return PGD_EINVAL;
  return append_impl(dims, k_new, v_new, nullptr, nullptr, slots, k_pool, v_pool, stream);
}

size_t pgd_paged_decode_workspace_bytes(const pgd_dims* dims, const pgd_decode_options* opts) {
  if (check_dims(dims) != PGD_OK) return 0;
  DeviceInfo* dev = nullptr;
  if (current_device(&dev) != PGD_OK) return 0;
  return workspace_bytes(dims, make_plan(dims, opts, dev->sm_count));
}

int pgd_attention_kernel_count(const pgd_dims* dims, int32_t table_rows, int32_t window,
                               const pgd_decode_options* opts, int32_t* count) {
  if (!count) return PGD_EINVAL;
  int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (table_rows < 0) return PGD_EINVAL;
  // The arguments are checked before the device is; AUTO's prefill choice
  // then depends on the SM count, as the split size does.
  int kernel = 0;
  if ((rc = resolve_kernel(dims, table_rows, table_rows > 0, opts, &kernel)) != PGD_OK) return rc;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev)) != PGD_OK) return rc;
  int parts = 1;
  if ((rc = resolve_kernel(dims, table_rows, table_rows > 0, opts, &kernel, dev->sm_count,
                           &parts, window)) != PGD_OK)
    return rc;
  const Plan pl = make_plan(dims, opts, dev->sm_count);
  if (dims->rows == 0) {
    *count = 0;
  } else if (kernel == PGD_KERNEL_PREFILL_UMMA || kernel == PGD_KERNEL_PREFILL_PAIR) {
    *count = prefill_umma_launches(dims->rows, dims->num_q_heads / dims->num_kv_heads, window,
                                   parts);
  } else if (kernel == PGD_KERNEL_PREFILL_TILED) {
    *count = 1;
  } else if ((kernel == PGD_KERNEL_AUTO && window > 0 && window <= kMaxWindowKernel) ||
             short_row_kernel(dims, window, opts, kernel, dev->sm_count)) {
    *count = 1;  // the window kernel
  } else {
    const int pages = span_pages(dims, window > 0 ? window : 0);
    *count = (pages + pl.pages_per_split - 1) / pl.pages_per_split > 1 ? 2 : 1;
  }
  return PGD_OK;
}

static int decode_impl(const pgd_dims* dims, int32_t table_rows, const int32_t* row_of,
                       const void* q, const void* k_pool, const void* v_pool,
                       const int32_t* table, const int32_t* positions, const float* sinks,
                       int32_t window, float scale, void* out, void* workspace,
                       size_t workspace_size, const pgd_decode_options* opts,
                       pgd_stream_t stream, const void* k_new = nullptr,
                       const void* v_new = nullptr) {
  int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (dims->rows == 0) return PGD_OK;
  DeviceInfo* dev = nullptr;
  Plan pl;
  DecodeParams p;
  if ((rc = prepare_attention(dims, table_rows, row_of, q, k_pool, v_pool, table, positions, sinks,
                              window, scale, out, workspace, workspace_size, opts, k_new, v_new,
                              &dev, &pl, &p)) != PGD_OK)
    return rc;

  int kernel = 0, parts = 1;
  if ((rc = resolve_kernel(dims, table_rows, row_of != nullptr, opts, &kernel, dev->sm_count,
                           &parts, window)) != PGD_OK)
    return rc;
  const int padded = padded_group(dims->num_q_heads / dims->num_kv_heads);
  // the tcgen05 prefills copy a head_dim-128 K page tile with one 3-D box;
  // each CTA of the paired prefill copies one 64-wide half of a V tile
  const bool tcgen05 = kernel == PGD_KERNEL_PREFILL_UMMA || kernel == PGD_KERNEL_PREFILL_PAIR;
  const int k_kind = tcgen05 ? kMapWholeTile : kMapBoxes;
  const int v_kind = kernel == PGD_KERNEL_PREFILL_UMMA ? kMapWholeTile : kMapBoxes;
  CUtensorMap k_map, v_map;
  if ((rc = encode_pool_map(&k_map, k_pool, dims, k_kind)) != PGD_OK) return rc;
  if ((rc = encode_pool_map(&v_map, v_pool, dims, v_kind)) != PGD_OK) return rc;

  const int grid_pages = span_pages(dims, p.window);
  const int grid_splits = (grid_pages + pl.pages_per_split - 1) / pl.pages_per_split;
  const int pages_per_cta = grid_pages < pl.pages_per_split ? grid_pages : pl.pages_per_split;
  const bool short_rows = short_row_kernel(dims, window, opts, kernel, dev->sm_count);
  const bool split = kernel == PGD_KERNEL_TENSOR_CORE || kernel == PGD_KERNEL_CUDA_CORE ||
                     (kernel == PGD_KERNEL_AUTO && !short_rows &&
                      !(window > 0 && window <= kMaxWindowKernel));
  if (split && !per_token_fits(dims)) return PGD_EUNSUPPORTED;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // prefill step: the tokens' K and V are written by a launch of their own
  // first (a token's keys are read by the other tokens of its row), which
  // also prepares the tcgen05 kernel's work counter and block order
  const bool prefill_write = k_new != nullptr && row_of != nullptr;
  CUtensorMap q_map;
  if (tcgen05 && (rc = encode_q_map(&q_map, q, dims)) != PGD_OK) return rc;
  if (prefill_write) {
    if (launch_prefill_write(p, dims->head_dim, tcgen05, st) != cudaSuccess)
      return PGD_ECUDA;
    p.k_new = p.v_new = nullptr;
    p.k_pool = p.v_pool = nullptr;
  }
  if (kernel == PGD_KERNEL_PREFILL_PAIR)
    return launch_prefill_pair(p, k_map, v_map, q_map, dev->sm_count, prefill_write, st) ==
                   cudaSuccess
               ? PGD_OK
               : PGD_ECUDA;
  if (kernel == PGD_KERNEL_PREFILL_UMMA)
    return launch_prefill_umma(p, k_map, v_map, q_map, dims->head_dim, dev->sm_count,
                               prefill_write, parts, st) == cudaSuccess
               ? PGD_OK
               : PGD_ECUDA;
  if (kernel == PGD_KERNEL_PREFILL_TILED)
    return launch_prefill_tiled(p, k_map, v_map, dims->head_dim, padded, st) == cudaSuccess
               ? PGD_OK
               : PGD_ECUDA;
  cudaError_t e =
      dims->head_dim == 64
          ? launch_decode_d64(p, k_map, v_map, padded, kernel, grid_splits, pages_per_cta,
                              short_rows, st)
          : launch_decode_d128(p, k_map, v_map, padded, kernel, grid_splits, pages_per_cta,
                               short_rows, st);
  return e == cudaSuccess ? PGD_OK : PGD_ECUDA;
}

int pgd_paged_decode_attention(const pgd_dims* dims, const void* q, const void* k_pool,
                               const void* v_pool, const int32_t* table,
                               const int32_t* positions, const float* sinks, int32_t window,
                               float scale, void* out, void* workspace, size_t workspace_size,
                               const pgd_decode_options* opts, pgd_stream_t stream) {
  return decode_impl(dims, dims ? dims->rows : 0, nullptr, q, k_pool, v_pool, table, positions,
                     sinks, window, scale, out, workspace, workspace_size, opts, stream);
}

int pgd_paged_decode_step(const pgd_dims* dims, const void* q, const void* k_new,
                          const void* v_new, void* k_pool, void* v_pool, const int32_t* table,
                          const int32_t* positions, const float* sinks, int32_t window,
                          float scale, void* out, void* workspace, size_t workspace_size,
                          const pgd_decode_options* opts, pgd_stream_t stream) {
  const int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (dims->rows > 0 && (!k_new || !v_new)) return PGD_EINVAL;
  return decode_impl(dims, dims->rows, nullptr, q, k_pool, v_pool, table, positions,
                     sinks, window, scale, out, workspace, workspace_size, opts, stream, k_new,
                     v_new);
}

int pgd_paged_prefill_attention(const pgd_dims* dims, int32_t table_rows, const void* q,
                                const void* k_pool, const void* v_pool, const int32_t* table,
                                const int32_t* rows, const int32_t* positions,
                                const float* sinks, int32_t window, float scale, void* out,
                                void* workspace, size_t workspace_size,
                                const pgd_decode_options* opts, pgd_stream_t stream) {
  const int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (dims->rows > 0 && !rows) return PGD_EINVAL;
  return decode_impl(dims, table_rows, rows, q, k_pool, v_pool, table, positions, sinks, window,
                     scale, out, workspace, workspace_size, opts, stream);
}

int pgd_paged_prefill_step(const pgd_dims* dims, int32_t table_rows, const void* q,
                           const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                           const int32_t* table, const int32_t* rows, const int32_t* positions,
                           const float* sinks, int32_t window, float scale, void* out,
                           void* workspace, size_t workspace_size,
                           const pgd_decode_options* opts, pgd_stream_t stream) {
  const int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (dims->rows > 0 && (!rows || !k_new || !v_new)) return PGD_EINVAL;
  return decode_impl(dims, table_rows, rows, q, k_pool, v_pool, table, positions, sinks, window,
                     scale, out, workspace, workspace_size, opts, stream, k_new, v_new);
}

int pgd_prefill_step_kernel_count(const pgd_dims* dims, int32_t table_rows, int32_t window,
                                  const pgd_decode_options* opts, int32_t* count) {
  if (!count) return PGD_EINVAL;
  if (table_rows <= 0) return PGD_EINVAL;
  int32_t attention = 0;
  int rc = pgd_attention_kernel_count(dims, table_rows, window, opts, &attention);
  if (rc != PGD_OK) return rc;
  if (dims->rows == 0) {
    *count = 0;
    return PGD_OK;
  }
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev)) != PGD_OK) return rc;
  int kernel = 0, parts = 1;
  if ((rc = resolve_kernel(dims, table_rows, true, opts, &kernel, dev->sm_count, &parts,
                           window)) != PGD_OK)
    return rc;
  // the write launch, then the attention kernels (the tcgen05 kernel alone:
  // the write launch prepared its counter and order; then the combine when
  // there are key parts)
  *count = 1 + (kernel == PGD_KERNEL_PREFILL_UMMA || kernel == PGD_KERNEL_PREFILL_PAIR
                    ? 1 + (parts > 1 ? 1 : 0)
                    : attention);
  return PGD_OK;
}

int pgd_get_device_error(pgd_stream_t stream) {
  DeviceInfo* dev = nullptr;
  int rc = current_device(&dev);
  if (rc != PGD_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return PGD_ECUDA;
  unsigned int word = 0;
  if (cudaMemcpyFromSymbol(&word, g_device_error, sizeof word) != cudaSuccess) return PGD_ECUDA;
  const unsigned int zero = 0;
  if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero) != cudaSuccess) return PGD_ECUDA;
  return (int)word;
}

int pgd_selftest_bounded_wait(int32_t* outcome, pgd_stream_t stream) {
  if (!outcome) return PGD_EINVAL;
  DeviceInfo* dev = nullptr;
  const int rc = current_device(&dev);
  if (rc != PGD_OK) return rc;
  return launch_bounded_wait_selftest(dev->err, outcome, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? PGD_OK
             : PGD_ECUDA;
}

const char* pgd_status_string(int status) {
  switch (status) {
    case PGD_OK: return "ok";
    case PGD_EINVAL: return "invalid argument";
    case PGD_EUNSUPPORTED: return "unsupported shape";
    case PGD_ECUDA: return "CUDA error";
    case PGD_EDEVICE_BOUNDS: return "device: table entry or position out of range";
    case PGD_EDEVICE_TIMEOUT: return "device: pipeline wait timed out";
    case PGD_EWORKSPACE: return "workspace too small";
    case PGD_ESCRATCH_LIMIT: return "problem needs more than the library's static scratch";
    default: return "unknown status";
  }
}

int pgd_version(void) { return 200; }

}  // extern "C"

// ---------------------------------------------------------------------------
// Decode without caller-provided workspace, for callers that cannot allocate
// device memory.  The split partials live in this file-scope array (one per
// device that loads the library, held until exit); the host needs its device
// address, looked up once per device.

namespace pgd {
namespace {

static __device__ __align__(256) unsigned char g_static_scratch[PGD_STATIC_SCRATCH_BYTES];

struct StaticScratch {
  std::once_flag once;
  cudaError_t status = cudaSuccess;
  void* ptr = nullptr;
};
StaticScratch g_static[kMaxDevices];

}  // namespace
}  // namespace pgd

extern "C" int pgd_paged_decode_attention_static(const pgd_dims* dims, const void* q,
                                                 const void* k_pool, const void* v_pool,
                                                 const int32_t* table, const int32_t* positions,
                                                 const float* sinks, int32_t window, float scale,
                                                 void* out, const pgd_decode_options* opts,
                                                 pgd_stream_t stream) {
  int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (dims->rows == 0) return PGD_OK;
  const size_t need = pgd_paged_decode_workspace_bytes(dims, opts);
  if (need == 0) return PGD_ECUDA;
  if (need > PGD_STATIC_SCRATCH_BYTES) return PGD_ESCRATCH_LIMIT;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PGD_ECUDA;
  StaticScratch& sc = g_static[dev];
  std::call_once(sc.once, [&] {
    sc.status = cudaGetSymbolAddress(&sc.ptr, g_static_scratch);
  });
  if (sc.status != cudaSuccess || sc.ptr == nullptr) return PGD_ECUDA;
  return pgd_paged_decode_attention(dims, q, k_pool, v_pool, table, positions, sinks, window,
                                    scale, out, sc.ptr, PGD_STATIC_SCRATCH_BYTES, opts, stream);
}
