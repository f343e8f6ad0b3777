// Host side of the C ABI declared in include/pgd_ext.h: argument validation
// and launches.
#include <cmath>

#include "pgd_ext_internal.h"
#include "pgd_host.h"

namespace pgd {
namespace {

// Whether the int32 arrays [a, a + na) and [b, b + nb) share a byte.
bool overlap(const int32_t* a, int64_t na, const int32_t* b, int64_t nb) {
  if (!a || !b || na <= 0 || nb <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + 4 * (uintptr_t)nb && y < x + 4 * (uintptr_t)na;
}

// Whether a token's `row` values of the bf16 tensor x (rows of them, `stride` values
// apart, stride >= row) share a byte with the `n` values at y.
bool rows_overlap(const void* x, int64_t rows, int64_t stride, int64_t row, const void* y,
                  int64_t n) {
  // in values: the first row that ends past y, against y's end
  const int64_t at = ((int64_t)reinterpret_cast<uintptr_t>(y) -
                      (int64_t)reinterpret_cast<uintptr_t>(x)) / 2;  // (both 16-byte aligned)
  const int64_t first = at < row ? 0 : (at - row) / stride + 1;
  return first < rows && first * stride < at + n;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// An int32 array of a call.
struct Array {
  const int32_t* at;
  int64_t n;
};

// Whether an array is misaligned, or an output overlaps an input or another output.
template <int NI, int NO>
bool arrays_clash(const Array (&in)[NI], const Array (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    if (!aligned4(out[i].at)) return true;
    for (const Array& a : in)
      if (!aligned4(a.at) || overlap(out[i].at, out[i].n, a.at, a.n)) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].at, out[i].n, out[j].at, out[j].n)) return true;
  }
  return false;
}

// Sizes of a table and a pool whose positions and slots are int32.
int check_table(int32_t rows, int32_t width, int32_t num_pages) {
  if (rows < 0 || width <= 0 || num_pages <= 0) return PGD_EINVAL;
  if ((int64_t)width * kPageSize > (int64_t)INT32_MAX ||
      (int64_t)num_pages * kPageSize > (int64_t)INT32_MAX)
    return PGD_EUNSUPPORTED;
  return PGD_OK;
}

// Where shared_decode's workspace keeps what; the total.
struct SharedLayout {
  size_t ml, off, bytes;
};
SharedLayout shared_layout(const pgd_dims* d) {
  // one a (row, head) for the shared pages, four for its own (of an even count of heads,
  // at an even place)
  const size_t group = d->num_q_heads / d->num_kv_heads;
  const size_t own = 4 * ((group + 1) & ~size_t(1));
  const size_t parts = (size_t)d->rows * d->num_kv_heads * (group + own) +
                       256 * (size_t)kMaxSharedCtas + 1;
  SharedLayout l;
  l.ml = parts * d->head_dim * sizeof(float);
  l.off = (l.ml + parts * 2 * sizeof(float) + 15) / 16 * 16;
  l.bytes = l.off + (size_t)d->rows * sizeof(SharedRecord) + kSharedCutBytes +
            16;  // (to a 32-byte boundary, for stores of 32 bytes)
  return l;
}

// SMs of the current device, for a plan (0: none; the plan is then the smallest device's).
int device_sms() {
  DeviceInfo* dev = nullptr;
  return current_device(&dev) == PGD_OK ? dev->sm_count : 0;
}

// Whether AUTO reads a call's rows one by one, groups or not: where all of their tables'
// pages fit L2, which then serves all but the first of a group's reads, and the shared kernel's
// cut, partials and their join cost more than it saves.  Rows by themselves against shared, us:
// 4 MB 12 : 15, 32 MB 8.8 : 16, 64 MB 12 : 17, 96 MB 13 : 17, 112 MB 17 : 21, 136 MB 19 : 19,
// 190 MB 19.4 : 18.3, 270 MB 34 : 20, 340 MB 43 : 22, 690 MB 60 : 24.
constexpr int64_t kSharedRowBytes = 128ll << 20;
bool shared_row_by_row(const pgd_dims* d) {
  return (int64_t)d->rows * d->num_kv_heads * d->max_pages_per_row * kPageSize * d->head_dim * 4 <=
         kSharedRowBytes;
}

int check_shared(const pgd_dims* d, int32_t groups) {
  const int rc = check_dims(d);
  if (rc != PGD_OK) return rc;
  if (groups < 0) return PGD_EINVAL;
  if (groups > kMaxSharedGroups || d->rows > kMaxGridYZ || d->layout == PGD_ROW_MAJOR)
    return PGD_EUNSUPPORTED;
  return PGD_OK;
}

}  // namespace
}  // namespace pgd

using namespace pgd;

extern "C" {

int pgdx_assign_pages(int32_t requests, int32_t max_pages_per_row, int32_t num_pages,
                      int32_t num_tokens, int32_t* table, const int32_t* cached,
                      const int32_t* new_tokens, const int32_t* free_pages, int32_t num_free,
                      const int32_t* free_head, int32_t* rows, int32_t* positions, int32_t* slots,
                      int32_t* starts, int32_t* lengths, int32_t* free_head_out,
                      pgd_stream_t stream) {
  if (requests < 0 || max_pages_per_row <= 0 || num_pages <= 0 || num_tokens < 0 || num_free < 0)
    return PGD_EINVAL;
  if (requests > 0 && (!table || !cached || !new_tokens || !lengths)) return PGD_EINVAL;
  if (num_free > 0 && !free_pages) return PGD_EINVAL;
  if (num_tokens > 0 && (!rows || !positions || !slots)) return PGD_EINVAL;
  if (!starts || !free_head_out) return PGD_EINVAL;
  const int32_t* in[] = {cached, new_tokens, free_pages, free_head};
  const int64_t in_n[] = {requests, requests, num_free, 1};
  const int32_t* out[] = {table, rows, positions, slots, starts, lengths, free_head_out};
  const int64_t out_n[] = {(int64_t)requests * max_pages_per_row, num_tokens, num_tokens,
                           num_tokens, (int64_t)requests + 1, requests, 1};
  for (int i = 0; i < 7; ++i) {
    if (!aligned4(out[i])) return PGD_EINVAL;
    for (int j = 0; j < 4; ++j)
      if (!aligned4(in[j]) || overlap(out[i], out_n[i], in[j], in_n[j])) return PGD_EINVAL;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out_n[i], out[j], out_n[j])) return PGD_EINVAL;
  }
  // positions and slots are int32
  if ((int64_t)max_pages_per_row * kPageSize > (int64_t)INT32_MAX ||
      (int64_t)num_pages * kPageSize > (int64_t)INT32_MAX)
    return PGD_EUNSUPPORTED;
  DeviceInfo* dev = nullptr;
  const int rc = current_device(&dev);
  if (rc != PGD_OK) return rc;
  AssignParams p;
  p.table = table;
  p.cached = cached;
  p.new_tokens = new_tokens;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.rows = rows;
  p.positions = positions;
  p.slots = slots;
  p.starts = starts;
  p.lengths = lengths;
  p.free_head_out = free_head_out;
  p.err = dev->err;
  p.requests = requests;
  p.maxp = max_pages_per_row;
  p.num_pages = num_pages;
  p.tokens = num_tokens;
  p.num_free = num_free;
  return launch_assign_pages(p, dev->sm_count, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? PGD_OK
             : PGD_ECUDA;
}

int pgdx_rotary_init(const pgdx_rotary_config* c, pgdx_rotary* out) {
  if (!c || !out) return PGD_EINVAL;
  const int rd = c->rotary_dim;
  if (rd < 16 || rd > 128 || rd % 16 != 0) return PGD_EUNSUPPORTED;
  if (c->interleaved != 0 && c->interleaved != 1) return PGD_EINVAL;
  if (!std::isfinite(c->theta) || !(c->theta > 1.0)) return PGD_EINVAL;
  const int kind = c->scaling;
  if (kind < PGDX_ROTARY_NONE || kind > PGDX_ROTARY_BANDED) return PGD_EINVAL;
  if (kind != PGDX_ROTARY_NONE && (!std::isfinite(c->factor) || !(c->factor >= 1.0)))
    return PGD_EINVAL;
  if ((kind == PGDX_ROTARY_YARN || kind == PGDX_ROTARY_BANDED) &&
      (!std::isfinite(c->original_positions) || !(c->original_positions > 0.0)))
    return PGD_EINVAL;
  if (kind == PGDX_ROTARY_YARN &&
      (!(c->beta_slow > 0.0) || !(c->beta_fast > c->beta_slow) || !std::isfinite(c->beta_fast)))
    return PGD_EINVAL;
  if (kind == PGDX_ROTARY_BANDED &&
      (!(c->low_band > 0.0) || !(c->high_band > c->low_band) || !std::isfinite(c->high_band)))
    return PGD_EINVAL;
  if (!std::isfinite(c->attention_factor) || c->attention_factor < 0.0) return PGD_EINVAL;
  const double two_pi = 6.283185307179586476925286766559;
  double theta = c->theta, factor = c->attention_factor;
  if (kind == PGDX_ROTARY_NTK) theta *= std::pow(c->factor, (double)rd / (rd - 2));
  if (!std::isfinite(theta)) return PGD_EINVAL;
  const double log_theta = std::log(theta);
  double a = 0.0, b = 0.0;
  if (kind == PGDX_ROTARY_YARN) {
    a = rd * std::log(c->original_positions / (c->beta_fast * two_pi)) / (2.0 * log_theta);
    b = rd * std::log(c->original_positions / (c->beta_slow * two_pi)) / (2.0 * log_theta);
    if (!c->exact_bounds) {
      a = std::floor(a);
      b = std::ceil(b);
    }
    a = std::fmax(a, 0.0);
    b = std::fmin(b, rd - 1.0);
    if (factor == 0.0) factor = 0.1 * std::log(c->factor) + 1.0;
  }
  if (factor == 0.0) factor = 1.0;
  out->rotary_dim = rd;
  out->interleaved = c->interleaved;
  out->factor = (float)factor;
  out->reserved = 0;
  for (int i = 0; i < 64; ++i) {
    out->turns[i] = 0;
    if (i >= rd / 2) continue;
    double f = std::exp(-2.0 * i / rd * log_theta);  // radians a position
    if (kind == PGDX_ROTARY_LINEAR) f /= c->factor;
    if (kind == PGDX_ROTARY_YARN) {
      const double ramp = std::fmin(std::fmax((i - a) / std::fmax(b - a, 0.001), 0.0), 1.0);
      f = f * (1.0 - ramp) + f / c->factor * ramp;
    }
    if (kind == PGDX_ROTARY_BANDED) {
      const double turns = c->original_positions * f / two_pi;
      const double share =
          std::fmin(std::fmax((turns - c->low_band) / (c->high_band - c->low_band), 0.0), 1.0);
      f = f * share + f / c->factor * (1.0 - share);
    }
    // f <= 1 radian: below 0.16 turns, so the product stays below 2^64
    out->turns[i] = (uint64_t)std::rint(std::ldexp(f / two_pi, 64));
  }
  return PGD_OK;
}

int pgdx_rotary_append(const pgd_dims* dims, const pgdx_rotary* rotary, const void* q,
                       int64_t q_stride, void* q_out, const void* k_new, int64_t k_stride,
                       const void* v_new, int64_t v_stride, const int32_t* table,
                       int32_t table_rows, const int32_t* token_rows, const int32_t* positions,
                       const int32_t* slots, void* k_pool, void* v_pool, pgd_stream_t stream) {
  int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (!rotary) return PGD_EINVAL;
  if (rotary->rotary_dim < 16 || rotary->rotary_dim % 16 != 0 ||
      rotary->rotary_dim > dims->head_dim || !std::isfinite(rotary->factor) ||
      (rotary->interleaved != 0 && rotary->interleaved != 1))
    return PGD_EINVAL;
  if (dims->rows == 0) return PGD_OK;
  if (!k_new || !v_new || !positions || !k_pool || !v_pool) return PGD_EINVAL;
  if ((q == nullptr) != (q_out == nullptr)) return PGD_EINVAL;
  if (!slots && !table && dims->layout != PGD_ROW_MAJOR) return PGD_EINVAL;
  if (!slots && token_rows && table_rows <= 0) return PGD_EINVAL;
  if (!slots && !table &&
      (int64_t)(token_rows ? table_rows : dims->rows) * dims->max_pages_per_row > dims->num_pages)
    return PGD_EINVAL;  // dense rows: every row needs its own P pages
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool) ||
      (q && (!aligned16(q) || !aligned16(q_out))))
    return PGD_EINVAL;
  const int64_t d = dims->head_dim, q_row = dims->num_q_heads * d, kv_row = dims->num_kv_heads * d;
  if (k_stride < kv_row || v_stride < kv_row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return PGD_EINVAL;
  if (q) {
    if (q_stride < q_row || q_stride % 8 != 0) return PGD_EINVAL;
    // q_out is q itself (in place), or apart from it
    const uintptr_t x = reinterpret_cast<uintptr_t>(q), y = reinterpret_cast<uintptr_t>(q_out);
    const uintptr_t x_end = x + 2 * ((uintptr_t)(dims->rows - 1) * q_stride + q_row);
    const uintptr_t y_end = y + 2 * (uintptr_t)dims->rows * q_row;
    if (x == y ? q_stride != q_row : (x < y_end && y < x_end)) return PGD_EINVAL;
    // k and v are read while q_out is written
    if (rows_overlap(k_new, dims->rows, k_stride, kv_row, q_out, dims->rows * q_row) ||
        rows_overlap(v_new, dims->rows, v_stride, kv_row, q_out, dims->rows * q_row))
      return PGD_EINVAL;
  }
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev)) != PGD_OK) return rc;
  RotaryParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  p.q_stride = q_stride;
  p.q_out_stride = q_row;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.table = table;
  p.row_of = token_rows;
  p.positions = positions;
  p.slots = slots;
  p.k_pool = static_cast<uint16_t*>(k_pool);
  p.v_pool = static_cast<uint16_t*>(v_pool);
  p.err = dev->err;
  p.rows = dims->rows;
  p.table_rows = table_rows;
  p.hq = dims->num_q_heads;
  p.hkv = dims->num_kv_heads;
  p.maxp = dims->max_pages_per_row;
  p.num_pages = dims->num_pages;
  p.layout = dims->layout;
  p.rotary = *rotary;
  return launch_rotary_append(p, dims->head_dim, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? PGD_OK
             : PGD_ECUDA;
}

static int attention_impl(const pgd_dims* dims, int32_t table_rows, const int32_t* row_of,
                          const pgdx_score* score, const void* q, const void* k_new,
                          const void* v_new, void* k_pool, void* v_pool, const int32_t* table,
                          const int32_t* positions, const float* sinks, int32_t window,
                          float scale, void* out, void* workspace, size_t workspace_size,
                          const pgd_decode_options* opts, pgd_stream_t stream) {
  int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  const bool prefill = row_of != nullptr;
  if (!score || !std::isfinite(score->softcap) || !aligned4(score->alibi_slopes) ||
      !aligned4(score->first_key) || !aligned4(score->prefix_len))
    return PGD_EINVAL;
  if (!prefill && score->prefix_len) return PGD_EINVAL;
  const int32_t asked = opts ? opts->kernel : PGD_KERNEL_AUTO;
  if (asked < PGD_KERNEL_AUTO || asked > PGD_KERNEL_PREFILL_PAIR) return PGD_EINVAL;
  if (asked == PGD_KERNEL_PREFILL_UMMA && !prefill) return PGD_EINVAL;
  if (asked != PGD_KERNEL_AUTO && asked != PGD_KERNEL_TENSOR_CORE &&
      asked != PGD_KERNEL_PREFILL_UMMA)
    return PGD_EUNSUPPORTED;
  if (!std::isfinite(scale)) return PGD_EINVAL;
  const bool capped = score->softcap > 0.f && scale != 0.f;  // a zero score is its own cap
  if (capped) {
    const float ratio = std::fabs(scale / score->softcap);
    // (a cap that far above the scores: cap_far's error of 2^-21 of it swamps them)
    if (ratio < 0x1p-50f) return PGD_EUNSUPPORTED;
    if (!std::isfinite(ratio) || score->softcap > 0x1p126f) return PGD_EINVAL;
  }
  if (dims->rows == 0) return PGD_OK;
  // (AUTO takes a prefill of more tokens in blocks)
  if (!per_token_fits(dims) && (!prefill || asked == PGD_KERNEL_TENSOR_CORE))
    return PGD_EUNSUPPORTED;
  DeviceInfo* dev = nullptr;
  Plan pl;
  ModParams p;
  if ((rc = prepare_attention(dims, table_rows, row_of, q, k_pool, v_pool, table, positions, sinks,
                              window, scale, out, workspace, workspace_size, opts, k_new, v_new,
                              &dev, &pl, &p)) != PGD_OK)
    return rc;
  p.cap_in = capped ? scale / score->softcap : 0.f;
  p.cap_out = capped ? (float)((double)score->softcap * 1.4426950408889634) : 0.f;
  const float a = std::fabs(p.cap_in), a2 = a * a, c = p.q_scale_log2;
  p.near_q[0] = kNear0 * c;
  p.near_q[1] = kNear1 * c * a2;
  p.near_q[2] = kNear2 * c * a2 * a2;
  p.a2 = a2;
  // The prefill's forms fold powers of a into their coefficients: each serves only
  // while those are normal numbers.
  const auto normal = [](float x) { return std::fabs(x) >= 0x1p-120f && std::fabs(x) <= 0x1p120f; };
  p.limit_near = normal(p.near_q[2]) && normal(c) ? kTanhNear / a : -1.f;
  p.limit_mid = normal(a2) ? kTanhMid / a : -1.f;
  p.limit_near2 = p.limit_near * fabsf(p.limit_near);
  // A row's reference is its first maximum, raised when a score exceeds it by more
  // than 2^8 (each raise is a pass over the row's outputs).  Capped scores without a
  // bias stay within the cap, cap_out in log2 units: up to 76 their reference is 0 to
  // begin with, weights no less than 2^-76, and is raised past 2^24, which a score in
  // the cap's near form (0.3 of 76) does not reach, so that pages in that form need no
  // look at it.  Weights up to 2^24 of 2^20 keys leave |V| up to 2^83 in range.
  p.near_fits = capped && !score->alibi_slopes && p.cap_out <= 76.f;
  static_assert(kTanhNear * 76.f < 24.f, "near scores within the slack");
  p.ref_log2 = p.near_fits ? 0.f : -INFINITY;
  p.slack_log2 = p.near_fits ? 24.f : 8.f;
  p.slopes = score->alibi_slopes;
  p.first_key = score->first_key;
  p.prefix_len = score->prefix_len;

  // The pages a token may span: a window bounds them, unless a prefix adds to it.
  const int32_t bound = p.prefix_len ? 0 : window;
  int kernel = 0, parts = 1;
  if ((rc = resolve_kernel(dims, table_rows, prefill, opts, &kernel, dev->sm_count, &parts,
                           bound)) != PGD_OK)
    return rc;
  if (kernel == PGD_KERNEL_PREFILL_PAIR || (prefill && !per_token_fits(dims)))
    kernel = PGD_KERNEL_PREFILL_UMMA;  // (the pair: AUTO's only)
  // AUTO takes a prefill of little work token by token: that costs about 5 us and
  // 4 + 2.2 pages ns for each token and kv head (pages: the most that one may span;
  // the width of the table, so that a short context in a wide one stays with the
  // blocks), the tcgen05 kernel 12 us at least.  On tables as wide as the context: 156
  // tokens over 800 positions with 2 kv heads 17 us so, 27 in blocks; 9 tokens over
  // 1660 with 8 heads 6 and 12; 178 tokens, 2 heads, window 12, 7 and 17; but 274, 8
  // heads, window 6, 21 and 23, and 372, window 64, 27 and 18.5.
  if (asked == PGD_KERNEL_AUTO && kernel == PGD_KERNEL_PREFILL_UMMA && per_token_fits(dims) &&
      (double)dims->rows * dims->num_kv_heads * (4.0 + 2.2 * span_pages(dims, bound)) < 14000.0)
    kernel = PGD_KERNEL_TENSOR_CORE;
  const bool tcgen05 = kernel == PGD_KERNEL_PREFILL_UMMA;
  CUtensorMap k_map, v_map, q_map;
  // the prefill copies a head_dim-128 page tile with one 3-D box
  const int kind = tcgen05 ? kMapWholeTile : kMapBoxes;
  if ((rc = encode_pool_map(&k_map, k_pool, dims, kind)) != PGD_OK) return rc;
  if ((rc = encode_pool_map(&v_map, v_pool, dims, kind)) != PGD_OK) return rc;
  if (tcgen05 && (rc = encode_q_map(&q_map, q, dims)) != PGD_OK) return rc;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool prefill_write = k_new != nullptr && prefill;
  if (prefill_write) {
    if (launch_mod_prefill_write(p, dims->head_dim, tcgen05, st) != cudaSuccess) return PGD_ECUDA;
    p.k_new = p.v_new = nullptr;
    p.k_pool = p.v_pool = nullptr;
  }
  cudaError_t e;
  if (tcgen05) {
    e = launch_mod_prefill(p, k_map, v_map, q_map, dims->head_dim, dev->sm_count, prefill_write,
                           parts, st);
  } else {
    const int pages = span_pages(dims, bound);
    const int splits = (pages + pl.pages_per_split - 1) / pl.pages_per_split;
    const int per_cta = pages < pl.pages_per_split ? pages : pl.pages_per_split;
    e = dims->head_dim == 64 ? launch_mod_decode_d64(p, k_map, v_map, splits, per_cta, st)
                             : launch_mod_decode_d128(p, k_map, v_map, splits, per_cta, st);
  }
  return e == cudaSuccess ? PGD_OK : PGD_ECUDA;
}

int pgdx_paged_decode(const pgd_dims* dims, const pgdx_score* score, const void* q,
                      const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                      const int32_t* table, const int32_t* positions, const float* sinks,
                      int32_t window, float scale, void* out, void* workspace,
                      size_t workspace_size, const pgd_decode_options* opts,
                      pgd_stream_t stream) {
  return attention_impl(dims, dims ? dims->rows : 0, nullptr, score, q, k_new, v_new, k_pool,
                        v_pool, table, positions, sinks, window, scale, out, workspace,
                        workspace_size, opts, stream);
}

int pgdx_paged_prefill(const pgd_dims* dims, int32_t table_rows, const pgdx_score* score,
                       const void* q, const void* k_new, const void* v_new, void* k_pool,
                       void* v_pool, const int32_t* table, const int32_t* rows,
                       const int32_t* positions, const float* sinks, int32_t window, float scale,
                       void* out, void* workspace, size_t workspace_size,
                       const pgd_decode_options* opts, pgd_stream_t stream) {
  const int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (!rows || table_rows <= 0) return dims->rows == 0 ? PGD_OK : PGD_EINVAL;
  return attention_impl(dims, table_rows, rows, score, q, k_new, v_new, k_pool, v_pool, table,
                        positions, sinks, window, scale, out, workspace, workspace_size, opts,
                        stream);
}

int pgdx_fork_rows(int32_t rows, int32_t max_pages_per_row, int32_t num_pages, int32_t* table,
                   const int32_t* lengths, const int32_t* parents, const int32_t* keep,
                   int32_t* shares, int32_t* free_pages, int32_t num_free,
                   const int32_t* free_head, int32_t* new_lengths, int32_t* sources,
                   int32_t* targets, int32_t* counts, int32_t* free_head_out,
                   pgd_stream_t stream) {
  int rc = check_table(rows, max_pages_per_row, num_pages);
  if (rc != PGD_OK) return rc;
  if (num_free < 0 || !shares || !free_head_out || (num_free > 0 && !free_pages))
    return PGD_EINVAL;
  if (rows > 0 && (!table || !lengths || !parents || !new_lengths || !sources || !targets ||
                   !counts))
    return PGD_EINVAL;
  const int64_t entries = (int64_t)rows * max_pages_per_row;
  const Array in[] = {{lengths, rows}, {parents, rows}, {keep, rows}, {free_head, 1}};
  const Array out[] = {{table, entries}, {shares, num_pages}, {free_pages, num_free},
                       {new_lengths, rows}, {sources, rows}, {targets, rows}, {counts, rows},
                       {free_head_out, 1}};
  if (arrays_clash(in, out)) return PGD_EINVAL;
  if (rows > kMaxForkRows || entries > (1 << 30)) return PGD_EUNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev)) != PGD_OK) return rc;
  ForkParams p;
  p.table = table;
  p.lengths = lengths;
  p.parents = parents;
  p.keep = keep;
  p.shares = shares;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.new_lengths = new_lengths;
  p.sources = sources;
  p.targets = targets;
  p.counts = counts;
  p.free_head_out = free_head_out;
  p.err = dev->err;
  p.rows = rows;
  p.width = max_pages_per_row;
  p.num_pages = num_pages;
  p.num_free = num_free;
  return launch_fork_rows(p, dev->sm_count, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PGD_OK
             : PGD_ECUDA;
}

int pgdx_copy_pages(const pgd_dims* dims, int32_t layers, void* const* k_pools,
                    void* const* v_pools, int32_t copies, const int32_t* sources,
                    const int32_t* targets, const int32_t* counts, pgd_stream_t stream) {
  int rc = check_dims(dims);
  if (rc != PGD_OK) return rc;
  if (layers < 0 || copies < 0) return PGD_EINVAL;
  if (dims->layout == PGD_ROW_MAJOR) return PGD_EUNSUPPORTED;
  if (layers == 0 || copies == 0) return PGD_OK;
  if (!k_pools || !v_pools || !sources || !targets) return PGD_EINVAL;
  if (!aligned4(sources) || !aligned4(targets) || !aligned4(counts)) return PGD_EINVAL;
  for (int32_t i = 0; i < layers; ++i)
    if (!k_pools[i] || !v_pools[i] || !aligned16(k_pools[i]) || !aligned16(v_pools[i]))
      return PGD_EINVAL;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev)) != PGD_OK) return rc;
  CopyParams p;
  p.sources = sources;
  p.targets = targets;
  p.counts = counts;
  p.err = dev->err;
  p.copies = copies;
  p.hkv = dims->num_kv_heads;
  p.num_pages = dims->num_pages;
  p.layout = dims->layout;
  for (int32_t first = 0; first < layers; first += kMaxCopyPools / 2) {
    p.pools = 0;
    for (int32_t i = first; i < layers && p.pools < kMaxCopyPools; ++i) {
      p.pool[p.pools++] = k_pools[i];
      p.pool[p.pools++] = v_pools[i];
    }
    if (launch_copy_pages(p, dims->head_dim, dev->sm_count,
                          reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
      return PGD_ECUDA;
  }
  return PGD_OK;
}

size_t pgdx_compact_workspace_bytes(int32_t num_pages) {
  if (num_pages <= 0) return 0;
  return compact_workspace_bytes(num_pages);
}

int pgdx_compact_pages(int32_t rows, int32_t max_pages_per_row, int32_t num_pages,
                       const int32_t* table, const int32_t* lengths, const int32_t* shares,
                       const int32_t* free_pages, int32_t num_free, const int32_t* free_head,
                       int32_t max_moves, int32_t* new_table, int32_t* new_shares,
                       int32_t* new_free, int32_t* sources, int32_t* targets, int32_t* end,
                       void* workspace, size_t workspace_size, pgd_stream_t stream) {
  int rc = check_table(rows, max_pages_per_row, num_pages);
  if (rc != PGD_OK) return rc;
  if (num_free < 0 || max_moves < 0 || !shares || !new_shares || !end) return PGD_EINVAL;
  if (rows > 0 && (!table || !lengths || !new_table)) return PGD_EINVAL;
  if (num_free > 0 && (!free_pages || !new_free)) return PGD_EINVAL;
  if (max_moves > 0 && (!sources || !targets)) return PGD_EINVAL;
  const int64_t entries = (int64_t)rows * max_pages_per_row;
  if (workspace_size < pgdx_compact_workspace_bytes(num_pages)) return PGD_EWORKSPACE;
  if (!workspace || !aligned16(workspace)) return PGD_EINVAL;
  // an output that is its input is in place
  const Array in[] = {{lengths, rows},
                      {free_head, 1},
                      {table, table == new_table ? 0 : entries},
                      {shares, shares == new_shares ? 0 : num_pages},
                      {free_pages, free_pages == new_free ? 0 : num_free}};
  const Array out[] = {{new_table, entries}, {new_shares, num_pages}, {new_free, num_free},
                       {sources, max_moves}, {targets, max_moves}, {end, 1},
                       {static_cast<int32_t*>(workspace),
                        (int64_t)(pgdx_compact_workspace_bytes(num_pages) / 4)}};
  if (arrays_clash(in, out)) return PGD_EINVAL;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev)) != PGD_OK) return rc;
  CompactParams p;
  p.table = table;
  p.lengths = lengths;
  p.shares = shares;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.new_table = new_table;
  p.new_shares = new_shares;
  p.new_free = new_free;
  p.sources = sources;
  p.targets = targets;
  p.end = end;
  p.bits = static_cast<uint32_t*>(workspace);
  p.err = dev->err;
  p.rows = rows;
  p.width = max_pages_per_row;
  p.num_pages = num_pages;
  p.num_free = num_free;
  p.max_moves = max_moves;
  return launch_compact_pages(p, dev->sm_count, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? PGD_OK
             : PGD_ECUDA;
}

size_t pgdx_shared_decode_workspace_bytes(const pgd_dims* dims, int32_t groups) {
  if (check_shared(dims, groups) != PGD_OK) return 0;
  const size_t shared = shared_layout(dims).bytes;
  const size_t rows = pgd::workspace_bytes(dims, make_plan(dims, nullptr, device_sms()));
  return shared > rows ? shared : rows;  // (for either kernel)
}

int pgdx_shared_decode(const pgd_dims* dims, int32_t groups, const int32_t* group_starts,
                       const int32_t* group_pages, const void* q, const void* k_new,
                       const void* v_new, void* k_pool, void* v_pool, const int32_t* table,
                       const int32_t* positions, const float* sinks, float scale, void* out,
                       void* workspace, size_t workspace_size, const pgd_decode_options* opts,
                       pgd_stream_t stream) {
  int rc = check_shared(dims, groups);
  if (rc != PGD_OK) return rc;
  const int32_t asked = opts ? opts->kernel : PGD_KERNEL_AUTO;
  if (asked < PGD_KERNEL_AUTO || asked > PGD_KERNEL_PREFILL_PAIR) return PGD_EINVAL;
  if (asked != PGD_KERNEL_AUTO && asked != PGD_KERNEL_TENSOR_CORE &&
      asked != PGD_KERNEL_PREFILL_UMMA)
    return PGD_EUNSUPPORTED;
  if (!std::isfinite(scale)) return PGD_EINVAL;
  if (dims->rows == 0) return PGD_OK;
  if (!q || !k_pool || !v_pool || !table || !positions || !out) return PGD_EINVAL;
  if (groups > 0 && (!group_starts || !group_pages)) return PGD_EINVAL;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) ||
      !aligned4(group_starts) || !aligned4(group_pages))
    return PGD_EINVAL;
  if ((k_new == nullptr) != (v_new == nullptr) ||
      (k_new && (!aligned16(k_new) || !aligned16(v_new))))
    return PGD_EINVAL;
  if (workspace_size < pgdx_shared_decode_workspace_bytes(dims, groups)) return PGD_EWORKSPACE;
  if (!workspace || !aligned16(workspace)) return PGD_EINVAL;
  if (asked == PGD_KERNEL_TENSOR_CORE || (asked == PGD_KERNEL_AUTO && shared_row_by_row(dims))) {
    const pgdx_score plain = {0.f, nullptr, nullptr, nullptr};
    return attention_impl(dims, dims->rows, nullptr, &plain, q, k_new, v_new, k_pool, v_pool, table,
                          positions, sinks, 0, scale, out, workspace, workspace_size, nullptr,
                          stream);
  }
  const SharedLayout l = shared_layout(dims);
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev)) != PGD_OK) return rc;
  char* ws =
      reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 31) & ~uintptr_t(31));
  SharedParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.table = table;
  p.positions = positions;
  p.starts = group_starts;
  p.pages = group_pages;
  p.sinks = sinks;
  p.out = static_cast<uint16_t*>(out);
  p.part_acc = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + l.ml);
  p.records = reinterpret_cast<SharedRecord*>(ws + l.off);
  p.cut = reinterpret_cast<SharedCut*>(ws + l.off + (size_t)dims->rows * sizeof(SharedRecord));
  p.err = dev->err;
  p.rows = dims->rows;
  p.groups = groups;
  p.hq = dims->num_q_heads;
  p.hkv = dims->num_kv_heads;
  p.group = dims->num_q_heads / dims->num_kv_heads;
  p.tile = 128 / p.group;
  p.block_inverse = (uint32_t)(((1ull << 32) + 2 * p.tile - 1) / (2 * p.tile));
  p.maxp = dims->max_pages_per_row;
  p.num_pages = dims->num_pages;
  p.layout = dims->layout;
  p.q_scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  p.k_pool = static_cast<uint16_t*>(k_pool);
  p.v_pool = static_cast<uint16_t*>(v_pool);
  CUtensorMap k_map, v_map, q_map;
  if ((rc = encode_pool_map(&k_map, k_pool, dims, kMapWholeTile)) != PGD_OK) return rc;
  if ((rc = encode_pool_map(&v_map, v_pool, dims, kMapWholeTile)) != PGD_OK) return rc;
  if ((rc = encode_q_map(&q_map, q, dims)) != PGD_OK) return rc;
  // (an even number: pairs)
  const int ctas = (dev->sm_count < kMaxSharedCtas ? dev->sm_count : kMaxSharedCtas) & ~1;
  if (ctas < 4) return PGD_EUNSUPPORTED;  // two for the groups' pages, two for the rows'
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dims->head_dim == 64 ? launch_shared_d64(p, k_map, v_map, q_map, ctas, st)
                           : launch_shared_d128(p, k_map, v_map, q_map, ctas, st);
  return e == cudaSuccess ? PGD_OK : PGD_ECUDA;
}

int pgdx_get_device_error(pgd_stream_t stream) {
  DeviceInfo* dev = nullptr;
  const int rc = current_device(&dev);
  if (rc != PGD_OK) return rc;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return PGD_ECUDA;
  unsigned int word = 0;
  if (cudaMemcpyFromSymbol(&word, g_device_error, sizeof word) != cudaSuccess) return PGD_ECUDA;
  const unsigned int zero = 0;
  if (word != 0 && cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero) != cudaSuccess)
    return PGD_ECUDA;
  return (int)word;
}

}  // extern "C"
