// Prefill attention with modified scores (paged_score.cuh) on the tcgen05
// tensor cores, sm_103a.
//
// What it computes (include/pgd_ext.h, pgdx_score): packed token p at position
// n of table row r attends, with each query head h of its group, over the keys
// lo .. hi of that row, lo = max(0, first_key, n - window + 1), hi = max(n,
// prefix_len - 1), with scores cap tanh(scale q.k / cap) - slope_h |n - j|, the
// sink in the denominator only; no key seen: zeros.
//
// Work items, their order and runs are those of the one-SM kernel without
// modified scores (paged_prefill_umma.cuh): (block of 2 x 128 / G consecutive
// packed tokens, kv head), two query tiles of 128 (token, head) rows; the
// tokens of a run share table row and first key and have consecutive
// positions, and a run is one pass over the pages that its tokens see.
//
// With a bias a run's pages are taken last first: the nearest keys, usually the
// largest scores, come early, and the running maximum of a softmax in one pass
// hardly rises after them.  Taken first to last every page raised it and O was
// rescaled each time: 895 us, so 712, for 64 heads of 64 over 4000 positions.
//
// What bounds it is the softmax: a page's 64 scores a row are 64 exponentials,
// 256 cycles of a sub-partition's special function unit for each warp, with
// about 300 other instructions, and every trip to TMEM or through a barrier costs
// hundreds of cycles.  So
//   - one warpgroup has a tile to itself, a thread to a row and page: no
//     exchange between threads, and registers for 64 scores and their
//     polynomials at once (208 a thread).  Two warpgroups to a tile, sharing
//     each page or taking pages in turn, have 104 and measured 1.3 to 2 times
//     slower, though twice the warps: what they gain in warps they lose in
//     registers moved, barriers and instructions fetched;
//   - each tile has two S buffers: S of the next page is computed under the
//     softmax of this one;
//   - a page is tried with the reference (the running maximum) as it is, a cap's
//     polynomial for small scores and a bias linear in the key, and what that
//     needs is looked at when the exponentials are there: no maximum to wait for
//     before them.  Where it did not hold for a row of the warp -- a run's first
//     page, a larger score, keys past the query with a bias -- S, still in TMEM,
//     is read again and the page taken in full (with the maximum first on every
//     page: 275 us, so 265, on the chunks below, before the issuers' last form and
//     the residual; 507 us, so 421, with 64 heads of 64);
//   - capped scores without a bias lie within the cap: their reference is 0 to
//     begin with, and scores in the cap's near form never raise it (caps to 52);
//   - a capped score is a polynomial in s^2 times s plus what the exponent needs
//     anyway: y = s Q(s^2) - m, four packed instructions for two keys, and the
//     largest s^2 tells whether it served;
//   - a bias is linear in the key up to the query: 16 keys against the first of
//     them from registers that last the run, the blocks' own offsets from the
//     reference in the subtraction that is there anyway (the whole bias per pair
//     of keys from constants: 712 us, so 650, on 64 heads of 64 over 4000
//     positions);
//   - masked keys are taken out 16 at a time, only where a row of the warp has
//     one (64 selects on every boundary page, in a copy of the page code: 113 us,
//     so 92, for prompts of documents with a prefix and a window);
//   - P is a bf16 head and residual, as in the other attention kernels, and P V two
//     chains of products: rounded to bf16 once an output would be off by as much
//     again as by its own rounding (0.0024 of the outputs' norm, of 0.0017), for
//     289 us in place of 239 with a cap and 273 of 232 without on the chunks below;
//   - a tile without rows of a run (a block that reaches into another row or
//     document) takes no part in it.
//
// Warps (384 threads):
//   0-7   softmax: tile t is warps 4t .. 4t + 3, a thread per query row.
//   8     producer: takes items from the counter, lays out their runs (checks
//         the table, zeroes uncovered outputs), copies Q and streams K pages.
//   9     S issuer and TMEM owner.  10 P V issuer; it zeroes a boundary page's V
//         rows outside the run's range (while the softmax of the page runs).
//   11    V pages.
// Shared memory: K and V rings of page tiles (four each at head_dim 128, eight
// at 64), Q (two buffers at 64, so that the next item's is there early); 192 KB
// of both.  TMEM: O_t at t D, then S of (tile, page mod 2), 64 columns each; P's
// heads, 32 columns of bf16 pairs, over the first half of its S and its residuals over
// the second, so S of the page after next waits for P V.  (With heads alone, P in
// columns of its own, S free once read and tried pages kept in registers: 274 us, of
// 265; 474 of 421 at head_dim 64.)
// Key parts as in the one-SM kernel.
//
// Measured (32 / 8 heads of 128, eight prompt chunks of up to 512 tokens behind
// up to 8192, 2.6e11 operations): 289 us capped, 904 TFLOP/s (315 after seconds of
// it, at the clocks the power limit then leaves), 273 without a cap, 280 with a bias,
// 306 with both (the one-SM kernel takes 334 us without a cap, 569 with the cap built
// into it); 64 / 8 heads of 64 behind up to 4000: 248 capped, 206 without, 224 with a
// bias, 297 with both.  One chunk behind 8000 positions 95 us; prompts of documents
// with prefix, window and bias 100 us.  A page takes about 2300 cycles: 1790 of the
// tensor cores at head_dim 128 (48 a product of S, 64 of P V, 0.29 of it the
// residual's; ncu: active for 65 % of the cycles), fewer at 64; instructions
// issued in 49 %; and the way from P through P V and the next S back to the softmax.
// Tried and left out, with P rounded once (16-21 % faster then): reading the next
// page's S while this one's exponentials run (311 us, of 309 then); a first reference
// from the raw products instead of the full path on a run's first page (252 of 246,
// 106 of 89); polling instead of suspended waits (the same); scalar instead of packed
// arithmetic for the cap (438 of 403).
//
// Every wait is bounded; a timeout records PGD_EDEVICE_TIMEOUT, stops all
// roles, drains in-flight copies and MMAs and frees TMEM before the CTA exits.
#pragma once

#include "paged_prefill_umma.cuh"
#include "pgd_ext_internal.h"

namespace pgd {

template <int D>
struct ModPrefillCfg {
  static constexpr int kRows = 128, kTiles = 2;
  static constexpr int kSoftmaxWarps = 8;
  static constexpr int kProducerWarp = 8, kMmaWarp = 9, kPvWarp = 10, kVWarp = 11;
  static constexpr int kThreads = 384;
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kPage * D * 2;
  static constexpr int kRing = D == 128 ? 4 : 8;
  static constexpr int kQBufs = D == 128 ? 1 : 2;
  static constexpr int kQBoxBytes = kRows * 128;
  static constexpr int kQTileBytes = kRows * D * 2;
  static constexpr int kQBytes = kTiles * kQTileBytes;
  static constexpr int kVOff = kRing * kTileBytes;
  static constexpr int kQOff = 2 * kRing * kTileBytes;
  static constexpr int kBarOff = kQOff + kQBufs * kQBytes;
  static constexpr int kNumBars = 4 * kRing + 6 * kTiles + 4 + 2 * kQBufs + 2;
  static constexpr int kSmemBytes = 1024 + kBarOff + kNumBars * 8;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kOCol = 0, kSCol = kTiles * D;
  // S of (tile t, page i): kSCol + (2 t + i % 2) kPage; P over it, bf16 pairs: heads, residuals
  static constexpr uint32_t kIdescS = umma_idesc_bf16(128, kPage, 0, 0);
  static constexpr uint32_t kIdescPV = umma_idesc_bf16(128, D, 0, 1);
  static_assert(D == 64 || D == 128, "head_dim");
  static_assert(kSCol + 2 * kTiles * kPage <= kTmemCols, "TMEM columns");
  static_assert(kSmemBytes + 24 * 1024 <= 227 * 1024, "shared memory (dynamic + static)");
};

// One work item as the producer laid it out for the other roles.
struct ModItem {
  int valid;  // 0: no more items
  int t_begin, t_end, kvh, runs;
  int part, parts;
  int run_end[257];
  int tok_row[256], tok_pos[256];    // row -1: no pass covers the token
  int tok_first[256], tok_hi[256];   // first key, last visible position
  int run_pg[256], run_last[256];    // pages of the run (of this key part); run_pg -1: no pass
  __device__ int lo(int k, int window) const {
    return max(window > 0 ? tok_pos[k] - window + 1 : 0, tok_first[k]);
  }
  // Whether tile t (of T tokens) has rows of the run of tokens rs .. re - 1.
  __device__ static bool takes_part(int t, int T, int rs, int re) {
    return rs < (t + 1) * T && re > t * T;
  }
};

// What the scores of a kernel may differ by (kernels are built for each, so that
// the page loop holds only its own case).
enum ModKind { kModMask = 0, kModCap = 1, kModBias = 2 };

// A row's scores in log2 units, less m: y_k = s_k Q(s_k^2) + A_k for N raw
// products s at positions rel, rel + 1, .. from the query's.
//   Q: c = scale log2 e without a cap, else the cap's polynomial with the
//      powers of a = scale / cap and the cap folded into its coefficients
//      (near, mid), or cap_far in its place.
//   A: the bias less m, linear in k where every key is at or before the query;
//      nslope is the bias per position of distance (log2 units, <= 0 usually).
// On the packed fp32 pipe, two keys at a time, but cap_far and the bias of
// keys past the query.
enum CapForm { kNoCap, kCapNear, kCapMid, kCapFar };

__device__ __forceinline__ float2 scaled2(float2 v, float2 add, const ModParams& p) {
  return __ffma2_rn(v, make_float2(p.q_scale_log2, p.q_scale_log2), add);
}
__device__ __forceinline__ float2 near2(float2 v, float2 add, const ModParams& p, float* most) {
  const float2 u = __fmul2_rn(v, v);
  if (most) *most = fmax3(*most, u.x, u.y);
  float2 q = __ffma2_rn(make_float2(p.near_q[2], p.near_q[2]), u,
                        make_float2(p.near_q[1], p.near_q[1]));
  q = __ffma2_rn(q, u, make_float2(p.near_q[0], p.near_q[0]));
  return __ffma2_rn(v, q, add);
}
__device__ __forceinline__ float2 mid2(float2 v, float2 add, const ModParams& p) {
  const float2 u = __fmul2_rn(__fmul2_rn(v, v), make_float2(p.a2, p.a2));
  float2 q = __ffma2_rn(make_float2(kMid5, kMid5), u, make_float2(kMid4, kMid4));
  q = __ffma2_rn(q, u, make_float2(kMid3, kMid3));
  q = __ffma2_rn(q, u, make_float2(kMid2, kMid2));
  q = __ffma2_rn(q, u, make_float2(kMid1, kMid1));
  q = __ffma2_rn(q, u, make_float2(kMid0, kMid0));
  return __ffma2_rn(__fmul2_rn(v, make_float2(p.q_scale_log2, p.q_scale_log2)), q, add);
}

// Usual scores, a cap's near form or none: y = s Q(s^2) + add.
// With a cap, *most becomes at least s^2.
template <int KIND>
__device__ __forceinline__ float2 usual2(float2 v, float2 add, const ModParams& p, float* most) {
  return (KIND & kModCap) ? near2(v, add, p, most) : scaled2(v, add, p);
}

// Any other: scores past a cap's near form, or with the bias of keys on both sides
// of the query (N of them, the first at rel from it), less m.
template <int KIND, int N>
__device__ __forceinline__ void any_scores(float (&s)[N], const ModParams& p, float nslope,
                                           int form, float rel, float m) {
  auto each = [&](auto score) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      float2 add = make_float2(-m, -m);
      if constexpr (KIND & kModBias) {
        add.x = fmaf(nslope, fabsf(rel + (float)k), -m);
        add.y = fmaf(nslope, fabsf(rel + (float)(k + 1)), -m);
      }
      const float2 y = score(make_float2(s[k], s[k + 1]), add);
      s[k] = y.x;
      s[k + 1] = y.y;
    }
  };
  if constexpr (KIND & kModCap) {
    if (form == kCapFar)
      each([&](float2 v, float2 add) {
        return make_float2(cap_far(v.x, p.cap_in, p.cap_out) + add.x,
                           cap_far(v.y, p.cap_in, p.cap_out) + add.y);
      });
    else if (form == kCapMid)
      each([&](float2 v, float2 add) { return mid2(v, add, p); });
    else
      each([&](float2 v, float2 add) { return near2(v, add, p, nullptr); });
  } else {
    each([&](float2 v, float2 add) { return scaled2(v, add, p); });
  }
}

// The score, without a bias, of the raw product s.
template <int KIND>
__device__ __forceinline__ float one_score(float s, const ModParams& p, int form) {
  if constexpr ((KIND & kModCap) == 0) return s * p.q_scale_log2;
  return form == kCapFar ? cap_far(s, p.cap_in, p.cap_out) : cap_mid(s, p.cap_in, p.cap_out);
}

// The largest of N values (N a multiple of 16).
template <int N>
__device__ __forceinline__ float row_max(const float (&s)[N]) {
  float top[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) top[j] = fmaxf(s[j], s[8 + j]);
#pragma unroll
  for (int k = 16; k < N; k += 16)
#pragma unroll
    for (int j = 0; j < 8; ++j) top[j] = fmax3(top[j], s[k + j], s[k + 8 + j]);
  return fmax3(fmax3(top[0], top[1], top[2]), fmax3(top[3], top[4], top[5]),
               fmaxf(top[6], top[7]));
}
template <int N>
__device__ __forceinline__ float row_min(const float (&s)[N]) {
  float low[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) low[j] = fminf(s[j], s[4 + j]);
#pragma unroll
  for (int k = 8; k < N; k += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) low[j] = fmin3(low[j], s[k + j], s[k + 4 + j]);
  return fminf(fminf(low[0], low[1]), fminf(low[2], low[3]));
}

// As mbar_wait_abortable, but the thread is suspended between looks at the
// barrier (20 us, or until the phase completes), and the waiting laid out of
// the way of the satisfied case.
__device__ __forceinline__ bool mbar_wait_suspended(uint64_t* bar, uint32_t parity,
                                                    unsigned int* err, volatile int* abort) {
  if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
  const unsigned long long t0 = global_ns();
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
        : "memory");
    if (done) return true;
    if (*abort) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      record_error(err, PGD_EDEVICE_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}

// Slopes to which a bias is taken in its linear form.  That adds up to 15 slope log2 e
// to a score and takes it off again: two roundings, 2^-23 of 15 slope in natural
// units, below 2^-17 up to here (from 1e6 on nothing of the score would be left).  A
// warp with a steeper row takes every page in full, key by key, where the nearest
// key's bias is exact: 186 us to this slope and 251 past it (8 chunks of 512 behind up
// to 4000, 64 / 8 heads of 64), 255 and 278 (32 / 8 heads of 128, up to 8192).
constexpr float kSteepSlope = 4.f;

// kParts: built for key parts (`parts` units per item, partials to
// part_acc / part_ml for the combine launch); otherwise parts is 1 and each
// item's outputs are written directly.
template <int D, bool kParts, int KIND>
__global__ void __launch_bounds__(ModPrefillCfg<D>::kThreads, 1)
    paged_prefill_mod_kernel(const __grid_constant__ CUtensorMap k_map,
                             const __grid_constant__ CUtensorMap v_map,
                             const __grid_constant__ CUtensorMap q_map, const ModParams p,
                             int* item_counter, const int* block_order, int parts,
                             float* part_acc, float* part_ml) {
  using C = ModPrefillCfg<D>;
  constexpr int R = C::kRing, QB = C::kQBufs;
  // With a bias a run's pages are taken last first: the scores then fall from
  // page to page (usually), and the reference never rises.
  constexpr bool kBack = (KIND & kModBias) != 0;
  const int G = p.group;
  const int T = C::kRows / G;  // tokens per tile
  const int tokens = C::kTiles * T;
  const int n_blocks = (p.rows + tokens - 1) / tokens;
  const int n_items = n_blocks * p.hkv;
  const int n_units = kParts ? n_items * parts : n_items;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  extern __shared__ unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* k_slots = base;
  unsigned char* v_slots = base + C::kVOff;
  unsigned char* q_smem = base + C::kQOff;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(base + C::kBarOff);  // K page landed
  uint64_t* k_empty = k_full + R;          // S of the tiles taking part done
  uint64_t* v_full = k_empty + R;          // V page landed
  uint64_t* v_empty = v_full + R;          // their P V done
  // [2 tile + (the tile's page) % 2]:
  uint64_t* s_full = v_empty + R;              // S of the page in TMEM
  uint64_t* p_full = s_full + 2 * C::kTiles;   // P in its place (O rescaled)
  uint64_t* o_done = p_full + 2 * C::kTiles;   // P V of the page done
  uint64_t* item_ready = o_done + 2 * C::kTiles;  // [item % 2] descriptor written
  uint64_t* item_free = item_ready + 2;        // [item % 2] read for the last time
  uint64_t* q_full = item_free + 2;            // [item % QB] Q landed
  uint64_t* q_free = q_full + QB;              // [item % QB] the item's S products done
  uint64_t* fin = q_free + QB;                 // [issuer] every MMA it issued done
  __shared__ ModItem items[2];
  __shared__ volatile int abort_flag;
  __shared__ uint32_t tmem_slot;

  if (tid == 0) {
    for (int s = 0; s < R; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int b = 0; b < 2 * C::kTiles; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 4);  // the warpgroup's warps
      mbar_init(&o_done[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&item_ready[b], 1);
      mbar_init(&item_free[b], C::kSoftmaxWarps + 3);  // softmax warps, issuers, V producer
    }
    for (int b = 0; b < QB; ++b) {
      mbar_init(&q_full[b], 1);
      mbar_init(&q_free[b], 1);
    }
    mbar_init(&fin[0], 1);
    mbar_init(&fin[1], 1);
    mbar_init_fence();
    abort_flag = 0;
  }
  {
    // rows past T * G of each Q tile hold no token: zero them once (the
    // per-item copies fill rows 0 .. T * G - 1 only)
    const int filled = T * G, gap = C::kRows - filled;
    for (int e = tid; e < QB * C::kTiles * C::kBoxes * gap * 8; e += C::kThreads) {
      const int ch = e & 7, r = filled + (e >> 3) % gap, box = (e >> 3) / gap;
      *reinterpret_cast<uint4*>(q_smem + box * C::kQBoxBytes + r * 128 + ch * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_shared();
  }
  if (warp == C::kMmaWarp) tmem_alloc(&tmem_slot, C::kTmemCols);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  // the set-up above touches only this CTA's shared memory and TMEM, so it
  // overlaps the kernel before; everything from here may read its writes
  pdl_wait();
  pdl_allow_dependents();
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait_suspended(bar, parity, p.err, &abort_flag);
  };
  auto all_ok = [&](bool v) { return __all_sync(0xffffffffu, v); };

  // One page tile (64 rows x D): head_dim 128 comes through its 3-D map as
  // both 64-wide boxes in one copy.
  auto load_tile = [&](unsigned char* dst, const CUtensorMap* map, int y, uint64_t* bar) {
    if constexpr (D == 128)
      tma_load_3d(dst, map, 0, y, 0, bar);
    else
      tma_load_2d(dst, map, 0, y, bar);
  };
  // Streams the pages of item `it` into one ring (whole warp), page number i
  // onwards: the table is looked up 16 pages at a time, one page a lane, one
  // look-up ahead.  `is_k`: K pages, and both pools' pages pulled into L2 when
  // they are looked up (the token blocks of a request reach each page together).
  auto stream_item = [&](const ModItem& it, bool is_k, int& i) -> bool {
    uint64_t* full = is_k ? k_full : v_full;
    uint64_t* empty = is_k ? k_empty : v_empty;
    unsigned char* slots = is_k ? k_slots : v_slots;
    const CUtensorMap* map = is_k ? &k_map : &v_map;
    for (int r = 0; r < it.runs; ++r) {
      const int first = it.run_pg[r], last = it.run_last[r];
      if (first < 0 || first > last) continue;
      const int row = it.tok_row[r == 0 ? 0 : it.run_end[r - 1]];
      const int pages = last - first + 1;
      auto look_up = [&](int n0) -> int {
        if (lane >= 16 || n0 + lane >= pages) return 0;
        const int pg = kBack ? last - n0 - lane : first + n0 + lane;
        return (int)tile_first_row(p.layout, page_of(p.table, row, pg, p.maxp), it.kvh, p.hkv,
                                   p.num_pages, p.maxp);
      };
      int y_next = look_up(0);
      for (int n0 = 0; n0 < pages; n0 += 16) {
        const int y = y_next;
        if (is_k && lane < 16 && n0 + lane < pages && n0 + lane >= R) {
          if constexpr (D == 128) {
            tma_prefetch_l2_3d(&k_map, 0, y, 0);
            tma_prefetch_l2_3d(&v_map, 0, y, 0);
          } else {
            tma_prefetch_l2_2d(&k_map, 0, y);
            tma_prefetch_l2_2d(&v_map, 0, y);
          }
        }
        y_next = look_up(n0 + 16);
        for (int j = 0; j < 16 && n0 + j < pages; ++j, ++i) {
          const int yj = __shfl_sync(0xffffffffu, y, j);
          const int s = i % R;
          if (i >= R && !all_ok(wait(&empty[s], ((i / R) - 1) & 1))) return false;
          if (lane == 0) {
            mbar_arrive_expect_tx(&full[s], C::kTileBytes);
            load_tile(slots + s * C::kTileBytes, map, yj, &full[s]);
          }
        }
      }
    }
    return true;
  };
  // no copy may still be landing in shared memory when the CTA exits
  auto drain = [&](uint64_t* full, int issued) {
    if (lane == 0)
      for (int j = max(0, issued - R); j < issued; ++j)
        mbar_wait_bounded(&full[j % R], (j / R) & 1, p.err);
  };

  // The softmax warpgroups hold 64 scores a thread: registers from the other
  // warpgroup (2 x 128 x 208 + 128 x 88 = 384 x 168, the launch's total).
  if (warp >= C::kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == C::kProducerWarp) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&v_map);
        prefetch_tensormap(&q_map);
      }
      int ik = 0, seq = 0;  // K pages issued, items with Q issued
      for (bool ok = true; ok; ++seq) {
        const int d = seq & 1;
        ModItem& it = items[d];
        int j = 0;
        if (lane == 0) j = atomicAdd(item_counter, 1);
        j = __shfl_sync(0xffffffffu, j, 0);
        // the descriptor slot holds item seq - 2 until every role is done with it
        if (seq >= 2 && !all_ok(wait(&item_free[d], ((seq >> 1) - 1) & 1))) break;
        if (j >= n_units) {
          if (lane == 0) {
            it.valid = 0;
            mbar_arrive(&item_ready[d]);
          }
          break;
        }
        // an item's key parts are taken one after another, so they run side by
        // side on different SMs
        const int item = kParts ? j / parts : j;
        const int blk = block_order ? block_order[item / p.hkv] : n_blocks - 1 - item / p.hkv;
        const int kvh = item % p.hkv;
        const int t_begin = blk * tokens, t_end = min(t_begin + tokens, p.rows);
        // the item's Q rows, [token][head] rows of 64 values, once the S products
        // that read the buffer last are done
        const int qb = seq % QB;
        if (seq >= QB && !all_ok(wait(&q_free[qb], ((seq / QB) - 1) & 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[qb], C::kTiles * C::kBoxes * T * G * 128);
          for (int t = 0; t < C::kTiles; ++t)
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_3d(
                  q_smem + qb * C::kQBytes + t * C::kQTileBytes + bx * C::kQBoxBytes, &q_map,
                  64 * bx, kvh * G, t_begin + t * T, &q_full[qb]);
        }
        // tokens: bad ones are reported, and left out of every run with those
        // that see no key (their outputs are zeroed below)
        const int count = t_end - t_begin;
        for (int k = lane; k < count; k += 32) {
          const int t = t_begin + k;
          int row = p.row_of[t], first = 0, hi = -1;
          const int pos = p.positions[t];
          bool bad = row < 0 || row >= p.table_rows || (pos >= 0 && pos / kPage >= p.maxp);
          if (!bad && pos >= 0) {
            const TokenSpan span = mod_span(p, t, row, pos);
            hi = span.hi;
            first = p.first_key ? max(p.first_key[t], 0) : 0;
            bad = hi / kPage >= p.maxp;
            if (span.lo > hi) row = -1;
          }
          if (bad) record_error(p.err, PGD_EDEVICE_BOUNDS);
          if (bad || pos < 0) row = -1;
          it.tok_row[k] = row;
          it.tok_pos[k] = pos;
          it.tok_first[k] = first;
          it.tok_hi[k] = hi;
        }
        __syncwarp();
        // runs: token k ends one when k + 1 starts another (or is past the end);
        // tokens left out in a row are one
        int runs = 0;
        for (int k0 = 0; k0 < count; k0 += 32) {
          const int k = k0 + lane;
          bool brk = false;
          if (k < count)
            brk = k + 1 == count || it.tok_row[k + 1] != it.tok_row[k] ||
                  (it.tok_row[k] >= 0 && (it.tok_pos[k + 1] != it.tok_pos[k] + 1 ||
                                          it.tok_first[k + 1] != it.tok_first[k]));
          const unsigned bal = __ballot_sync(0xffffffffu, brk);
          if (brk) it.run_end[runs + __popc(bal & ((1u << lane) - 1u))] = k + 1;
          runs += __popc(bal);
        }
        if (lane == 0) {
          it.runs = runs;
          it.valid = 1;
          it.t_begin = t_begin;
          it.t_end = t_end;
          it.kvh = kvh;
          it.part = kParts ? j % parts : 0;
          it.parts = kParts ? parts : 1;
        }
        __syncwarp();
        // each run's pages; a table entry outside the pool among them (all of the
        // run's, whatever the key part) leaves it out: zero outputs, reported,
        // before any copy is issued
        for (int r = 0; r < runs; ++r) {
          const int rs = r == 0 ? 0 : it.run_end[r - 1], re = it.run_end[r];
          const int row = it.tok_row[rs];
          int first = -1, last = -1;
          if (row >= 0) {
            first = it.lo(rs, p.window) / kPage;
            last = it.tok_hi[re - 1] / kPage;
            bool bad = false;
            for (int pg = first + lane; pg <= last; pg += 32) {
              const int page = page_of(p.table, row, pg, p.maxp);
              bad |= page < 0 || page >= p.num_pages;
            }
            if (__any_sync(0xffffffffu, bad)) {
              if (lane == 0) record_error(p.err, PGD_EDEVICE_BOUNDS);
              first = -1;
            } else if constexpr (kParts) {
              const int64_t n = last - first + 1;
              const int f = first;
              first = f + (int)(n * it.part / it.parts);
              last = f + (int)(n * (it.part + 1) / it.parts) - 1;
            }
          }
          if (lane == 0) {
            it.run_pg[r] = first;
            it.run_last[r] = last;
          }
          if (first >= 0) continue;
          // outputs of tokens that no pass covers
          const int per_token = G * (D / 8);
          for (int e = lane; e < (re - rs) * per_token; e += 32) {
            const int tl = rs + e / per_token;
            const int g = (e / (D / 8)) % G, ch = e % (D / 8);
            uint16_t* o = p.out + ((size_t)(t_begin + tl) * p.hq + kvh * G + g) * D;
            reinterpret_cast<uint4*>(o)[ch] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_ready[d]);
        ok = stream_item(it, true, ik);
      }
      drain(k_full, ik);
      if (lane == 0)
        for (int j = max(0, seq - QB); j < seq; ++j)
          mbar_wait_bounded(&q_full[j % QB], (j / QB) & 1, p.err);
    } else if (warp == C::kVWarp) {
      // ------------------------------------------------------------ V producer
      int iv = 0;
      for (int seq = 0;; ++seq) {
        const int d = seq & 1;
        if (!all_ok(wait(&item_ready[d], (seq >> 1) & 1))) break;
        const ModItem& it = items[d];
        if (!it.valid) break;
        if (!stream_item(it, false, iv)) break;
        __syncwarp();  // every lane is done with the descriptor (trailing runs without pages)
        if (lane == 0) mbar_arrive(&item_free[d]);
      }
      drain(v_full, iv);
    } else if (warp == C::kMmaWarp) {
      // ------------------------------------------------------------ S issuer
      // (What it and the P V issuer do between a barrier and the products it allows
      // is on every tile's path.  Both wait as whole warps and issue under
      // elect_lane: 249 us where one thread of S and lane 0 of P V took 261, and
      // 473 of 595 at head_dim 64 without cap or bias.)
      const uint32_t k_addr = smem_addr(k_slots);
      int i = 0;                    // page over all items
      int it_[C::kTiles] = {0, 0};  // pages that each tile took part in
      bool ok = true;
      for (int seq = 0; ok; ++seq) {
        const int d = seq & 1, qb = seq % QB;
        if (!all_ok(wait(&item_ready[d], (seq >> 1) & 1))) break;
        const ModItem& it = items[d];
        if (!it.valid) break;
        if (!all_ok(wait(&q_full[qb], (seq / QB) & 1))) break;
        const uint32_t q_addr = smem_addr(q_smem + qb * C::kQBytes);
        int rs = 0;
        for (int r = 0; r < it.runs && ok; ++r) {
          const int first = it.run_pg[r], last = it.run_last[r], re = it.run_end[r];
          const bool part[2] = {ModItem::takes_part(0, T, rs, re),
                                ModItem::takes_part(1, T, rs, re)};
          rs = re;
          if (first < 0) continue;
          for (int n = 0; n <= last - first && ok; ++n, ++i) {
            const int s = i % R;
            if (!all_ok(wait(&k_full[s], (i / R) & 1))) {
              ok = false;
              break;
            }
            const uint64_t kd = umma_desc_sw128(k_addr + s * C::kTileBytes, 16, 1024);
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t) {
              if (!part[t]) continue;
              const int m = it_[t]++, b = 2 * t + (m & 1);
              // the columns are free: P V of the tile's page before last is done
              if (m >= 2 && !all_ok(wait(&o_done[b], ((m >> 1) - 1) & 1))) {
                ok = false;
                break;
              }
              tc_fence_after_sync();
              const uint64_t qd = umma_desc_sw128(q_addr + t * C::kQTileBytes, 16, 1024);
              if (elect_lane()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                  umma_bf16(tmem + C::kSCol + b * kPage,
                            umma_desc_advance(qd, (kk >> 2) * C::kQBoxBytes + (kk & 3) * 32),
                            umma_desc_advance(kd, (kk >> 2) * kBoxBytes + (kk & 3) * 32),
                            C::kIdescS, kk > 0);
                umma_commit(&s_full[b]);
              }
            }
            if (ok && elect_lane()) umma_commit(&k_empty[s]);
          }
        }
        if (ok && elect_lane()) {
          umma_commit(&q_free[qb]);
          mbar_arrive(&item_free[d]);
        }
      }
      // every MMA this thread issued completes before TMEM is freed
      if (it_[0] + it_[1] > 0 && elect_lane()) {
        umma_commit(&fin[0]);
        mbar_wait_bounded(&fin[0], 0, p.err);
      }
    } else if (warp == C::kPvWarp) {
      // ------------------------------------------------------------ P V issuer
      // (the whole warp zeroes boundary pages, one lane issues)
      const uint32_t v_addr = smem_addr(v_slots);
      int i = 0;                    // page over all items
      int it_[C::kTiles] = {0, 0};  // pages that each tile took part in
      bool ok = true;
      for (int seq = 0; ok; ++seq) {
        const int d = seq & 1;
        if (!all_ok(wait(&item_ready[d], (seq >> 1) & 1))) break;
        const ModItem& it = items[d];
        if (!it.valid) break;
        int rs = 0;
        for (int r = 0; r < it.runs && ok; ++r) {
          const int first = it.run_pg[r], last = it.run_last[r], re = it.run_end[r];
          const bool part[2] = {ModItem::takes_part(0, T, rs, re),
                                ModItem::takes_part(1, T, rs, re)};
          // keys that the run's rows see (V of the others is zeroed)
          const int lo = first < 0 ? 0 : it.lo(rs, p.window), hi = it.tok_hi[re - 1];
          rs = re;
          if (first < 0) continue;
          for (int n = 0; n <= last - first && ok; ++n, ++i) {
            const int s = i % R;
            if (!all_ok(wait(&v_full[s], (i / R) & 1))) {
              ok = false;
              break;
            }
            const int pos0 = (kBack ? last - n : first + n) * kPage;
            const int rlo = lo - pos0, rhi = hi - pos0;
            if (rlo > 0 || rhi < kPage - 1) {  // a boundary page
              unsigned char* vt = v_slots + s * C::kTileBytes;
              for (int e = lane; e < kPage * (D / 8); e += 32) {
                const int k = e / (D / 8), ch = e % (D / 8);
                if (k < rlo || k > rhi)
                  *reinterpret_cast<uint4*>(vt + (ch >> 3) * kBoxBytes + k * 128 +
                                            (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_shared();  // the zeros are read by the tensor core
              __syncwarp();
            }
            const uint64_t vd = umma_desc_sw128(v_addr + s * C::kTileBytes, kBoxBytes, 1024);
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t) {
              if (!part[t]) continue;
              const int m = it_[t]++, b = 2 * t + (m & 1);
              if (!all_ok(wait(&p_full[b], (m >> 1) & 1))) {
                ok = false;
                break;
              }
              tc_fence_after_sync();
              const uint32_t pa = tmem + C::kSCol + b * kPage;
              if (elect_lane()) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)  // P's heads, then its residuals
                  umma_bf16_tmem_a(tmem + C::kOCol + t * D, pa + 8 * kk,
                                   umma_desc_advance(vd, (kk & 3) * 2048), C::kIdescPV,
                                   !(n == 0 && kk == 0));
                umma_commit(&o_done[b]);
              }
            }
            if (ok && elect_lane()) umma_commit(&v_empty[s]);
          }
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&item_free[d]);
      }
      // every MMA this warp issued completes before TMEM is freed
      if (it_[0] + it_[1] > 0 && elect_lane()) {
        umma_commit(&fin[1]);
        mbar_wait_bounded(&fin[1], 0, p.err);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------ softmax
    const int m = tid & 127, t = tid >> 7;  // row; tile
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t o_col = lane_base + C::kOCol + t * D;
    constexpr bool kCap = (KIND & kModCap) != 0, kBias = (KIND & kModBias) != 0;
    int i = 0;  // this tile's pages (over all items)
    bool ok = true;
    const int tl = t * T + m / G, g = m % G;  // token of the block, head of the group
    const bool in_tile = m / G < T;
    for (int seq = 0; ok; ++seq) {
      const int d = seq & 1;
      if (!all_ok(wait(&item_ready[d], (seq >> 1) & 1))) break;
      const ModItem& it = items[d];
      if (!it.valid) break;
      const int t_begin = it.t_begin, h0 = it.kvh * G;
      const bool row_ok = in_tile && t_begin + tl < it.t_end;
      // (loaded here, needed later)
      const float slope = kBias ? p.slopes[h0 + g] : 0.f;
      const float sink = !kParts && p.sinks ? p.sinks[h0 + g] : -INFINITY;
      int rs = 0, re = 0;
      for (int r = 0; r < it.runs && ok; ++r) {
        rs = re;
        re = it.run_end[r];
        const int first = it.run_pg[r], last = it.run_last[r];
        const bool live = row_ok && tl >= rs && tl < re;
        // with key parts, a row's partial of this part at [token][head][part]
        auto unit_of = [&]() {
          return ((size_t)(it.t_begin + tl) * p.hq + it.kvh * G + g) * it.parts + it.part;
        };
        if (first < 0 || first > last) {
          // no pass covers these tokens (their outputs are zeroed, the combine
          // leaves them), or the key part has none of their pages
          if constexpr (kParts) {
            if (live) {
              const size_t u = unit_of();
              part_ml[2 * u] = -INFINITY;
              part_ml[2 * u + 1] = first < 0 ? -1.f : 0.f;
            }
          }
          continue;
        }
        if (!ModItem::takes_part(t, T, rs, re)) continue;
        // keys lo .. hi of this row in these pages; rows of other runs go along
        // behind every key and unmasked (their P and O stay their own and are
        // not stored: masking them would cost the run's pages their fast form)
        const int pos = live ? it.tok_pos[tl] : 1 << 30;
        const int lo = live ? it.lo(tl, p.window) : 0;
        const int hi = live ? it.tok_hi[tl] : 1 << 30;
        // the keys that every row of the warp sees; whether one sees keys past itself
        const int lo_all = __reduce_max_sync(0xffffffffu, lo);
        const int hi_all = __reduce_min_sync(0xffffffffu, hi);
        const bool ahead = kBias && __any_sync(0xffffffffu, hi > pos);
        const bool steep = kBias && __any_sync(0xffffffffu, live && fabsf(slope) > kSteepSlope);
        const float nslope = -slope * kLog2e;  // bias per position of distance, log2 units
        float2 step[8];  // bias of 16 keys against the first of them
        if constexpr (kBias) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            step[j] = make_float2(-nslope * (float)(2 * j), -nslope * (float)(2 * j + 1));
        }
        float m_run = p.ref_log2;  // the row's reference (its lazy maximum), log2 units
        float l = 0.f;            // row sum relative to it
        bool begun = p.ref_log2 != -INFINITY;  // every live row of the warp has one
        for (int n = 0; n <= last - first; ++n, ++i) {
          const int pg = kBack ? last - n : first + n;
          const int sb = 2 * t + (i & 1);
          const uint32_t s_col = lane_base + C::kSCol + sb * kPage;
          if (!all_ok(wait(&s_full[sb], (i >> 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const int pos0 = pg * kPage;
          const int k_lo = lo - pos0, k_hi = hi - pos0;  // this row's keys of the page
          // The page is tried as a usual one first: a cap's near form or none, a bias
          // linear in the key, the reference as it is.  Whether that held is known
          // when the exponentials are; if not for a row of the warp, S, still in
          // place, is read again and taken in full.
          const bool linear =
              !steep &&
              (!ahead || __all_sync(0xffffffffu, pos0 + min(k_hi, kPage - 1) <= pos));
          float sv[kPage];
          auto read_s = [&]() {
#pragma unroll
            for (int q = 0; q < kPage / 16; ++q)
              tmem_ld16(s_col + 16 * q, *reinterpret_cast<float(*)[16]>(&sv[16 * q]));
            tmem_wait_ld();
          };
          // Masks go 16 keys at a time, and only where some row of the warp has one:
          // most boundary pages are cut in one or two of their four blocks.
          const bool whole = pos0 >= lo_all && pos0 + kPage - 1 <= hi_all;
          auto mask_to = [&](float value) {
#pragma unroll
            for (int q = 0; q < kPage; q += 16)
              if (pos0 + q < lo_all || pos0 + q + 15 > hi_all) {
#pragma unroll
                for (int k = q; k < q + 16; ++k) sv[k] = k >= k_lo && k <= k_hi ? sv[k] : value;
              }
          };
          // Usual scores: less ref, or with a bias each block of 16 against the bias
          // of its first key, block_bias (then less ref).
          float most[4];
          auto usual_block = [&](int q, float ref) {
            if (q == 0) {
#pragma unroll
              for (int j = 0; j < 4; ++j) most[j] = 0.f;
            }
#pragma unroll
            for (int k = 16 * q; k < 16 * q + 16; k += 2) {
              const float2 y =
                  usual2<KIND>(make_float2(sv[k], sv[k + 1]),
                               kBias ? step[k / 2 % 8] : make_float2(-ref, -ref), p,
                               &most[k / 2 % 4]);
              sv[k] = y.x;
              sv[k + 1] = y.y;
            }
          };
          auto usual_scores = [&](float ref) {
#pragma unroll
            for (int q = 0; q < kPage / 16; ++q) usual_block(q, ref);
          };
          const float rel = (float)(pos0 - pos);
          auto block_bias = [&](int q, float ref) {
            return fmaf(-nslope, rel + (float)(16 * q), -ref);
          };
          auto usual_top = [&](float ref) {
            float top = -INFINITY;
#pragma unroll
            for (int q = 0; q < kPage / 16; ++q)
              top = fmaxf(top, block_bias(q, ref) +
                                   row_max(*reinterpret_cast<float(*)[16]>(&sv[16 * q])));
            return top;
          };
          // P = exp2(scores + offset) of a block, as bf16 heads to w and residuals to
          // wl; added to the sums
          uint32_t w[kPage / 2], wl[kPage / 2];
          float2 sum2[4];
          auto exp_block = [&](int q, float offset) {
            if (q == 0) {
#pragma unroll
              for (int j = 0; j < 4; ++j) sum2[j] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int k = 16 * q; k < 16 * q + 16; k += 2) {
              float2 y = make_float2(sv[k], sv[k + 1]);
              if constexpr (kBias) y = __fadd2_rn(y, make_float2(offset, offset));
              const float2 x = make_float2(exp2_approx(y.x), exp2_approx(y.y));
              sum2[k / 2 & 3] = __fadd2_rn(sum2[k / 2 & 3], x);
              const uint32_t h = pack_bf16x2(x.x, x.y);
              const float2 r = __ffma2_rn(make_float2(bf16_lo(h), bf16_hi(h)),
                                          make_float2(-1.f, -1.f), x);
              w[k / 2] = h;
              wl[k / 2] = pack_bf16x2(r.x, r.y);
            }
          };
          auto page_sum = [&]() {
            const float2 s2 =
                __fadd2_rn(__fadd2_rn(sum2[0], sum2[1]), __fadd2_rn(sum2[2], sum2[3]));
            return s2.x + s2.y;
          };
          bool done = false;
          // Capped scores have a stretch of code of their own for pages without masks
          // (one chunk: 95 us, of 105; with a bias it cost more instruction fetches
          // than it saved, 98 of 89 us for prompts of documents).  It goes block by block,
          // the polynomial of one under the exponentials of the one before (289 us on
          // the header's chunks; 302 with all polynomials first).
          constexpr bool kStraight = KIND == kModCap;
          if (kStraight && whole && begun) {
            read_s();
            const float ref = m_run;
#pragma unroll
            for (int q = 0; q < kPage / 16; ++q) {
              usual_block(q, ref);
              exp_block(q, 0.f);
            }
            const float most2 = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
            float top = -ref;  // (where near scores fit: nothing to bound)
            if (!p.near_fits) top = fmaf(sqrtf(most2), fabsf(p.q_scale_log2), -ref);
            const bool held = !live || (!(top > p.slack_log2) && !(most2 > p.limit_near2));
            done = __all_sync(0xffffffffu, held);
            if (done) l += page_sum();
          } else if (__builtin_expect(linear && begun, 1)) {
            read_s();
            if (kCap && !whole) mask_to(__int_as_float(0x7fffffff));  // (max passes over NaN)
            const float ref = m_run;  // (of a row that is not live, perhaps -inf)
            usual_scores(ref);
            if (!whole) mask_to(-INFINITY);
            const float most2 = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
            // the largest score less the reference, or a bound of it
            float top;
            if constexpr (kBias) {
              top = usual_top(ref);
            } else if constexpr (kCap) {
              top = -ref;  // (as above)
              if (!p.near_fits) top = fmaf(sqrtf(most2), fabsf(p.q_scale_log2), -ref);
            } else {
              top = row_max(sv);
            }
#pragma unroll
            for (int q = 0; q < kPage / 16; ++q) exp_block(q, kBias ? block_bias(q, ref) : 0.f);
            const bool held =
                !live || (!(top > p.slack_log2) && (!kCap || !(most2 > p.limit_near2)));
            done = __all_sync(0xffffffffu, held);
            if (done) l += page_sum();
          }
          if (__builtin_expect(!done, 0)) {
            read_s();
            // The cap's form for the warp's largest product, and the page's maximum:
            // of the products (a score without a bias grows, or falls, with them; max
            // and min pass over a NaN), or with a bias of the scores.
            int form = kNoCap;
            float mx = -INFINITY;
            if ((kCap || !kBias) && !whole) mask_to(__int_as_float(0x7fffffff));
            if constexpr (kCap) {
              const float low = row_min(sv), top = row_max(sv);
              const float most = live ? fmaxf(fabsf(low), fabsf(top)) : 0.f;
              form = !__any_sync(0xffffffffu, most > p.limit_near)  ? kCapNear
                     : !__any_sync(0xffffffffu, most > p.limit_mid) ? kCapMid
                                                                    : kCapFar;
              if constexpr (!kBias)
                mx = fmaxf(one_score<KIND>(top, p, form), one_score<KIND>(low, p, form));
            } else if constexpr (!kBias) {
              mx = p.q_scale_log2 * (p.q_scale_log2 > 0.f ? row_max(sv) : row_min(sv));
            }
            const bool usual = linear && form <= kCapNear;
            if constexpr (kBias) {
              if (usual)
                usual_scores(0.f);
              else
                any_scores<KIND>(sv, p, nslope, form, rel, 0.f);
              if (!whole) mask_to(-INFINITY);
              mx = usual ? usual_top(0.f) : row_max(sv);
            }
            // the row's reference, raised when the maximum exceeds it by the slack
            // (O is then rescaled; a run's first page finds none)
            float alpha = 1.f;
            if (mx > m_run + p.slack_log2) {
              alpha = m_run == -INFINITY || n == 0 ? 1.f : exp2_approx(m_run - mx);
              l *= alpha;  // (0 before the first key)
              m_run = mx;
            }
            begun = __all_sync(0xffffffffu, !live || m_run != -INFINITY);
            if (__any_sync(0xffffffffu, alpha != 1.f)) {
              // O holds the pages before, once P V of the last of them is done
              if (!all_ok(wait(&o_done[sb ^ 1], ((i - 1) >> 1) & 1))) {
                ok = false;
                break;
              }
              tc_fence_after_sync();
#pragma unroll 1
              for (int j = 0; j < D / 16; ++j) {
                float ov[16];
                tmem_ld16(o_col + 16 * j, ov);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) ov[k] *= alpha;
                tmem_st16(o_col + 16 * j, ov);
              }
            }
            const float ref = m_run == -INFINITY ? 0.f : m_run;
            if constexpr (!kBias) {
              any_scores<KIND>(sv, p, nslope, form, 0.f, ref);
              if (!whole) mask_to(-INFINITY);
            }
#pragma unroll
            for (int q = 0; q < kPage / 16; ++q)
              exp_block(q, usual ? block_bias(q, ref) : -ref);
            l += page_sum();
          }
#pragma unroll
          for (int q = 0; q < kPage / 32; ++q) {
            tmem_st16(s_col + 16 * q, *reinterpret_cast<uint32_t(*)[16]>(&w[16 * q]));
            tmem_st16(s_col + kPage / 2 + 16 * q, *reinterpret_cast<uint32_t(*)[16]>(&wl[16 * q]));
          }
          tmem_wait_st();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[sb]);
        }

        if (!ok) break;

        // end of run: the O_t row once P V of the last page is done
        if (!all_ok(wait(&o_done[2 * t + ((i - 1) & 1)], ((i - 1) >> 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        float inv = 1.f;
        float* arow = nullptr;
        if constexpr (kParts) {
          // the row's partial over this part's keys, unnormalised (the sink
          // and the other parts are merged by the combine launch)
          if (live) {
            const size_t u = unit_of();
            part_ml[2 * u] = m_run;
            part_ml[2 * u + 1] = l;
            arow = part_acc + u * D;
          }
        } else if (live) {
          const float sk = sink * kLog2e;
          const float mf = fmaxf(m_run, sk);
          const float scl = exp2_approx(m_run - mf);
          const float total = fmaf(l, scl, exp2_approx(sk - mf));
          inv = l == 0.f ? 0.f : scl / total;
        }
        uint16_t* orow = p.out + ((size_t)(t_begin + (live ? tl : 0)) * p.hq + h0 + g) * D;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          float ov[64];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            tmem_ld16(o_col + 64 * j + 16 * q, *reinterpret_cast<float(*)[16]>(&ov[16 * q]));
          tmem_wait_ld();
          if (!live) continue;
          if constexpr (kParts) {
            float4* dst = reinterpret_cast<float4*>(arow + 64 * j);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              dst[k] = make_float4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(orow + 64 * j);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_uint4(pack_bf16x2(ov[8 * k] * inv, ov[8 * k + 1] * inv),
                                  pack_bf16x2(ov[8 * k + 2] * inv, ov[8 * k + 3] * inv),
                                  pack_bf16x2(ov[8 * k + 4] * inv, ov[8 * k + 5] * inv),
                                  pack_bf16x2(ov[8 * k + 6] * inv, ov[8 * k + 7] * inv));
          }
        }
        tc_fence_before_sync();
      }
      if (!ok) break;
      // this item's descriptor is no longer read
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_free[d]);
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, bool kParts, int KIND>
cudaError_t launch_prefill_mod_kernel(const ModParams& p, const CUtensorMap& k_map,
                                      const CUtensorMap& v_map, const CUtensorMap& q_map,
                                      unsigned ctas, int* counter, const int* order, int parts,
                                      float* part_acc, float* part_ml, cudaStream_t stream) {
  using C = ModPrefillCfg<D>;
  auto kern = paged_prefill_mod_kernel<D, kParts, KIND>;
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(kern, dim3(ctas), dim3(C::kThreads), C::kSmemBytes, stream, k_map, v_map,
                    q_map, p, counter, order, parts, part_acc, part_ml);
}

// As launch_prefill_umma: `prepared` -- the step's write launch has zeroed the
// work counter and written the block order; `parts` > 1 -- key parts, merged by
// a combine launch.
template <int D, int KIND>
cudaError_t launch_prefill_mod(const ModParams& p, const CUtensorMap& k_map,
                               const CUtensorMap& v_map, const CUtensorMap& q_map, int sm_count,
                               bool prepared, int parts, cudaStream_t stream) {
  using C = ModPrefillCfg<D>;
  if (parts < 1 || (parts > 1 && (parts > p.max_splits - 1 || p.rows > 65535)))
    return cudaErrorInvalidValue;
  if (p.rows == 0) return cudaSuccess;
  const int tokens = C::kTiles * (C::kRows / p.group);
  const int n_blocks = (p.rows + tokens - 1) / tokens;
  int* counter = reinterpret_cast<int*>(p.ws_acc);
  const int64_t units = (int64_t)n_blocks * p.hkv * parts;
  // longest first, unless every unit has an SM at once
  const bool sorted = prepared || units > sm_count;
  int* order =
      sorted && p.window == 0 && n_blocks <= kMaxSortedBlocks ? counter + 4 : nullptr;
  cudaError_t e;
  if (!prepared) {
    e = order ? launch_pdl(prefill_block_order_kernel<D, ModScore>, dim3(1),
                           dim3(block_order_threads(n_blocks)), 0, stream, p, tokens, n_blocks,
                           counter, order)
              : cudaMemsetAsync(counter, 0, sizeof(int), stream);
    if (e != cudaSuccess) return e;
  }
  const unsigned ctas = (unsigned)(units < sm_count ? units : sm_count);
  if (parts == 1)
    return launch_prefill_mod_kernel<D, false, KIND>(p, k_map, v_map, q_map, ctas, counter, order,
                                                     1, nullptr, nullptr, stream);
  float* part_acc = prefill_part_acc(p, n_blocks);
  e = launch_prefill_mod_kernel<D, true, KIND>(p, k_map, v_map, q_map, ctas, counter, order, parts,
                                               part_acc, p.ws_ml, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefill_part_combine_kernel<D>, dim3((p.hq + 3) / 4, p.rows), dim3(128), 0,
                    stream, p, parts, static_cast<const float*>(part_acc),
                    static_cast<const float*>(p.ws_ml));
}

}  // namespace pgd
