// Decode attention of rows that share leading pages, sm_103a: every shared
// page is read once for all rows of its group, on the tcgen05 tensor cores.
//
// What it computes is the decode attention of paged_decode.cuh (grouped-query
// attention with sinks; Mistral 7B Instruct v0.3 model files,
// src/attention.linnet, decode_paged; GPT-OSS 20B model files,
// src/attention.linnet, SinkAttention) for rows in groups: the rows b of group
// g, starts[g] <= b < starts[g + 1], hold the same first pages[g] pages.  With
// the softmax split at the end of those pages,
//   (m, l, o) over a set of keys: m >= max_j x_j, l = sum_j 2^(x_j - m),
//   o = sum_j 2^(x_j - m) v_j   (x_j = scale log2 e q . k_j),
// any parts of a row's keys join as M = max m_i, out = sum_i 2^(m_i - M) o_i /
// (sum_i 2^(m_i - M) l_i + 2^(sink - M)).
//
// Work items.  (group, block of 2 x 128 / G rows, kv head) over the shared
// pages: two query tiles of 128 (row, head) pairs, one per TMEM lane, that
// share each K and V page; one tile where a block's rows fit it.  (row, kv head)
// over the row's own pages: one tile of G live lanes -- tensor time of a page
// (384 cycles at head_dim 128) is half of what an SM's share of the HBM
// bandwidth takes for its bytes, so the empty lanes cost nothing.
// All items' pages form one sequence, cut into near-equal ranges, one a CTA
// (one CTA per SM): no CTA ends early, whatever the groups' and rows' lengths.
// A CTA's range covers the end of one item, whole items, the start of another;
// each such segment leaves partials (m, l, o), which the combine launch joins.
// Segments walk a staircase (each next one is of the next item or the next
// CTA), so segment (item, cta) keeps its partials at
//   [live lanes of the items before] + 256 * cta + lane
// without a table.  Offsets: every CTA sums the items' weights itself (two
// barriers, 1.5 us, less than a launch); CTA 0 leaves them for the combine.
//
// Roles of a CTA (384 threads): warps 0-3 and 4-7 softmax of tile 0 and 1, one
// thread a TMEM lane (one-tile items alternate between the tiles, so that one's
// end overlaps the next one's pages); warp 8 producer (segments, Q, K and V by
// TMA, the step's append); warp 9 issues S = Q K^T, warp 10 O += P V:
//   S into one of a tile's two buffers of 64 columns, P over it as a bf16 head
//   and residual (weights to 2^-17, as in every attention kernel here), O in
//   TMEM, rescaled only when a row's maximum rises by more than 2^8.
// Every wait is bounded; a timeout records PGD_EDEVICE_TIMEOUT, stops all
// roles, drains copies and products in flight and frees TMEM.
#pragma once

#include "paged_decode.cuh"
#include "paged_prefill_umma.cuh"
#include "pgd_ext_internal.h"
#include "pgd_umma.cuh"

namespace pgd {

template <int D, int STAGES>
struct SharedCfg {
  static constexpr int kLanes = 128;  // (row, head) pairs of a tile
  static constexpr int kTiles = 2;
  static constexpr int kSoftmaxWarps = 8;
  static constexpr int kProducerWarp = 8, kSWarp = 9, kPvWarp = 10;
  static constexpr int kThreads = 384;
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kPage * D * 2;
  static constexpr int kStages = STAGES;
  static constexpr int kQBoxBytes = kLanes * 128;
  static constexpr int kQTileBytes = kBoxes * kQBoxBytes;
  static constexpr int kSegs = 4;  // segment descriptors in flight
  // Q of a row's own pages: its G heads alone, 8 lanes a box; the products read
  // 128 lanes from there, whatever follows it (lanes that no one reads)
  static constexpr int kSmallQBytes = kBoxes * 1024;
  static constexpr int kQOff = 0;
  static constexpr int kSmallQOff = kTiles * kQTileBytes;
  static constexpr int kStageOff = kSmallQOff + kSegs * kSmallQBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kBarOff = kStageOff + STAGES * kStageBytes;
  static constexpr int kNumBars = 4 * STAGES + 3 * kTiles * 2 + 3 * kSegs + kTiles + 2;
  static constexpr int kSmemBytes = 1024 + kBarOff + kNumBars * 8;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kSCol = kTiles * D;
  static constexpr uint32_t kIdescS = umma_idesc_bf16(128, kPage, 0, 0);
  static constexpr uint32_t kIdescPV = umma_idesc_bf16(128, D, 0, 1);
  static_assert(kSCol + kTiles * 2 * kPage <= kTmemCols, "TMEM columns");
  static_assert(kSmallQOff + (kSegs - 1) * kSmallQBytes + (kBoxes - 1) * 1024 + kQBoxBytes <=
                    kBarOff,
                "a small Q's product stays in the CTA's shared memory");
  static_assert((2 * kMaxSharedGroups + 1) * 4 <= STAGES * kStageBytes, "groups in the stages");
  static_assert(kSmemBytes + 4096 <= 227 * 1024, "shared memory");
};

// Weight of a page in the cut: two tiles' products and exponentials take longer
// than the page's bytes, one tile's do not.
constexpr int kWeightOne = 4, kWeightTwo = 7;

// A run of pages of one item, as the producer lays it out for the other roles.
struct SharedSeg {
  int valid;            // 0: no more
  int tiles, tile;      // one tile: which
  int q_tile;           // first Q tile; -1: the small Q of the descriptor's slot
  int row0, rows, kvh;  // rows of the block
  int pages;            // 0: a page outside the pool, nothing is read
  int rhi;              // last visible position of the last page
  long long part;       // first partial
};

// An entry of the list: a group's shared pages, or a row's own.
struct SharedItem {
  long long weight;  // of all its (block, kv head) pairs
  int pages, first;  // of one pair; the first one's place in the table row
  int unit;          // a page's weight
  int count;         // blocks
  int n;             // own pages: the row's position
  bool bad;
};

__device__ __forceinline__ SharedItem shared_group(const SharedParams& p, int s, int e,
                                                   int pages) {
  const int tile = 128 / p.group, block = 2 * tile;
  SharedItem it;
  it.bad = pages < 0 || pages > p.maxp;
  it.pages = it.bad || e <= s ? 0 : pages;
  it.first = 0;
  it.n = 0;
  it.count = (e - s + block - 1) / block;
  it.unit = e - s > tile ? kWeightTwo : kWeightOne;
  it.weight = (long long)it.count * p.hkv * it.pages * it.unit;
  return it;
}

// `shared`: pages of the row's group (0: in none).
__device__ __forceinline__ SharedItem shared_row(const SharedParams& p, int b, int shared) {
  SharedItem it;
  it.n = p.positions[b];
  it.bad = shared < 0 || shared > p.maxp ||
           (it.n >= 0 && (it.n / kPage >= p.maxp || it.n / kPage < shared));
  it.first = shared;
  it.pages = it.n < 0 || it.bad ? 0 : it.n / kPage + 1 - shared;
  it.count = 1;
  it.unit = kWeightOne;
  it.weight = (long long)p.hkv * it.pages * it.unit;
  return it;
}

// The last g of 0 .. groups with starts[g] <= b, -1: none.  Rows of g = -1 and
// g = groups are in no group.
__device__ __forceinline__ int shared_find(const int* starts, int groups, int b) {
  int lo = -1, hi = groups + 1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= b)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int D, int STAGES>
__global__ void __launch_bounds__(SharedCfg<D, STAGES>::kThreads, 1)
    shared_decode_kernel(const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map,
                         const __grid_constant__ CUtensorMap q_map,
                         const __grid_constant__ CUtensorMap q_small_map, const SharedParams p) {
  using C = SharedCfg<D, STAGES>;
  const int G = p.group;
  const int T = C::kLanes / G;  // rows of a tile
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;

  extern __shared__ unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* q_smem = base;
  unsigned char* q_small = base + C::kSmallQOff;
  unsigned char* stages = base + C::kStageOff;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(base + C::kBarOff);
  uint64_t* k_empty = k_full + STAGES;
  uint64_t* v_full = k_empty + STAGES;
  uint64_t* v_empty = v_full + STAGES;
  uint64_t* s_full = v_empty + STAGES;     // [tile][buffer] S in TMEM
  uint64_t* p_full = s_full + 4;           // P over it
  uint64_t* o_done = p_full + 4;           // P V of it done
  uint64_t* seg_ready = o_done + 4;        // [slot] descriptor written
  uint64_t* seg_free = seg_ready + C::kSegs;
  uint64_t* q_full = seg_free + C::kSegs;  // [slot] the segment's Q landed
  uint64_t* q_free = q_full + C::kSegs;    // [Q tile] its segment's S products done
  uint64_t* fin = q_free + C::kTiles;      // [issuer] all its products done
  __shared__ SharedSeg segs[C::kSegs];
  __shared__ volatile int abort_flag;
  __shared__ uint32_t tmem_slot;
  __shared__ long long warp_sum[C::kThreads / 32];
  __shared__ long long start_rem;
  __shared__ int start_item, start_group;
  __shared__ int y_ring[32];

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);  // the tile's warps
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < C::kSegs; ++i) {
      mbar_init(&seg_ready[i], 1);
      mbar_init(&seg_free[i], 2 + C::kSoftmaxWarps);
      mbar_init(&q_full[i], 1);
    }
    for (int i = 0; i < C::kTiles; ++i) mbar_init(&q_free[i], 1);
    mbar_init(&fin[0], 1);
    mbar_init(&fin[1], 1);
    mbar_init_fence();
    abort_flag = 0;
    start_item = -1;
  }
  if (warp == C::kSWarp) tmem_alloc(&tmem_slot, C::kTmemCols);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  // everything before touches this CTA's own memory only
  pdl_wait();
  pdl_allow_dependents();

  // ---------------------------------------------------------------- the cut
  const int S = p.groups, items = S + p.rows;
  long long Q, u0, u1;  // units a CTA, this one's range
  {
    int* g_start = reinterpret_cast<int*>(stages);  // [S + 1], then pages [S]
    int* g_pages = g_start + S + 1;
    bool unsorted = false;
    for (int g = tid; S > 0 && g <= S; g += C::kThreads) {
      const int s = p.starts[g], before = g > 0 ? p.starts[g - 1] : 0;
      unsorted |= s < before || s > p.rows;
      g_start[g] = s;
      if (g < S) g_pages[g] = p.pages[g];
    }
    unsorted = __syncthreads_or(unsorted);  // every row is bad then
    auto item_at = [&](int i, int& g) {
      if (i < S) {
        g = i;
        return shared_group(p, g_start[i], g_start[i + 1], g_pages[i]);
      }
      g = S > 0 ? shared_find(g_start, S, i - S) : -1;
      return shared_row(p, i - S, g >= 0 && g < S ? g_pages[g] : 0);
    };
    // thread i sums a run of the list
    const int run = (items + C::kThreads - 1) / C::kThreads;
    const int i0 = min(tid * run, items), i1 = min(i0 + run, items);
    long long sum = 0;
    if (!unsorted)
      for (int i = i0; i < i1; ++i) {
        int g;
        sum += item_at(i, g).weight;
      }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += a;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long at = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w < warp) at += warp_sum[w];
      total += warp_sum[w];
    }
    Q = (total + ctas - 1) / ctas;
    if (Q < p.min_units) Q = p.min_units;
    u0 = min(Q * cta, total);
    u1 = min(u0 + Q, total);
    if (cta == 0 && tid == 0) {
      p.item_off[items] = Q;
      if (unsorted) record_error(p.err, PGD_EDEVICE_BOUNDS);
    }
    if (cta == 0 || (at <= u0 && u0 < at + sum)) {
      for (int i = i0; i < i1; ++i) {
        int g = -1;
        SharedItem it;
        it.weight = 0;
        it.bad = true;
        if (!unsorted) it = item_at(i, g);
        if (cta == 0) {  // for the combine; without pages: -1, bad -2
          p.item_off[i] = it.weight > 0 ? at : (it.bad ? -2 : -1);
          if (i >= S) p.row_group[i - S] = g < S ? g : -1;
          if (it.bad) record_error(p.err, PGD_EDEVICE_BOUNDS);
        }
        if (at <= u0 && u0 < at + it.weight && u0 < u1) {
          start_item = i;
          start_group = g;
          start_rem = u0 - at;
        }
        at += it.weight;
      }
    }
  }
  fence_proxy_async_shared();  // the stages are TMA's from here on
  __syncthreads();

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait_abortable(bar, parity, p.err, &abort_flag);
  };
  auto all_ok = [&](bool v) { return __all_sync(0xffffffffu, v); };

  if (warp == C::kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tensormap(&k_map);
      prefetch_tensormap(&v_map);
      prefetch_tensormap(&q_map);
      prefetch_tensormap(&q_small_map);
    }
    auto load_tile = [&](unsigned char* dst, const CUtensorMap* map, int y, uint64_t* bar) {
      if constexpr (D == 128)
        tma_load_3d(dst, map, 0, y, 0, bar);
      else
        tma_load_2d(dst, map, 0, y, bar);
    };
    int kn = 0, vn = 0;       // K and V copies issued
    int seq = 0, qn = 0;      // segments laid out, and with their Q issued
    int q_next = 0;           // Q tile of the next one-tile block
    int q_used[2] = {0, 0};   // segments that took each Q tile
    int tile_next = 0;        // tile of the next one-tile segment
    bool ok = true;
    // The pages of this segment: descriptor, Q, the step's append, then K and V.
    auto segment = [&](const SharedItem& it, bool own, int row0, int rows, int kvh, int pg0,
                       int pg1) -> bool {
      const int d = seq % C::kSegs;
      SharedSeg& sg = segs[d];
      if (seq >= C::kSegs && !all_ok(wait(&seg_free[d], (seq / C::kSegs - 1) & 1))) return false;
      const int count = pg1 - pg0;
      const int32_t* trow = p.table + (size_t)row0 * p.maxp + it.first + pg0;
      bool bad = false;
      for (int k = lane; k < count; k += 32) bad |= trow[k] < 0 || trow[k] >= p.num_pages;
      bad = __any_sync(0xffffffffu, bad);
      const int tiles = rows > T ? 2 : 1;
      const int q_tile = own ? -1 : tiles == 2 ? 0 : q_next;
      if (lane == 0) {
        sg.valid = 1;
        sg.tiles = tiles;
        sg.tile = tiles == 2 ? 0 : tile_next;
        sg.q_tile = q_tile;
        sg.row0 = row0;
        sg.rows = rows;
        sg.kvh = kvh;
        sg.pages = bad ? 0 : count;
        sg.rhi = own && pg1 == it.pages ? it.n % kPage : kPage - 1;
        // live lanes of the items before: the groups', then the rows' own
        sg.part = 256ll * cta + (long long)row0 * p.hq + (long long)kvh * rows * G +
                  (own ? (long long)p.rows * p.hq : 0ll);
        if (bad) record_error(p.err, PGD_EDEVICE_BOUNDS);
        mbar_arrive(&seg_ready[d]);
      }
      __syncwarp();
      ++seq;
      if (tiles == 1) tile_next ^= 1;
      if (bad) {
        if (lane == 0) mbar_arrive(&q_full[d]);
        qn = seq;
        return true;
      }
      if (own) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[d], C::kBoxes * G * 128);
          for (int bx = 0; bx < C::kBoxes; ++bx)
            tma_load_3d(q_small + d * C::kSmallQBytes + bx * 1024, &q_small_map, 64 * bx, kvh * G,
                        row0, &q_full[d]);
        }
      } else {
        // once the products that read these Q tiles are done
        for (int t = q_tile; t < q_tile + tiles; ++t) {
          if (q_used[t] > 0 && !all_ok(wait(&q_free[t], (q_used[t] - 1) & 1))) return false;
          ++q_used[t];
        }
        q_next = tiles == 2 ? 0 : q_next ^ 1;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[d], tiles * C::kBoxes * T * G * 128);
          for (int t = 0; t < tiles; ++t)
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_3d(q_smem + (q_tile + t) * C::kQTileBytes + bx * C::kQBoxBytes, &q_map,
                          64 * bx, kvh * G, row0 + t * T, &q_full[d]);
        }
      }
      qn = seq;
      if (p.k_new != nullptr && own && pg1 == it.pages) {
        // the step's key and value at position n, ahead of the copy of their page
        const int page = trow[count - 1];
        const size_t dst = ((size_t)tile_first_row(p.layout, page, kvh, p.hkv, p.num_pages,
                                                   p.maxp) + it.n % kPage) * D;
        const size_t src = ((size_t)row0 * p.hkv + kvh) * D;
        if (lane < 2 * (D / 8)) {
          const int c = lane % (D / 8);
          const bool is_v = lane >= D / 8;
          *reinterpret_cast<uint4*>((is_v ? p.v_pool : p.k_pool) + dst + 8 * c) =
              *reinterpret_cast<const uint4*>((is_v ? p.v_new : p.k_new) + src + 8 * c);
        }
        asm volatile("fence.proxy.async.global;" ::: "memory");
        __syncwarp();
      }
      for (int k = 0; k < count; ++k) {
        if ((k & 31) == 0) {
          __syncwarp();
          if (k + lane < count)
            y_ring[lane] = (int)tile_first_row(p.layout, trow[k + lane], kvh, p.hkv, p.num_pages,
                                               p.maxp);
          __syncwarp();
        }
        const int st = kn % STAGES;
        const uint32_t ph = (kn / STAGES - 1) & 1;
        unsigned char* slot = stages + st * C::kStageBytes;
        if (kn >= STAGES && !all_ok(wait(&k_empty[st], ph))) return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(&k_full[st], C::kTileBytes);
          load_tile(slot, &k_map, y_ring[k & 31], &k_full[st]);
        }
        ++kn;
        if (vn >= STAGES && !all_ok(wait(&v_empty[st], ph))) return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(&v_full[st], C::kTileBytes);
          load_tile(slot + C::kTileBytes, &v_map, y_ring[k & 31], &v_full[st]);
        }
        ++vn;
      }
      return true;
    };
    // walk the list from the start item on
    long long u = u0, rem = 0;
    int item = start_item, g = start_group;
    if (item >= 0) rem = start_rem;
    while (ok && u < u1 && item >= 0 && item < items) {
      const bool own = item >= S;
      SharedItem it;
      int s, e;
      if (!own) {
        s = p.starts[item];
        e = p.starts[item + 1];
        it = shared_group(p, s, e, p.pages[item]);
      } else {
        s = item - S;
        e = s + 1;
        while (g < S && S > 0 && p.starts[g + 1] <= s) ++g;
        it = shared_row(p, s, g >= 0 && g < S ? p.pages[g] : 0);
      }
      if (it.weight > 0) {
        const int block = 2 * T;
        const long long per = (long long)it.pages * it.unit;  // of one (block, kv head)
        int bh = (int)(rem / per);
        long long at = rem - bh * per;
        for (; ok && u < u1 && bh < it.count * p.hkv; ++bh, at = 0) {
          // the pages whose weight begins in [u, u1)
          const int pg0 = (int)((at + it.unit - 1) / it.unit);
          const int pg1 = (int)min((long long)it.pages, (u1 - u + at + it.unit - 1) / it.unit);
          u += per - at;
          const int row0 = s + bh / p.hkv * block;
          if (pg0 < pg1)
            ok = segment(it, own, row0, min(block, e - row0), bh % p.hkv, pg0, pg1);
        }
      }
      rem = 0;
      if (++item == S) g = -1;
    }
    if (ok) {  // the end
      const int d = seq % C::kSegs;
      if ((seq < C::kSegs || all_ok(wait(&seg_free[d], (seq / C::kSegs - 1) & 1))) && lane == 0) {
        segs[d].valid = 0;
        mbar_arrive(&seg_ready[d]);
      }
    }
    // drain: no copy may still be landing when the CTA exits
    if (lane == 0) {
      for (int j = max(0, kn - STAGES); j < kn; ++j)
        mbar_wait_bounded(&k_full[j % STAGES], (j / STAGES) & 1, p.err);
      for (int j = max(0, vn - STAGES); j < vn; ++j)
        mbar_wait_bounded(&v_full[j % STAGES], (j / STAGES) & 1, p.err);
      for (int j = max(0, qn - C::kSegs); j < qn; ++j)
        mbar_wait_bounded(&q_full[j % C::kSegs], (j / C::kSegs) & 1, p.err);
    }
  } else if (warp == C::kSWarp) {
    // ------------------------------------------------------------ S issuer
    if (lane == 0) {
      int i = 0;             // pages
      int ip[2] = {0, 0};    // pages of each tile
      bool issued = false, ok = true;
      for (int seq = 0; ok; ++seq) {
        const int d = seq % C::kSegs;
        if (!wait(&seg_ready[d], (seq / C::kSegs) & 1)) break;
        const SharedSeg& sg = segs[d];
        if (!sg.valid) break;
        if (!wait(&q_full[d], (seq / C::kSegs) & 1)) break;
        const bool small = sg.q_tile < 0;
        const uint32_t q_addr =
            small ? smem_addr(q_small) + d * C::kSmallQBytes
                  : smem_addr(q_smem) + sg.q_tile * C::kQTileBytes;
        const uint32_t box = small ? 1024 : C::kQBoxBytes;
        const int t0 = sg.tile, t1 = t0 + sg.tiles, pages = sg.pages;
        for (int k = 0; k < pages && ok; ++k, ++i) {
          const int st = i % STAGES;
          if (!wait(&k_full[st], (i / STAGES) & 1)) {
            ok = false;
            break;
          }
          const uint64_t kd = umma_desc_sw128(smem_addr(stages) + st * C::kStageBytes, 16, 1024);
          for (int t = t0; t < t1; ++t) {
            const int n = ip[t], tb = 2 * t + (n & 1);
            // the buffer holds P of the tile's page n - 2 until P V has read it
            if (n >= 2 && !wait(&o_done[tb], (n / 2 - 1) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint32_t sb = tmem + C::kSCol + tb * kPage;
            const uint64_t qd = umma_desc_sw128(q_addr + (t - t0) * C::kQTileBytes, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_bf16(sb, umma_desc_advance(qd, (kk >> 2) * box + (kk & 3) * 32),
                        umma_desc_advance(kd, (kk >> 2) * kBoxBytes + (kk & 3) * 32), C::kIdescS,
                        kk > 0);
            umma_commit(&s_full[tb]);
            ++ip[t];
            issued = true;
          }
          if (ok) umma_commit(&k_empty[st]);
        }
        if (!ok) break;
        if (!small && pages > 0)
          for (int t = 0; t < sg.tiles; ++t) umma_commit(&q_free[sg.q_tile + t]);
        mbar_arrive(&seg_free[d]);
      }
      if (issued) {  // TMEM is freed once every product is done
        umma_commit(&fin[0]);
        mbar_wait_bounded(&fin[0], 0, p.err);
      }
    }
  } else if (warp == C::kPvWarp) {
    // ------------------------------------------------------------ P V issuer
    if (lane == 0) {
      int i = 0;
      int ip[2] = {0, 0};
      bool issued = false, ok = true;
      for (int seq = 0; ok; ++seq) {
        const int d = seq % C::kSegs;
        if (!wait(&seg_ready[d], (seq / C::kSegs) & 1)) break;
        const SharedSeg& sg = segs[d];
        if (!sg.valid) break;
        const int t0 = sg.tile, t1 = t0 + sg.tiles, pages = sg.pages;
        for (int k = 0; k < pages && ok; ++k, ++i) {
          const int st = i % STAGES;
          if (!wait(&v_full[st], (i / STAGES) & 1)) {
            ok = false;
            break;
          }
          const uint64_t vd = umma_desc_sw128(
              smem_addr(stages) + st * C::kStageBytes + C::kTileBytes, kBoxBytes, 1024);
          for (int t = t0; t < t1; ++t) {
            const int n = ip[t], tb = 2 * t + (n & 1);
            // (P of a segment's first page comes after its tile's last O was read)
            if (!wait(&p_full[tb], (n / 2) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint32_t pb = tmem + C::kSCol + tb * kPage, od = tmem + t * D;
            // keys 16 kk ..: P's head in columns 8 kk, its residual 32 further
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16_tmem_a(od, pb + 8 * kk, umma_desc_advance(vd, kk * 2048), C::kIdescPV,
                               k > 0 || kk > 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16_tmem_a(od, pb + 32 + 8 * kk, umma_desc_advance(vd, kk * 2048), C::kIdescPV,
                               true);
            umma_commit(&o_done[tb]);
            ++ip[t];
            issued = true;
          }
          if (ok) umma_commit(&v_empty[st]);
        }
        if (ok) mbar_arrive(&seg_free[d]);
      }
      if (issued) {
        umma_commit(&fin[1]);
        mbar_wait_bounded(&fin[1], 0, p.err);
      }
    }
  } else if (warp < C::kSoftmaxWarps) {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2, m = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float c = p.q_scale_log2;
    const float cc = c > 0.f ? c : 1.f;  // folded into the exponent's FMA if positive
    int n = 0;  // pages of this tile
    int i = 0;  // pages
    bool ok = true;
    for (int seq = 0; ok; ++seq) {
      const int d = seq % C::kSegs;
      if (!all_ok(wait(&seg_ready[d], (seq / C::kSegs) & 1))) break;
      const SharedSeg& sg = segs[d];
      if (!sg.valid) break;
      const int pages = sg.pages, t0 = sg.tile, rhi = sg.rhi;
      const bool mine = t >= t0 && t < t0 + sg.tiles;
      // lanes that hold a (row, head) pair: the tile's first ones
      const int lanes = mine ? min(max(sg.rows - (t - t0) * T, 0), T) * G : 0;
      const long long part = sg.part + (long long)(t - t0) * T * G + m;
      const bool live = m < lanes;
      const bool live_warp = 32 * (warp & 3) < lanes;
      if (mine && pages == 0 && live) {  // not read: the row's output is zero
        p.part_ml[2 * part] = -INFINITY;
        p.part_ml[2 * part + 1] = -1.f;
      }
      if (mine && pages > 0) {
        float m_run = -INFINITY, l = 0.f;
        for (int k = 0; k < pages; ++k, ++n) {
          const int tb = 2 * t + (n & 1);
          const uint32_t scol = lane_base + C::kSCol + tb * kPage;
          if (!all_ok(wait(&s_full[tb], (n / 2) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          if (live_warp) {
            float sv[kPage];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              tmem_ld16(scol + 16 * q, *reinterpret_cast<float(*)[16]>(&sv[16 * q]));
            tmem_wait_ld();
            if (!(c > 0.f)) {
#pragma unroll
              for (int j = 0; j < kPage; ++j) sv[j] *= c;
            }
            if (k == pages - 1 && rhi < kPage - 1) {
#pragma unroll
              for (int j = 0; j < kPage; ++j)
                if (j > rhi) sv[j] = -INFINITY;
            }
            float top[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) top[j] = fmax3(sv[j], sv[8 + j], sv[16 + j]);
#pragma unroll
            for (int j = 0; j < 8; ++j) top[j] = fmax3(top[j], sv[24 + j], sv[32 + j]);
#pragma unroll
            for (int j = 0; j < 8; ++j) top[j] = fmax3(top[j], sv[40 + j], sv[48 + j]);
#pragma unroll
            for (int j = 0; j < 8; ++j) top[j] = fmaxf(top[j], sv[56 + j]);
            const float mx = fmax3(fmax3(top[0], top[1], top[2]), fmax3(top[3], top[4], top[5]),
                                   fmaxf(top[6], top[7])) * cc;
            float alpha = 1.f;
            bool rose = false;
            if (mx > m_run + kLazyRescaleLog2) {
              if (m_run != -INFINITY) {
                alpha = exp2_approx(m_run - mx);
                rose = true;
                l *= alpha;
              }
              m_run = mx;
            }
            const float nml = m_run == -INFINITY ? 0.f : -m_run;
            const float2 cc2 = make_float2(cc, cc), nml2 = make_float2(nml, nml);
            const float2 minus1 = make_float2(-1.f, -1.f);
            float2 sum2[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) sum2[j] = make_float2(0.f, 0.f);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t hw[16], lw[16];
#pragma unroll
              for (int w = 0; w < 16; ++w) {
                const float2 y = __ffma2_rn(
                    make_float2(sv[32 * q + 2 * w], sv[32 * q + 2 * w + 1]), cc2, nml2);
                const float2 x = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                sum2[w & 3] = __fadd2_rn(sum2[w & 3], x);
                hw[w] = pack_bf16x2(x.x, x.y);
                const float2 rr =
                    __ffma2_rn(make_float2(bf16_lo(hw[w]), bf16_hi(hw[w])), minus1, x);
                lw[w] = pack_bf16x2(rr.x, rr.y);
              }
              tmem_st16(scol + 16 * q, hw);
              tmem_st16(scol + 32 + 16 * q, lw);
            }
            const float2 s4 =
                __fadd2_rn(__fadd2_rn(sum2[0], sum2[1]), __fadd2_rn(sum2[2], sum2[3]));
            l += s4.x + s4.y;
            if (__any_sync(0xffffffffu, rose)) {
              // O holds P V up to the page before, which must be done
              const int tp = 2 * t + ((n - 1) & 1);
              if (!all_ok(wait(&o_done[tp], ((n - 1) / 2) & 1))) {
                ok = false;
                break;
              }
              tc_fence_after_sync();
#pragma unroll
              for (int q = 0; q < D / 16; ++q) {
                float ov[16];
                tmem_ld16(lane_base + t * D + 16 * q, ov);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) ov[j] *= alpha;
                tmem_st16(lane_base + t * D + 16 * q, ov);
              }
            }
          }
          if (k == pages - 1 && rhi < kPage - 1) {
            // V rows past the last position may hold anything: zero weights need zeros
            const int ik = i + k;
            if (!all_ok(wait(&v_full[ik % STAGES], (ik / STAGES) & 1))) {
              ok = false;
              break;
            }
            unsigned char* vt = stages + (ik % STAGES) * C::kStageBytes + C::kTileBytes;
            for (int e = (rhi + 1) * (D / 8) + m; e < kPage * (D / 8); e += C::kLanes) {
              const int row = e / (D / 8), ch = e % (D / 8);
              *reinterpret_cast<uint4*>(vt + (ch >> 3) * kBoxBytes + row * 128 + (ch & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_shared();
          }
          tmem_wait_st();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[tb]);
        }
        if (!ok) break;
        // the segment's partials once P V of its last page is done
        const int tl = 2 * t + ((n - 1) & 1);
        if (!all_ok(wait(&o_done[tl], ((n - 1) / 2) & 1))) break;
        tc_fence_after_sync();
        if (live_warp) {
          if (live) {
            p.part_ml[2 * part] = m_run;
            p.part_ml[2 * part + 1] = l;
          }
          float* arow = p.part_acc + part * D;
#pragma unroll
          for (int q = 0; q < D / 16; ++q) {
            float ov[16];
            tmem_ld16(lane_base + t * D + 16 * q, ov);
            tmem_wait_ld();
            if (live) {
              float4* dst = reinterpret_cast<float4*>(arow + 16 * q);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                dst[j] = make_float4(ov[4 * j], ov[4 * j + 1], ov[4 * j + 2], ov[4 * j + 3]);
            }
          }
        }
        tc_fence_before_sync();
      }
      i += pages;
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_free[d]);
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::kSWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins a (row, query head)'s partials: those over its group's pages, then those
// over its own, each kind one a CTA of the range that its pages fell to, 256
// places apart.  Zeros for an inactive row (n < 0), for one that the cut found
// bad, and where a page was outside the pool (l < 0).  One warp each.
template <int D>
__global__ void __launch_bounds__(128) shared_combine_kernel(const SharedParams p) {
  constexpr int kDims = D / 32;
  using Vec = typename std::conditional<kDims == 2, float2, float4>::type;
  const int b = blockIdx.y;
  const int h = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  // (inputs of the kernel before as well, which waited for them)
  const float sk = p.sinks && h < p.hq ? p.sinks[h] * kLog2e : -INFINITY;
  pdl_wait();
  pdl_allow_dependents();
  if (h >= p.hq) return;
  uint16_t* o = p.out + ((size_t)b * p.hq + h) * D + lane * kDims;
  const int S = p.groups, items = S + p.rows;
  const long long Q = p.item_off[items];
  const long long own_off = p.item_off[S + b];
  const int g = p.row_group[b];
  float res[kDims];
#pragma unroll
  for (int j = 0; j < kDims; ++j) res[j] = 0.f;
  if (own_off >= 0) {
    const int G = p.group, kvh = h / G, T = 128 / G, block = 2 * T;
    long long at[2] = {0, 0};  // first partial of each kind
    int count[2] = {0, 0};
    int shared = 0;
    if (g >= 0) {
      const long long off = p.item_off[g];
      const int s = p.starts[g], e = p.starts[g + 1];
      shared = p.pages[g];
      if (off >= 0) {
        const SharedItem it = shared_group(p, s, e, shared);
        const int blk = (b - s) / block, row0 = s + blk * block, rows = min(block, e - row0);
        const long long first =
            off + ((long long)blk * p.hkv + kvh) * it.pages * it.unit;
        const long long c0 = first / Q, c1 = (first + (long long)(it.pages - 1) * it.unit) / Q;
        count[0] = (int)(c1 - c0) + 1;
        at[0] = 256 * c0 + (long long)row0 * p.hq + (long long)kvh * rows * G +
                (b - row0) * G + h % G;
      }
    }
    {
      const SharedItem it = shared_row(p, b, shared);
      const long long first = own_off + (long long)kvh * it.pages * it.unit;
      const long long c0 = first / Q, c1 = (first + (long long)(it.pages - 1) * it.unit) / Q;
      count[1] = (int)(c1 - c0) + 1;
      at[1] = 256 * c0 + (long long)p.rows * p.hq + (long long)b * p.hq + h;
    }
    const int n = count[0] + count[1];
    auto place = [&](int i) {
      return i < count[0] ? at[0] + 256ll * i : at[1] + 256ll * (i - count[0]);
    };
    float mx = sk;
    bool skipped = false, nan = false;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      const float2 ml = i < n ? *reinterpret_cast<const float2*>(p.part_ml + 2 * place(i))
                              : make_float2(-INFINITY, 0.f);
      mx = fmaxf(mx, warp_max(ml.x));
      skipped |= __any_sync(0xffffffffu, ml.y < 0.f);
      nan |= __any_sync(0xffffffffu, ml.y != ml.y);
    }
    if (!skipped && (nan || mx == -INFINITY)) {
      const uint16_t v = nan ? 0x7fff : 0;
#pragma unroll
      for (int j = 0; j < kDims; ++j) o[j] = v;
      return;
    }
    if (!skipped) {
      float den = exp2_approx(sk - mx);
      for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const float2 ml = i < n ? *reinterpret_cast<const float2*>(p.part_ml + 2 * place(i))
                                : make_float2(-INFINITY, 0.f);
        const float f = i < n ? exp2_approx(ml.x - mx) : 0.f;
        den += warp_sum(ml.y * f);
        const int some = min(32, n - i0);
#pragma unroll 4
        for (int k = 0; k < some; ++k) {
          const float fk = __shfl_sync(0xffffffffu, f, k);
          const Vec v =
              *reinterpret_cast<const Vec*>(p.part_acc + place(i0 + k) * D + lane * kDims);
          res[0] = fmaf(v.x, fk, res[0]);
          res[1] = fmaf(v.y, fk, res[1]);
          if constexpr (kDims == 4) {
            res[2] = fmaf(v.z, fk, res[2]);
            res[3] = fmaf(v.w, fk, res[3]);
          }
        }
      }
      const float inv = 1.f / den;
#pragma unroll
      for (int j = 0; j < kDims; ++j) res[j] *= inv;
    }
  }
  if constexpr (kDims == 4)
    *reinterpret_cast<uint2*>(o) =
        make_uint2(pack_bf16x2(res[0], res[1]), pack_bf16x2(res[2], res[3]));
  else
    *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(res[0], res[1]);
}

template <int D, int STAGES>
cudaError_t launch_shared(const SharedParams& p, const CUtensorMap& k_map,
                          const CUtensorMap& v_map, const CUtensorMap& q_map,
                          const CUtensorMap& q_small_map, int ctas, cudaStream_t stream) {
  using C = SharedCfg<D, STAGES>;
  auto kern = shared_decode_kernel<D, STAGES>;
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
  }
  e = launch_pdl(kern, dim3(ctas), dim3(C::kThreads), C::kSmemBytes, stream, k_map, v_map, q_map,
                 q_small_map, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(shared_combine_kernel<D>, dim3((p.hq + 3) / 4, p.rows), dim3(128), 0, stream,
                    p);
}

}  // namespace pgd
