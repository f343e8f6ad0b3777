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
// over the row's own pages: G query heads, on mma.sync (MmaConsumer of
// paged_decode.cuh), four warps taking pages in turn -- a tile of tcgen05 would
// have G of 128 lanes in use and one warp's exponentials to wait for on every
// page (measured so: a page of 16 KB in 0.8 us, its share of HBM 0.37).
// The blocks' pages form one sequence, the rows' own another, each cut into ranges
// of near-equal weight, one a CTA (one CTA per SM; the blocks' CTAs first): no CTA ends
// early, whatever the groups' and rows' lengths.  A CTA's range covers the end of one
// item, whole items, the start of another; each such segment leaves partials (m, l, o),
// which the combine launch joins.  Segments walk a staircase (each next one is of the
// next item or the next CTA), so segment (item, cta) keeps its partials at
//   [partials of the items before] + 256 * cta + its own
// without a table: a block's, one per lane, then a row's, one per head from each of
// the four warps that had a page (a merge of the warps cost 2 us a segment).  Offsets:
// every CTA sums the items' weights itself (three barriers, less than a launch); the
// last CTA leaves them for the combine.
//
// What bounds it (H query heads a kv head, pages of 64 x D):
//   few rows a group: the bytes.  16 groups of 4 rows (32/8 heads of 128, 500 to 6000
//   shared positions): 238 MB in 52 us; 131 rows, 128 of them over one prompt (64/8 heads of
//   64): 288 MB in 63 us.  Of that 5 us pass from the launch to the first copies and 1 to the
//   join, which takes 6 to 9: chains of loads, in code that no SM has in its caches yet.
//   many rows: the tensor cores.  A page of two tiles costs 2090 cycles at D = 128, of
//   which the products need 1792: per tile S 8 x 48 (N = 64: the 128 x 16 operand's
//   shared-memory reads are longer than the product) and P V 8 x 64 (head and residual).
//   256 rows over 32768 positions and 16 to 1024 of their own (32/8 heads of 128): 185 us,
//   1110 TFLOP/s of products, 757 without the residual's.
//   rows' own pages beside those: the way into their SMs, 32 KB in 600 cycles (53 bytes a
//   cycle); more stages for them or copies issued in pairs change nothing.
//
// Roles of a CTA (384 threads): warps 0-3 and 4-7 softmax of tile 0 and 1, one
// thread a TMEM lane (one-tile blocks alternate between the tiles, so that one's
// end overlaps the next one's pages), and the own pages' consumers; warp 8 lays
// out the segments and copies Q and K (TMA; and appends the step's key and value),
// warp 11 copies V; warp 9 issues S = Q K^T, warp 10 O += P V:
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
  static constexpr int kProducerWarp = 8, kSWarp = 9, kPvWarp = 10, kVWarp = 11;
  static constexpr int kThreads = 384;
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kPage * D * 2;
  static constexpr int kStages = STAGES;
  static constexpr int kAhead = STAGES;  // (page, kv head) tiles asked of L2 before the cut
  static constexpr int kQBoxBytes = kLanes * 128;
  static constexpr int kQTileBytes = kBoxes * kQBoxBytes;
  // segments in flight: a short one's round (its row's q, its pages, its products) takes 4-6 us
  static constexpr int kSegs = 16;
  static constexpr int kStageOff = kTiles * kQTileBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kBarOff = kStageOff + STAGES * kStageBytes;
  static constexpr int kNumBars = 4 * STAGES + 3 * kTiles * 2 + 2 * kSegs + 2 * kTiles + 2;
  static constexpr int kSmemBytes = 1024 + kBarOff + kNumBars * 8;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kSCol = kTiles * D;
  static constexpr uint32_t kIdescS = umma_idesc_bf16(128, kPage, 0, 0);
  static constexpr uint32_t kIdescPV = umma_idesc_bf16(128, D, 0, 1);
  static_assert(kSCol + kTiles * 2 * kPage <= kTmemCols, "TMEM columns");
  static_assert((2 * kMaxSharedGroups + 1) * 4 <= STAGES * kStageBytes, "groups in the stages");
  static_assert(kSmemBytes + kSegs * 32 + 448 <= 227 * 1024, "shared memory (dynamic + static)");
  static_assert((2 * kMaxSharedGroups + 2) * 4 + kMaxSharedGroups * 8 + kThreads * 16 <=
                    STAGES * kStageBytes,
                "their offsets and the list of items behind them");
};

// Weights in the cut, in about 0.05 us on GB300, fitted to what CTAs of mixed calls
// took: a page of a block of one or two tiles (one tile's takes its share of HBM, two
// tiles' products longer), a page of a row's own, and what a (block or row, kv head)
// costs besides.  (A row's own at 10 and 8, as where they alone load HBM: 256 rows over
// 32768 shared positions 198 us in place of 185, 131 rows of 64 heads 63.8 in place of 62.9.)
constexpr int kUnitOne = 13, kUnitTwo = 23, kUnitOwn = 8, kFixedBlock = 60, kFixedOwn = 6;
constexpr int kMinPages = 4;  // of a CTA's range, at least

// A run of pages of one item, as the producer lays it out for the other roles.
struct alignas(16) SharedSeg {
  long long part;       // first partial
  int pages;            // 0: a page outside the pool, nothing is read
  int row0, kvh, rows;  // rows of the block
  int what;             // the fields below (0: no more)
  int pad;
  __device__ static int fields(bool own, int tiles, int tile, int q_tile, int rhi) {
    return 1 | (own ? 2 : 0) | tiles << 2 | tile << 4 | q_tile << 5 | rhi << 8;
  }
  __device__ bool own() const { return what & 2; }    // a row's own pages
  __device__ int tiles() const { return what >> 2 & 3; }
  __device__ int tile() const { return what >> 4 & 1; }    // a block of one tile: which
  __device__ int q_tile() const { return what >> 5 & 1; }  // its first Q tile
  __device__ int rhi() const { return what >> 8; }  // last visible position of the last page
};
static_assert(sizeof(SharedSeg) == 32, "counted in SharedCfg");

// An entry of the list: a group's shared pages, or a row's own.
struct SharedItem {
  int pages, first;  // of one (block, kv head); the first one's place in the table row
  int unit, fixed;   // a page's weight, and a (block, kv head)'s besides
  int count;         // blocks
  int n;             // own pages: the row's position
  bool bad;
  __device__ long long pair() const { return fixed + (long long)pages * unit; }
  __device__ long long weight(int hkv) const { return pages > 0 ? count * hkv * pair() : 0; }
};

// Blocks of n rows, and the block of row n of a group: n / (2 tile) by a multiplication
// (exact for n up to 65535 + 2 tile).
__device__ __forceinline__ int shared_block_of(const SharedParams& p, int n) {
  return (int)__umulhi((unsigned)n, p.block_inverse);
}
__device__ __forceinline__ int shared_blocks(const SharedParams& p, int n) {
  return shared_block_of(p, n + 2 * p.tile - 1);
}

__device__ __forceinline__ SharedItem shared_group(const SharedParams& p, int s, int e,
                                                   int pages) {
  SharedItem it;
  it.bad = pages < 0 || pages > p.maxp;
  it.pages = it.bad || e <= s ? 0 : pages;
  it.first = 0;
  it.n = 0;
  it.count = shared_blocks(p, e - s);
  it.unit = e - s > p.tile ? kUnitTwo : kUnitOne;
  it.fixed = kFixedBlock;
  return it;
}

// A row at position n; `shared`: pages of its group (0: in none).
__device__ __forceinline__ SharedItem shared_row(const SharedParams& p, int n, int shared) {
  SharedItem it;
  it.n = n;
  it.bad = shared < 0 || shared > p.maxp ||
           (it.n >= 0 && (it.n / kPage >= p.maxp || it.n / kPage < shared));
  it.first = shared;
  it.pages = it.n < 0 || it.bad ? 0 : it.n / kPage + 1 - shared;
  it.count = 1;
  it.unit = kUnitOwn;
  it.fixed = kFixedOwn;
  return it;
}

// a / b of weights, a >= 0, b > 0 (64-bit division is a hundred instructions).
__device__ __forceinline__ long long shared_divide(long long a, long long b) {
  return (a | b) >> 32 == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The ranges of the blocks' weights and of the rows': so many CTAs each, an even number
// (a pair of CTAs is a TPC, whose SMs slow each other's pages where one reads shared
// pages and the other rows' own; one such pair among 76 shows little: any number takes 52.3,
// 63.1, 185.2 us in place of 51.9, 62.9, 184.5 for the header's three calls), whichever even
// number leaves the least to the most loaded one.
struct alignas(16) SharedCut {
  long long blocks;  // weight of all blocks
  long long block_range, row_range;  // weight of a CTA's range
  float block_inverse, row_inverse;  // 1 / these, near enough for ctas
  int block_ctas, pad;
  __device__ long long begin(int cta, long long total) const {
    return cta < block_ctas ? min(block_range * cta, blocks)
                            : min(blocks + row_range * (cta - block_ctas), total);
  }
  __device__ static int cta_of(long long at, long long range, float inverse) {
    const int n = (int)((float)at * inverse);  // off by one at most
    const long long rest = at - n * range;
    return rest < 0 ? n - 1 : rest >= range ? n + 1 : n;
  }
  __device__ int block_cta(long long at) const { return cta_of(at, block_range, block_inverse); }
  __device__ int row_cta(long long at) const {
    return block_ctas + cta_of(at - blocks, row_range, row_inverse);
  }
};
static_assert(sizeof(SharedCut) == kSharedCutBytes, "the host's share of the workspace");

// A CTA's range where n of them take a weight: no less than weight / n (by 2^-20, more than the
// three roundings can take off), and no less than four pages of a row's own.
__device__ __forceinline__ long long shared_range(long long weight, int n) {
  constexpr long long least = kMinPages * kUnitOwn;
  static_assert(least >= kUnitTwo, "no range between two pages' beginnings");
  return max((long long)(__fdividef((float)weight, (float)n) * 1.000001f) + 1, least);
}

__device__ __forceinline__ SharedCut shared_cut(long long blocks, long long total, int ctas) {
  const long long rows = total - blocks;
  SharedCut c;
  c.pad = 0;
  c.blocks = blocks;
  c.block_ctas = blocks == 0 ? 0 : ctas;
  if (blocks > 0 && rows > 0) {
    const float share = __fdividef((float)blocks, (float)total) * (float)ctas;
    int n = min(max((int)share & ~1, 2), ctas - 2);  // or two more
    if (n + 2 < ctas && (float)blocks * (float)(ctas - n - 2) > (float)rows * (float)n) n += 2;
    c.block_ctas = n;
  }
  c.block_range = shared_range(blocks, max(c.block_ctas, 1));
  c.row_range = shared_range(rows, max(ctas - c.block_ctas, 1));
  c.block_inverse = __fdividef(1.f, (float)c.block_range);
  c.row_inverse = __fdividef(1.f, (float)c.row_range);
  return c;
}

// Pages whose weight begins before n (>= 0) of one (block or row, kv head)'s, `unit` each.
__device__ __forceinline__ int shared_pages_before(long long n, int unit) {
  const unsigned m = (unsigned)n + unit - 1;  // (2^25 pages at most)
  return (int)(unit == kUnitTwo ? m / kUnitTwo : unit == kUnitOne ? m / kUnitOne : m / kUnitOwn);
}

// The rows' partials come after the blocks', at an even place (as all steps from there
// are): two heads' (m, l) are stored together.
__device__ __forceinline__ long long shared_own_part(const SharedParams& p) {
  return ((long long)p.rows * p.hq + 1) & ~1ll;
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

// The number of copies issued, as one warp leaves it for the others: what was written
// before it is seen with it.
__device__ __forceinline__ void shared_store_count(int* at, int n) {
  asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(smem_addr(at)), "r"(n) : "memory");
}
__device__ __forceinline__ int shared_load_count(const int* at) {
  int n;
  asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(n) : "r"(smem_addr(at)) : "memory");
  return n;
}

// Waits until more than n copies are issued, or the n of `total` (-1: not known yet),
// and returns how many are; -1 where it gives up (as mbar_wait_abortable).  A consumer's wait
// comes before its wait for the copy itself, whose parity it would take for the
// round's before if it came a round early.
__device__ __forceinline__ int shared_wait_count(const int* issued, const int* total, int n,
                                                 unsigned int* err, volatile int* abort) {
  int c = shared_load_count(issued);
  if (c > n) return c;
  const unsigned long long t0 = global_ns();
  for (uint32_t it = 1;; ++it) {
    if (total != nullptr && shared_load_count(total) == n) return n;
    __nanosleep(20);
    c = shared_load_count(issued);
    if (c > n) return c;
    if ((it & 63u) == 0u) {
      if (*abort) return -1;
      if (global_ns() - t0 > kWaitLimitNs) {
        record_error(err, PGD_EDEVICE_TIMEOUT);
        *abort = 1;
        return -1;
      }
    }
  }
}

// Asks for `bytes` (of 16) at a 16-byte boundary.
__device__ __forceinline__ void prefetch_l2(const void* at, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}

// 32 bytes, a whole sector, at a 32-byte boundary.
__device__ __forceinline__ void store8(float* at, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

struct SharedScore {
  using Params = SharedParams;
  static constexpr bool kMod = false;
};

template <int D, int STAGES>
__global__ void __launch_bounds__(SharedCfg<D, STAGES>::kThreads, 1)
    shared_decode_kernel(const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map,
                         const __grid_constant__ CUtensorMap q_map, const SharedParams p) {
  using C = SharedCfg<D, STAGES>;
  const int G = p.group;
  const int T = p.tile;  // rows of a tile
  const int Gp = (G + 1) & ~1;  // heads of a row's partial
  const long long own_part = shared_own_part(p);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;

  extern __shared__ unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* q_smem = base;
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
  uint64_t* q_full = seg_free + C::kSegs;  // [block % 2] its Q landed
  uint64_t* q_free = q_full + 2;           // [Q tile] its block's S products done
  uint64_t* fin = q_free + C::kTiles;      // [issuer] all its products done
  __shared__ SharedSeg segs[C::kSegs];
  __shared__ volatile int abort_flag;
  __shared__ uint32_t tmem_slot;
  __shared__ long long warp_sum[C::kThreads / 32];
  __shared__ long long start_rem, block_weight;
  __shared__ int start_item;
  // tile rows of the pages by page % 64 (K is never that far ahead of V: a page's
  // consumer needs both, and eight or so are at work), how many copies are issued, and
  // of how many K copies in all (-1: not known yet)
  __shared__ int y_ring[64];
  __shared__ int k_issued, v_issued, k_total;

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
    }
    for (int i = 0; i < C::kTiles; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_free[i], 1);
    }
    mbar_init(&fin[0], 1);
    mbar_init(&fin[1], 1);
    mbar_init_fence();
    abort_flag = 0;
    k_issued = v_issued = 0;
    k_total = -1;
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
  long long u0, u1;  // this CTA's range of weights
  // pages, first page, first row, end or position of each item, where every thread has one
  int4* list = reinterpret_cast<int4*>(base + C::kBarOff) - C::kThreads;  // (the last stage's end)
  {
    int* g_start = reinterpret_cast<int*>(stages);  // [S + 1], then pages [S]
    int* g_pages = g_start + S + 1;
    // thread i sums a run of the list
    const int run = (items + C::kThreads - 1) / C::kThreads;
    const int i0 = min(tid * run, items), i1 = min(i0 + run, items);
    const int n_mine = run == 1 && tid >= S && tid < items ? p.positions[tid - S] : -1;
    bool unsorted = false;
    for (int g = tid; S > 0 && g <= S; g += C::kThreads) {
      const int s = p.starts[g], before = g > 0 ? p.starts[g - 1] : 0;
      unsorted |= s < before || s > p.rows;
      g_start[g] = s;
      if (g < S) g_pages[g] = p.pages[g];
    }
    unsorted = __syncthreads_or(unsorted);  // every row is bad then
    // some of the groups' pages on their way to L2 while the cut is made: whose they are
    // shows only then, and HBM would wait for it (16 groups of 4 rows
    // 53.8 -> 53.1 us)
    int ahead_id = -1;
    const int ahead = cta / max(S, 1) * C::kAhead + lane;  // a (page, kv head) of group cta % S
    if (warp == C::kVWarp && lane < C::kAhead && S > 0 && !unsorted) {
      const int g = cta % S, pages = g_pages[g];
      if (g_start[g] < g_start[g + 1] && pages <= p.maxp && ahead / p.hkv < pages)
        ahead_id = p.table[(size_t)g_start[g] * p.maxp + ahead / p.hkv];
    }
    auto item_at = [&](int i, int& g) {
      if (i < S) {
        g = i;
        return shared_group(p, g_start[i], g_start[i + 1], g_pages[i]);
      }
      g = S > 0 ? shared_find(g_start, S, i - S) : -1;
      return shared_row(p, run == 1 ? n_mine : p.positions[i - S],
                        g >= 0 && g < S ? g_pages[g] : 0);
    };
    long long sum = 0, blocks_sum = 0;  // of these items, and of those that are blocks
    int g_mine = -1;
    bool bad_mine = unsorted;
    if (!unsorted)
      for (int i = i0; i < i1; ++i) {
        const SharedItem it = item_at(i, g_mine);
        if (i == S) blocks_sum = sum;
        sum += it.weight(p.hkv);
        bad_mine = it.bad;
        if (run == 1)  // the producer's list
          list[i] = i < S ? make_int4(it.pages, 0, g_start[i], g_start[i + 1])
                          : make_int4(it.pages, it.first, i - S, it.n);
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
    if (i0 <= S && S < i1) block_weight = at + blocks_sum;  // (there is a row)
    __syncthreads();
    if (ahead_id >= 0 && ahead_id < p.num_pages) {
      const size_t at_page =
          tile_first_row(p.layout, ahead_id, ahead % p.hkv, p.hkv, p.num_pages, 1) * (size_t)D;
      prefetch_l2(p.k_pool + at_page, C::kTileBytes);
      prefetch_l2(p.v_pool + at_page, C::kTileBytes);
    }
    const SharedCut cut = shared_cut(block_weight, total, ctas);
    u0 = cut.begin(cta, total);
    u1 = cut.begin(cta + 1, total);
    // the last CTA, whose range may be short, leaves the combine what it needs
    const bool records = cta == ctas - 1;
    if (records && tid == 0) {
      *p.cut = cut;
      if (unsorted) record_error(p.err, PGD_EDEVICE_BOUNDS);
    }
    auto each_item = [&](auto f) {  // f(item, group, offset, weight, bad) of this thread's items
      long long off = at;
      for (int i = i0; i < i1; ++i) {
        int g = g_mine;
        long long weight = sum;
        bool bad = bad_mine;
        if (run > 1 && !unsorted) {
          const SharedItem it = item_at(i, g);
          weight = it.weight(p.hkv);
          bad = it.bad;
        }
        f(i, g, off, weight, bad);
        off += weight;
      }
    };
    if (u0 < u1 && at <= u0 && u0 < at + sum)
      each_item([&](int i, int, long long off, long long weight, bool) {
        if (off <= u0 && u0 < off + weight) {
          start_item = i;
          start_rem = u0 - off;
        }
      });
    if (records) {
      long long* g_off = reinterpret_cast<long long*>(stages + ((2 * S + 1) * 4 + 7) / 8 * 8);
      each_item([&](int i, int, long long off, long long weight, bool bad) {
        if (i < S) g_off[i] = weight > 0 ? off : -1;
        if (bad) record_error(p.err, PGD_EDEVICE_BOUNDS);
      });
      __syncthreads();
      each_item([&](int i, int g, long long off, long long weight, bool) {
        if (i < S) return;
        const bool grouped = g >= 0 && g < S && !unsorted;
        SharedRecord r;
        r.own = weight > 0 ? off : -1;
        r.group = grouped ? g_off[g] : -1;
        r.start = grouped ? g_start[g] : 0;
        r.end = grouped ? g_start[g + 1] : 0;
        r.shared = grouped ? g_pages[g] : 0;
        r.n = run == 1 ? n_mine : p.positions[i - S];
        const int4* words = reinterpret_cast<const int4*>(&r);
        int4* to = reinterpret_cast<int4*>(p.records + (i - S));
        to[0] = words[0];
        to[1] = words[1];
      });
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
    }
    auto load_tile = [&](unsigned char* dst, const CUtensorMap* map, int y, uint64_t* bar) {
      if constexpr (D == 128)
        tma_load_3d(dst, map, 0, y, 0, bar);
      else
        tma_load_2d(dst, map, 0, y, bar);
    };
    int kn = 0, ks = 0;       // K copies issued, the next one's stage
    uint32_t kph = 1;         // parity of the stage's last round (the first waits for none)
    int seq = 0;              // segments laid out
    int blocks_seen = 0;      // blocks' segments
    int q_next = 0;           // Q tile of the next one-tile block
    int q_used0 = 0, q_used1 = 0;  // segments that took each Q tile
    int tile_next = 0;        // tile of the next one-tile block
    bool ok = true;
    const bool page_major = p.layout == PGD_PAGE_MAJOR;
    const int y_page = (page_major ? p.hkv : 1) * kPage;     // tile rows from page to page
    const int y_head = (page_major ? 1 : p.num_pages) * kPage;  // and from head to head
    // a row's own pages: the first 32 and whether all are in the pool, kept from
    // head to head, and the next row's first 32, loaded meanwhile
    int row_seen = -1, row_id = 0, next_row = -1, next_id = 0;
    bool row_bad = false;
    auto in_pool = [&](int id) { return id >= 0 && id < p.num_pages; };
    // Descriptors of `heads` (at most kSegs) kv heads from kvh on, one a lane, their
    // partials part_step apart.
    auto describe = [&](int heads, long long part, int part_step, int pages, int row0, int kvh,
                        int rows, int what) -> bool {
      const int s = seq + lane, d = s % C::kSegs;
      const bool writes = lane < heads;
      if (!all_ok(!writes || s < C::kSegs || wait(&seg_free[d], (s / C::kSegs - 1) & 1)))
        return false;
      if (writes) {
        const long long at = part + lane * part_step;
        int4* to = reinterpret_cast<int4*>(&segs[d]);
        to[0] = make_int4((int)at, (int)(at >> 32), pages, row0);
        to[1] = make_int4(kvh + lane, rows, what, 0);
        mbar_arrive(&seg_ready[d]);
      }
      seq += heads;
      return true;
    };
    auto copy_k = [&](int y) -> bool {
      if (kn >= STAGES && !all_ok(wait(&k_empty[ks], kph))) return false;
      if (elect_lane()) {
        mbar_arrive_expect_tx(&k_full[ks], C::kTileBytes);
        load_tile(stages + ks * C::kStageBytes, &k_map, y, &k_full[ks]);
        y_ring[kn & 63] = y;
        shared_store_count(&k_issued, kn + 1);
      }
      ++kn;
      if (++ks == STAGES) {
        ks = 0;
        kph ^= 1;
      }
      return true;
    };
    // Pages 0 .. count - 1 at trow, 32 ids at a time (the first 32 in `id`), one a lane.
    auto copy_pages = [&](const int32_t* trow, int id, int count, int y0) -> bool {
      for (int k = 0;;) {
        const int n = min(count - k, 32);
        const int ahead = k + 32 + lane < count ? trow[k + 32 + lane] : 0;
        for (int j = 0; j < n; ++j)
          if (!copy_k(__shfl_sync(0xffffffffu, id, j) * y_page + y0)) return false;
        k += n;
        if (k >= count) return true;
        id = ahead;
      }
    };
    // Pages pg0 .. pg1 - 1 of a block's `pages` shared ones, by the table row of its first
    // row that is neither inactive nor in error (those may hold others, or none).
    auto block_segment = [&](int row0, int rows, int kvh, int pages, int pg0, int pg1) -> bool {
      auto holds = [&](int row) { return shared_row(p, p.positions[row], pages).pages > 0; };
      const int32_t* trow = p.table + (size_t)row0 * p.maxp + pg0;
      int count = pg1 - pg0, id = lane < count ? trow[lane] : 0;
      if (!holds(row0)) {
        int at = 0;
        unsigned held = 0;
        for (; at < rows && held == 0; at += 32)
          held = __ballot_sync(0xffffffffu, at + lane < rows && holds(row0 + at + lane));
        if (held == 0) count = 0;  // none: nothing is read
        trow += (size_t)(held ? at - 32 + __ffs(held) - 1 : 0) * p.maxp;
        id = lane < count ? trow[lane] : 0;
      }
      bool bad = lane < count && !in_pool(id);
      for (int k = lane + 32; k < count; k += 32) bad |= !in_pool(trow[k]);
      bad = __any_sync(0xffffffffu, bad);
      if (bad && lane == 0) record_error(p.err, PGD_EDEVICE_BOUNDS);
      if (bad) count = 0;
      const int tiles = rows > T ? 2 : 1;
      const int q_tile = tiles == 2 ? 0 : q_next;
      // (partials of the items before: one a lane)
      if (!describe(1, 256ll * cta + (long long)row0 * p.hq + (long long)kvh * rows * G, 0,
                    count, row0, kvh, rows,
                    SharedSeg::fields(false, tiles, tiles == 2 ? 0 : tile_next, q_tile, kPage - 1)))
        return false;
      if (count == 0) return true;
      if (tiles == 1) tile_next ^= 1;
      // Q, once the products that read its tiles are done
      if (q_tile == 0) {
        if (q_used0 > 0 && !all_ok(wait(&q_free[0], (q_used0 - 1) & 1))) return false;
        ++q_used0;
      }
      if (q_tile + tiles == 2) {
        if (q_used1 > 0 && !all_ok(wait(&q_free[1], (q_used1 - 1) & 1))) return false;
        ++q_used1;
      }
      q_next = tiles == 2 ? 0 : q_next ^ 1;
      if (lane == 0) {
        uint64_t* full = &q_full[blocks_seen & 1];
        mbar_arrive_expect_tx(full, tiles * C::kBoxes * T * G * 128);
        for (int t = 0; t < tiles; ++t)
          for (int bx = 0; bx < C::kBoxes; ++bx)
            tma_load_3d(q_smem + (q_tile + t) * C::kQTileBytes + bx * C::kQBoxBytes, &q_map,
                        64 * bx, kvh * G, row0 + t * T, full);
      }
      ++blocks_seen;
      return copy_pages(trow, id, count, kvh * y_head);
    };
    // Pages pg0 .. pg1 - 1 of a row's own, `pages` from place `first` of its table row on, for
    // `heads` kv heads from kvh on.  (All heads' descriptors at once: head by head, a row of
    // one page took the producer 0.8 us a head.)
    auto row_segments = [&](int heads, int row, int kvh, int first, int pages, int n, int pg0,
                            int pg1) -> bool {
      const int32_t* trow = p.table + (size_t)row * p.maxp + first;
      if (row_seen != row) {
        row_seen = row;
        row_id = next_row == row ? next_id : lane < pages ? trow[lane] : 0;
        bool bad = lane < pages && !in_pool(row_id);
        for (int k = lane + 32; k < pages; k += 32) bad |= !in_pool(trow[k]);
        row_bad = __any_sync(0xffffffffu, bad);
      }
      const int count = pg1 - pg0;
      const bool last = pg1 == pages;
      // (partials of the items before: four a head)
      if (!describe(heads, 256ll * cta + own_part + 4ll * Gp * ((long long)row * p.hkv + kvh),
                    4 * Gp, row_bad ? 0 : count, row, kvh, 1,
                    SharedSeg::fields(true, 1, 0, 0, last ? n % kPage : kPage - 1)))
        return false;
      if (row_bad) {
        if (lane == 0) record_error(p.err, PGD_EDEVICE_BOUNDS);
        return true;
      }
      if (p.k_new != nullptr && last) {
        // The step's keys and values at position n, ahead of the copies of their page.  (They
        // hold up the producer: a step of 16 groups of 4 rows takes 74 us, of 131 rows of 64
        // heads 75, of 256 rows over 32768 shared positions 274, where kv_append_paged and
        // the attention take 55, 66 and 188.)
        constexpr int kWords = D / 8;
        const size_t dst = ((size_t)trow[pages - 1] * y_page + kvh * y_head + n % kPage) * D;
        const size_t src = ((size_t)row * p.hkv + kvh) * D;
        for (int k = lane; k < 2 * kWords * heads; k += 32) {
          const int c = k % kWords, h = k / (2 * kWords);
          const bool is_v = k / kWords % 2;
          *reinterpret_cast<uint4*>((is_v ? p.v_pool : p.k_pool) + dst + (size_t)h * y_head * D +
                                    8 * c) =
              *reinterpret_cast<const uint4*>((is_v ? p.v_new : p.k_new) + src + (size_t)h * D +
                                              8 * c);
        }
        asm volatile("fence.proxy.async.global;" ::: "memory");
        __syncwarp();
      }
      const int id = pg0 == 0 ? row_id : lane < count ? trow[pg0 + lane] : 0;
      for (int h = kvh; h < kvh + heads; ++h)
        if (!copy_pages(trow + pg0, id, count, h * y_head)) return false;
      return true;
    };
    // walk the list from the start item on, 32 entries at a time, one a lane
    constexpr int kMaxHeads = C::kSegs / 2;  // described ahead of their copies
    const int T2 = 2 * T;
    long long u = u0, rem = start_item >= 0 ? start_rem : 0;
    int win = -32;
    int l_first = 0, l_pages = 0, l_n = 0, l_row = 0, l_end = 0;
    for (int item = start_item; ok && u < u1 && item >= 0 && item < items; ++item, rem = 0) {
      if (item >= win + 32) {
        // (the first time round the last stage still holds the list)
        const bool listed = win < 0 && items <= C::kThreads;
        win = item;
        const int i = win + lane;
        l_pages = 0;
        if (i < items && listed) {
          const int4 it = list[i];
          l_pages = it.x;
          l_first = it.y;
          l_row = it.z;
          l_n = l_end = it.w;
        } else if (i < items) {
          SharedItem it;
          if (i < S) {
            l_row = p.starts[i];
            l_end = p.starts[i + 1];
            it = shared_group(p, l_row, l_end, p.pages[i]);
          } else {
            l_row = i - S;
            const int g = S > 0 ? shared_find(p.starts, S, l_row) : -1;
            it = shared_row(p, p.positions[l_row], g >= 0 && g < S ? p.pages[g] : 0);
          }
          l_first = it.first;
          l_pages = it.pages;
          l_n = it.n;
        }
        if (i >= S) l_end = l_row + 1;
        if (listed) fence_proxy_async_shared();
        __syncwarp();
      }
      const int j = item - win;
      const bool own = item >= S;
      const int pages = __shfl_sync(0xffffffffu, l_pages, j);
      if (pages == 0) continue;
      const int first = __shfl_sync(0xffffffffu, l_first, j), n = __shfl_sync(0xffffffffu, l_n, j);
      const int s = __shfl_sync(0xffffffffu, l_row, j), e = __shfl_sync(0xffffffffu, l_end, j);
      const int unit = own ? kUnitOwn : e - s > T ? kUnitTwo : kUnitOne;
      const int fixed = own ? kFixedOwn : kFixedBlock;
      // the next row's page ids, needed once this row's heads are through
      int ahead_row = -1, ahead_id = 0;
      if (own && j < 31) {
        const int np = __shfl_sync(0xffffffffu, l_pages, j + 1);
        const int nf = __shfl_sync(0xffffffffu, l_first, j + 1);
        if (np > 0) {
          ahead_row = s + 1;
          if (lane < np) ahead_id = p.table[(size_t)(s + 1) * p.maxp + nf + lane];
        }
      }
      const long long per = fixed + (long long)pages * unit;  // of one (block, kv head)
      const int blocks = own ? 1 : shared_blocks(p, e - s);
      int bh = rem == 0 ? 0 : (int)shared_divide(rem, per);
      long long at = rem - bh * per;
      int blk = bh < p.hkv ? 0 : bh / p.hkv, kvh = bh - blk * p.hkv;
      for (; ok && u < u1 && blk < blocks; at = 0) {
        // the pages whose weight begins in [u, u1)
        int pg0 = 0, pg1 = pages;
        if (at > fixed) pg0 = shared_pages_before(at - fixed, unit);
        const long long left = u1 - u + at;
        if (left < per)
          pg1 = left > fixed ? min(pages, shared_pages_before(left - fixed, unit)) : 0;
        // whole rows' heads together
        int heads = 1;
        if (own && at == 0 && left >= 2 * per) {
          heads = min(p.hkv - kvh, kMaxHeads);
          if (left < heads * per) heads = (int)shared_divide(left, per);
        }
        u += heads * per - at;
        if (pg0 < pg1)
          ok = own ? row_segments(heads, s, kvh, first, pages, n, pg0, pg1)
                   : block_segment(s + blk * T2, min(T2, e - s - blk * T2), kvh, pages, pg0, pg1);
        kvh += heads;
        if (kvh == p.hkv) {
          kvh = 0;
          ++blk;
        }
      }
      next_row = ahead_row;
      next_id = ahead_id;
    }
    if (ok) {  // the end
      const int d = seq % C::kSegs;
      if ((seq < C::kSegs || all_ok(wait(&seg_free[d], (seq / C::kSegs - 1) & 1))) && lane == 0) {
        segs[d].what = 0;
        mbar_arrive(&seg_ready[d]);
      }
    }
    // drain: no copy may still be landing when the CTA exits
    if (lane == 0) {
      shared_store_count(&k_total, kn);
      for (int j = max(0, kn - STAGES); j < kn; ++j)
        mbar_wait_bounded(&k_full[j % STAGES], (j / STAGES) & 1, p.err);
      for (int j = max(0, blocks_seen - 2); j < blocks_seen; ++j)
        mbar_wait_bounded(&q_full[j & 1], (j / 2) & 1, p.err);
    }
  } else if (warp == C::kVWarp) {
    // ------------------------------------------------------------ V producer
    int vn = 0, vs = 0;  // copies issued, the next one's stage
    uint32_t vph = 1;
    bool ok = true;
    while (ok) {
      int issued = lane == 0 ? shared_wait_count(&k_issued, &k_total, vn, p.err, &abort_flag) : 0;
      issued = __shfl_sync(0xffffffffu, issued, 0);
      if (issued <= vn) break;  // the end
      for (; vn < issued; ++vn) {
        if (vn >= STAGES && !all_ok(wait(&v_empty[vs], vph))) {
          ok = false;
          break;
        }
        const int y = y_ring[vn & 63];
        if (elect_lane()) {
          mbar_arrive_expect_tx(&v_full[vs], C::kTileBytes);
          unsigned char* slot = stages + vs * C::kStageBytes + C::kTileBytes;
          if constexpr (D == 128)
            tma_load_3d(slot, &v_map, 0, y, 0, &v_full[vs]);
          else
            tma_load_2d(slot, &v_map, 0, y, &v_full[vs]);
          shared_store_count(&v_issued, vn + 1);
        }
        if (++vs == STAGES) {
          vs = 0;
          vph ^= 1;
        }
      }
    }
    if (lane == 0)
      for (int j = max(0, vn - STAGES); j < vn; ++j)
        mbar_wait_bounded(&v_full[j % STAGES], (j / STAGES) & 1, p.err);
  } else if (warp == C::kSWarp) {
    // ------------------------------------------------------------ S issuer
    // (It and the P V issuer are on every tile's path: both wait as whole warps and
    // issue under elect_lane, which leaves the products' operands in uniform registers;
    // one thread each took 240 us for 256 rows over 32768 shared positions.)
    int i = 0, st = 0;     // pages, and the next one's stage
    uint32_t ph = 0;       // its parity
    int ip[2] = {0, 0};    // pages of each tile
    int blocks = 0;
    bool issued = false, ok = true;
    auto skip = [&](int pages) {
      i += pages;
      st = i % STAGES;
      ph = (i / STAGES) & 1;
    };
    for (int seq = 0; ok; ++seq) {
      const int d = seq % C::kSegs;
      if (!all_ok(wait(&seg_ready[d], (seq / C::kSegs) & 1))) break;
      const SharedSeg sg = segs[d];
      if (sg.what == 0) break;
      if (sg.own() || sg.pages == 0) {
        skip(sg.pages);
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_free[d]);
        continue;
      }
      if (!all_ok(wait(&q_full[blocks & 1], (blocks / 2) & 1))) break;
      ++blocks;
      const int t0 = sg.tile(), t1 = t0 + sg.tiles();
      const uint64_t q0 =
          umma_desc_sw128(smem_addr(q_smem) + (sg.q_tile() - t0) * C::kQTileBytes, 16, 1024);
      const uint64_t k0 = umma_desc_sw128(smem_addr(stages), 16, 1024);
      for (int k = 0; k < sg.pages && ok; ++k) {
        if (!all_ok(wait(&k_full[st], ph))) {
          ok = false;
          break;
        }
        const uint64_t kd = umma_desc_advance(k0, st * C::kStageBytes);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t < t0 || t >= t1) continue;
          const int n = ip[t], tb = 2 * t + (n & 1);
          // the buffer holds P of the tile's page n - 2 until P V has read it
          if (n >= 2 && !all_ok(wait(&o_done[tb], (n / 2 - 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t qd = umma_desc_advance(q0, t * C::kQTileBytes);
          if (elect_lane()) {
            // (the last tile's P V, whose commit covers the other's: that page's V slot is
            // free; the last two pages' the softmax warps free)
            if (k >= 2 && t == t1 - 1)
              mbar_arrive(&v_empty[st >= 2 ? st - 2 : st + STAGES - 2]);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_bf16(tmem + C::kSCol + tb * kPage,
                        umma_desc_advance(qd, (kk >> 2) * C::kQBoxBytes + (kk & 3) * 32),
                        umma_desc_advance(kd, (kk >> 2) * kBoxBytes + (kk & 3) * 32), C::kIdescS,
                        kk > 0);
            umma_commit(&s_full[tb]);
          }
          ++ip[t];
          issued = true;
        }
        if (!ok) break;
        ++i;
        if (++st == STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
      if (elect_lane()) {
        for (int t = 0; t < sg.tiles(); ++t) umma_commit(&q_free[sg.q_tile() + t]);
        mbar_arrive(&seg_free[d]);
      }
    }
    if (issued && elect_lane()) {  // TMEM is freed once every product is done
      umma_commit(&fin[0]);
      mbar_wait_bounded(&fin[0], 0, p.err);
    }
  } else if (warp == C::kPvWarp) {
    // ------------------------------------------------------------ P V issuer
    int i = 0, st = 0;
    uint32_t ph = 0;
    int ip[2] = {0, 0};
    bool issued = false, ok = true;
    for (int seq = 0; ok; ++seq) {
      const int d = seq % C::kSegs;
      if (!all_ok(wait(&seg_ready[d], (seq / C::kSegs) & 1))) break;
      const SharedSeg sg = segs[d];
      if (sg.what == 0) break;
      if (sg.own()) {
        i += sg.pages;
        st = i % STAGES;
        ph = (i / STAGES) & 1;
      }
      const int t0 = sg.tile(), t1 = t0 + sg.tiles(), pages = sg.own() ? 0 : sg.pages;
      const uint64_t v0 =
          umma_desc_sw128(smem_addr(stages) + C::kTileBytes, kBoxBytes, 1024);
      for (int k = 0; k < pages && ok; ++k) {
        if (!all_ok(wait(&v_full[st], ph))) {
          ok = false;
          break;
        }
        const uint64_t vd = umma_desc_advance(v0, st * C::kStageBytes);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t < t0 || t >= t1) continue;
          const int n = ip[t], tb = 2 * t + (n & 1);
          // (P of a segment's first page comes after its tile's last O was read)
          if (!all_ok(wait(&p_full[tb], (n / 2) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t pb = tmem + C::kSCol + tb * kPage;
          // keys 16 kk ..: P's head in columns 8 kk, its residual 32 further
          if (elect_lane()) {
            // (the last tile's S was read, whose commit covers the other's: K's slot is free)
            if (t == t1 - 1) mbar_arrive(&k_empty[st]);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_bf16_tmem_a(tmem + t * D, pb + 8 * kk,
                               umma_desc_advance(vd, (kk & 3) * 2048), C::kIdescPV,
                               k > 0 || kk > 0);
            umma_commit(&o_done[tb]);
          }
          ++ip[t];
          issued = true;
        }
        if (!ok) break;
        ++i;
        if (++st == STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&seg_free[d]);
    }
    if (issued && elect_lane()) {
      umma_commit(&fin[1]);
      mbar_wait_bounded(&fin[1], 0, p.err);
    }
  } else if (warp < C::kSoftmaxWarps) {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2, m = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float c = p.q_scale_log2;
    const float cc = c > 0.f ? c : 1.f;  // folded into the exponent's FMA if positive
    int n = 0;   // pages of this tile
    int i = 0;   // pages
    int turn = 0;  // the next segment's first warp, % 8
    bool ok = true;
    for (int seq = 0; ok; ++seq) {
      const int d = seq % C::kSegs;
      if (!all_ok(wait(&seg_ready[d], (seq / C::kSegs) & 1))) break;
      const SharedSeg sg = segs[d];
      if (sg.what == 0) break;
      const int pages = sg.pages;
      if (sg.own()) {
        // at most four of the warps a segment, the next ones the next: page k is warp
        // (turn + k % 4) % 8's, and partial k % 4
        const int k0 = (warp - turn) & 7;  // this warp's first page
        turn += min(pages, 4);
        if (k0 < min(pages, 4)) {
          MmaConsumer<D, SharedScore> cons;
          cons.init(p, sg.row0, sg.kvh * G, lane, nullptr);
          for (int k = k0; k < pages; k += 4) {
            const int ik = i + k, st = ik % STAGES;
            const uint32_t ph = (ik / STAGES) & 1;
            if (!all_ok(shared_wait_count(&k_issued, nullptr, ik, p.err, &abort_flag) > ik) ||
                !all_ok(wait(&k_full[st], ph))) {
              ok = false;
              break;
            }
            unsigned char* kt = stages + st * C::kStageBytes;
            auto k_done = [&]() {  // K's slot is free while the weights are computed
              __syncwarp();
              if (lane == 0) mbar_arrive(&k_empty[st]);
            };
            const int rhi = k == pages - 1 ? sg.rhi() : kPage - 1;
            auto v_ready = [&]() {
              ok = all_ok(shared_wait_count(&v_issued, nullptr, ik, p.err, &abort_flag) > ik) &&
                   all_ok(wait(&v_full[st], ph));
              // V rows past the last position may hold anything: zero weights need
              // zeros (eight lanes a row: lanes 128 bytes apart would meet at one bank)
              unsigned char* vt = kt + C::kTileBytes;
              for (int r = rhi + 1 + (lane >> 3); r < kPage; r += 4)
#pragma unroll
                for (int bx = 0; bx < C::kBoxes; ++bx)
                  *reinterpret_cast<uint4*>(vt + bx * kBoxBytes + r * 128 + (lane & 7) * 16) =
                      make_uint4(0u, 0u, 0u, 0u);
              __syncwarp();
            };
            if (cons.template page<4>(smem_addr(kt), kt + C::kTileBytes, 0, rhi, lane, k_done,
                                      v_ready))
              fence_proxy_async_shared();
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_empty[st]);
          }
          if (!ok) break;
          cons.finish();
          const long long part = sg.part + k0 * Gp;
          if (2 * cons.tig < Gp) {
            float* acc = p.part_acc + (part + 2 * cons.tig) * D + cons.gid;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[(e & 1) * D + 16 * mt + (e >> 1) * 8] = cons.o[mt][e];
            if (cons.gid == 0)
              *reinterpret_cast<float4*>(p.part_ml + 2 * (part + 2 * cons.tig)) =
                  make_float4(cons.m[0], cons.l[0], cons.m[1], cons.l[1]);
          }
        } else if (pages == 0 && warp == 0 && lane < Gp) {
          // not read: the row's output is zero
          p.part_ml[2 * (sg.part + lane)] = -INFINITY;
          p.part_ml[2 * (sg.part + lane) + 1] = -1.f;
        }
        i += pages;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_free[d]);
        continue;
      }
      const int t0 = sg.tile();
      const bool mine = t >= t0 && t < t0 + sg.tiles();
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
        if (t == t0 + sg.tiles() - 1 && (warp & 3) == 0 && lane == 0)
          for (int k = max(pages - 2, 0); k < pages; ++k) mbar_arrive(&v_empty[(i + k) % STAGES]);
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
              store8(arow + 16 * q, ov);
              store8(arow + 16 * q + 8, ov + 8);
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

// Joins the partials of a (row, query head): those over its group's pages, one a CTA of the
// range that they fell to, then those over its own, up to four a CTA.  Zeros for an
// inactive row (n < 0), for one that the cut found bad, and where a page was outside the
// pool (l < 0); NaN where a score was NaN (l is NaN, the maxima pass over it).  A warp each,
// a CTA the heads of a kv head.  Bound by latency: 0.9 us after the other kernel's end the
// row's record (0.6 us), from which the places of the partials are worked out (1.5, most of
// it instructions on their way to the SM), then 32 partials' (m, l), one a lane, and the
// first four partials' values load together (1.3), and four at a time from there (0.7 each;
// eight or sixteen: more registers and, what counts more for so short a kernel, more code;
// 16 groups of 4 rows 54 us in all, 56, 58).
template <int D>
__global__ void __launch_bounds__(256) shared_combine_kernel(const SharedParams p) {
  constexpr int kDims = D / 32, kBatch = 4;
  const int kvh = blockIdx.x, b = blockIdx.y, g_head = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group, Gp = (G + 1) & ~1, h = kvh * G + g_head;
  const float sink = p.sinks ? p.sinks[h] * kLog2e : -INFINITY;  // (an input of both kernels)
  pdl_wait();
  pdl_allow_dependents();
  const int4* words = reinterpret_cast<const int4*>(p.records + b);
  const int4 w0 = words[0], w1 = words[1];
  const SharedCut cut = *p.cut;
  SharedRecord r;
  *reinterpret_cast<int4*>(&r) = w0;
  *(reinterpret_cast<int4*>(&r) + 1) = w1;
  const long long own_off = r.own;
  const SharedItem group = shared_group(p, r.start, r.end, r.shared);
  const SharedItem own = shared_row(p, r.n, r.shared);
  uint16_t* out = p.out + ((size_t)b * p.hq + h) * D + lane * kDims;
  float res[kDims];
#pragma unroll
  for (int j = 0; j < kDims; ++j) res[j] = 0.f;
  if (own_off >= 0) {
    // the shared pages' partials
    long long at0 = 0;
    int count0 = 0;
    if (r.group >= 0) {
      const int block = 2 * p.tile, blk = shared_block_of(p, b - r.start);
      const int row0 = r.start + blk * block;
      const int rows = min(block, r.end - row0);
      const long long first =
          r.group + ((long long)blk * p.hkv + kvh) * group.pair() + group.fixed;
      const int c0 = cut.block_cta(first);
      count0 = cut.block_cta(first + (long long)(group.pages - 1) * group.unit) - c0 + 1;
      at0 = 256ll * c0 + (long long)row0 * p.hq + (long long)kvh * rows * G + (b - row0) * G +
            g_head;
    }
    // its own pages': range i of a CTA has one for each page, at most four
    const long long first = own_off + kvh * own.pair() + own.fixed;
    const int c0 = cut.row_cta(first);
    const int ranges = cut.row_cta(first + (long long)(own.pages - 1) * own.unit) - c0 + 1;
    const long long rest = cut.blocks + (c0 - cut.block_ctas + 1) * cut.row_range - first;
    const long long at1 = 256ll * c0 + shared_own_part(p) +
                          4ll * Gp * ((long long)b * p.hkv + kvh);
    // pages that start before the end of range i
    auto before = [&](int i) {
      return i + 1 >= ranges
                 ? own.pages
                 : shared_pages_before(rest + i * cut.row_range, own.unit);
    };
    int count = count0;
    for (int i = 0, pg = 0; i < ranges; ++i) {
      const int end = before(i);
      count += min(end - pg, 4);
      pg = end;
    }
    auto own_place = [&](int j) {  // j of the row's own partials
      long long at = at1;
      for (int i = 0, pg = 0; i + 1 < ranges; ++i) {
        const int end = before(i), some = min(end - pg, 4);
        if (j < some) break;
        j -= some;
        pg = end;
        at += 256;
      }
      return at + j * Gp;
    };
    auto place = [&](int i) {
      return i < count0 ? at0 + 256ll * i : own_place(i - count0) + g_head;
    };
    auto values = [&](int i, float* v) {
      using Vec = typename std::conditional<kDims == 2, float2, float4>::type;
      *reinterpret_cast<Vec*>(v) =
          *reinterpret_cast<const Vec*>(p.part_acc + place(i) * D + lane * kDims);
    };
    auto weight = [&](int i) {
      if (i >= count) return make_float2(-INFINITY, 0.f);
      return *reinterpret_cast<const float2*>(p.part_ml + 2 * place(i));
    };
    float2 ml = weight(lane);
    alignas(16) float v[kBatch][kDims];
    auto load = [&](int i0) {  // four partials' values
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i0 + k < count) values(i0 + k, v[k]);
    };
    load(0);
    float mx = sink;
    bool skipped = false, nan = false;
    for (int i0 = 0; i0 < count; i0 += 32) {
      const float2 w = i0 == 0 ? ml : weight(i0 + lane);
      mx = fmaxf(mx, warp_max(w.x));
      skipped |= __any_sync(0xffffffffu, w.y < 0.f);
      nan |= __any_sync(0xffffffffu, w.y != w.y);
    }
    const float ref = mx == -INFINITY ? 0.f : mx;
    float den = exp2_approx(sink - ref);
    for (int i0 = 0; i0 < count; i0 += 32) {
      if (i0 > 0) ml = weight(i0 + lane);
      const float f = exp2_approx(ml.x - ref);  // (past the end: 0)
      den += warp_sum(ml.y * f);
      const int some = min(32, count - i0);
      for (int k0 = 0; k0 < some; k0 += kBatch) {
        if (i0 + k0 > 0) load(i0 + k0);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const float fk = __shfl_sync(0xffffffffu, f, k0 + k);
          if (i0 + k0 + k < count)
#pragma unroll
            for (int j = 0; j < kDims; ++j) res[j] = fmaf(v[k][j], fk, res[j]);
        }
      }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int j = 0; j < kDims; ++j) res[j] = skipped ? 0.f : nan ? NAN : res[j] * inv;
  }
  if constexpr (kDims == 4)
    *reinterpret_cast<uint2*>(out) =
        make_uint2(pack_bf16x2(res[0], res[1]), pack_bf16x2(res[2], res[3]));
  else
    *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(res[0], res[1]);
}

template <int D, int STAGES>
cudaError_t launch_shared(const SharedParams& p, const CUtensorMap& k_map,
                          const CUtensorMap& v_map, const CUtensorMap& q_map, int ctas,
                          cudaStream_t stream) {
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
  // Clusters of two put neighbouring CTAs on the two SMs of a TPC: an SM that reads
  // rows' own pages (mma.sync) slows its neighbour's tcgen05 products, so both had better
  // do the same (256 rows over 32768 shared positions: 185 us, 226 without clusters).
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, k_map, v_map, q_map, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(shared_combine_kernel<D>, dim3(p.hkv, p.rows), dim3(32 * p.group), 0, stream,
                    p);
}

}  // namespace pgd
