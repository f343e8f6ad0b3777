// Pages that several table rows hold: rows forked, reordered, cut back and
// released over reference counts, pages copied, and the pool compacted.
#include <cooperative_groups.h>

#include <atomic>

#include "pgd_device.cuh"
#include "pgd_ext_internal.h"

namespace pgd {

namespace cg = cooperative_groups;

// Exclusive sum of v over the CTA's 1024 threads; `total` gets the sum.  `warps`:
// 33 words of shared memory, free again after the caller's next barrier.
__device__ __forceinline__ int block_scan(int v, int* warps, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int in = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) in += a;
  }
  if (lane == 31) warps[warp] = in;
  __syncthreads();
  if (warp == 0) {
    int a = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, a, o);
      if (lane >= o) a += x;
    }
    warps[lane] = a;
  }
  __syncthreads();
  total = warps[31];
  return in - v + (warp ? warps[warp - 1] : 0);
}

// The shared-memory opt-in is per device; set it once on each.
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<bool>* configured) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && configured[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64)
    configured[dev].store(true, std::memory_order_release);
  return e;
}

// One cluster of `ctas` CTAs of 1024 threads.
template <class Params>
cudaError_t launch_cluster(void (*kernel)(Params), int ctas, size_t smem, cudaStream_t stream,
                           const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(1024);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// ------------------------------------------------------------------ fork_rows

// One cluster; its CTAs share out the rows (a warp each) and meet at cluster
// barriers, since every step needs the counts that the one before left:
//   1  a parent of c >= 2 children: its pages' shares grow by c - 1
//   2  entries that no child takes over: their pages' shares fall by one, so
//      a page that nobody holds any more is left at -1
//   3  the first such entry (row-major) claims the page: min of -2^31 + entry
//   4  claims counted by row; meanwhile each row whose last page is in part use
//      leaves that page (one share less)
//   5  the claimed pages go to the list; a last page that all its holders left
//      (-1) is claimed by the lowest of them, which keeps it
//   6  the other rows take pages off the list, in row order
//   7  the rows are moved, a slab of columns at a time through shared memory
//      (a row may be its neighbour's parent and child at once)
// Shares in between stay above -2^30 (a row's claims and its leaving its last
// page count one each); claims of entries are below that, claims of last pages
// from there up, so that neither is taken for the other.
constexpr int kForkThreads = 1024;
constexpr int kForkClaim = INT32_MIN, kForkTail = INT32_MIN / 2;

struct ForkRow {
  int parent;  // -1: none
  int kept, pages, had;  // positions and pages of the row, pages of its parent
};

__device__ __forceinline__ int fork_length(const ForkParams& p, int r) {
  const int n = p.lengths[r];
  return n >= 0 && n <= p.width * kPage ? n : 0;  // (reported once, below)
}

__device__ __forceinline__ ForkRow fork_row(const ForkParams& p, int r) {
  ForkRow f;
  f.parent = p.parents[r];
  if (f.parent < 0 || f.parent >= p.rows) f.parent = -1;
  const int n = f.parent < 0 ? 0 : fork_length(p, f.parent);
  f.kept = n;
  if (p.keep) f.kept = min(n, max(p.keep[r], 0));
  f.pages = (f.kept + kPage - 1) / kPage;
  f.had = (n + kPage - 1) / kPage;
  return f;
}

__global__ void __launch_bounds__(kForkThreads) fork_rows_kernel(ForkParams p) {
  extern __shared__ int smem[];
  int* children = smem;            // [rows]
  int* least = children + p.rows;  // [rows] fewest pages that a child takes
  int* slab = least + p.rows;
  __shared__ int warps[33];
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), cta = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gwarp = cta * (kForkThreads / 32) + warp, gwarps = ctas * (kForkThreads / 32);
  const int gtid = cta * kForkThreads + tid, gthreads = ctas * kForkThreads;
  auto in_pool = [&](int page) { return page >= 0 && page < p.num_pages; };
  auto report = [&]() { record_error(p.err, PGD_EDEVICE_BOUNDS); };

  for (int r = tid; r < p.rows; r += kForkThreads) {
    children[r] = 0;
    least[r] = INT32_MAX;
  }
  pdl_wait();
  pdl_allow_dependents();
  const int head0 = p.free_head ? *p.free_head : 0;
  const bool bad_head = head0 < 0 || head0 > p.num_free;
  if (bad_head && gtid == 0) report();
  __syncthreads();
  for (int r = tid; r < p.rows; r += kForkThreads) {
    const ForkRow f = fork_row(p, r);
    if (f.parent >= 0) {
      atomicAdd(&children[f.parent], 1);
      atomicMin(&least[f.parent], f.pages);
    }
    if (cta == 0) {
      const int n = p.lengths[r], q = p.parents[r];
      if (n < 0 || n > p.width * kPage || q < -1 || q >= p.rows) report();
    }
  }
  __syncthreads();
  // old row i loses entries lo .. hi - 1 (some child, if any, takes fewer pages)
  auto dropped = [&](int i, int& lo, int& hi) {
    hi = (fork_length(p, i) + kPage - 1) / kPage;
    lo = children[i] == 0 ? 0 : min(least[i], hi);
  };

  // 1
  for (int i = gwarp; i < p.rows; i += gwarps) {
    const int more = children[i] - 1;
    if (more < 1) continue;
    const int had = (fork_length(p, i) + kPage - 1) / kPage;
    for (int e = lane; e < had; e += 32) {
      const int page = p.table[(size_t)i * p.width + e];
      if (in_pool(page)) atomicAdd(&p.shares[page], more);
      else report();
    }
  }
  cluster.sync();
  // 2
  for (int i = gwarp; i < p.rows; i += gwarps) {
    if (children[i] == 0) {
      const int had = (fork_length(p, i) + kPage - 1) / kPage;
      for (int e = lane; e < had; e += 32) {
        const int page = p.table[(size_t)i * p.width + e];
        if (in_pool(page)) atomicSub(&p.shares[page], 1);
        else report();
      }
    }
    const ForkRow f = fork_row(p, i);
    for (int e = f.pages + lane; e < f.had; e += 32) {
      const int page = p.table[(size_t)f.parent * p.width + e];
      if (in_pool(page)) atomicSub(&p.shares[page], 1);
      else report();
    }
  }
  cluster.sync();
  // 3
  for (int i = gwarp; i < p.rows; i += gwarps) {
    int lo, hi;
    dropped(i, lo, hi);
    for (int e = lo + lane; e < hi; e += 32) {
      const int page = p.table[(size_t)i * p.width + e];
      if (!in_pool(page)) continue;
      const int held = __ldcg(&p.shares[page]);
      if (held < 0) {
        if (held < -1 && held > kForkTail) report();  // given back more often than held
        atomicMin(&p.shares[page], kForkClaim + (int)((size_t)i * p.width + e));
      }
    }
  }
  cluster.sync();
  // 4: the claims of a row are counted in its place of `sources`
  auto claimed = [&](int i, int e, int& page) {
    page = p.table[(size_t)i * p.width + e];
    return in_pool(page) &&
           __ldcg(&p.shares[page]) == kForkClaim + (int)((size_t)i * p.width + e);
  };
  for (int i = gwarp; i < p.rows; i += gwarps) {
    int lo, hi, n = 0, page;
    dropped(i, lo, hi);
    for (int e = lo + lane; e < hi; e += 32) n += claimed(i, e, page);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) p.sources[i] = n;
  }
  auto tail_page = [&](const ForkRow& f) {  // -1: the last page is full, or there is none
    return f.kept % kPage ? p.table[(size_t)f.parent * p.width + f.pages - 1] : -1;
  };
  for (int r = gtid; r < p.rows; r += gthreads) {
    const int page = tail_page(fork_row(p, r));
    if (in_pool(page)) atomicSub(&p.shares[page], 1);
  }
  cluster.sync();
  // 5
  int freed = 0;  // of all rows
  for (int r0 = 0; r0 < p.rows; r0 += kForkThreads) {
    const int r = r0 + tid;
    int total;
    const int at = block_scan(r < p.rows ? __ldcg(&p.sources[r]) : 0, warps, total);
    if (r < p.rows) slab[r] = freed + at;
    freed += total;
    __syncthreads();
  }
  const int head1 = bad_head ? head0 : max(head0 - freed, 0);  // the list after the pages freed
  if (!bad_head && head0 < freed && gtid == 0) report();      // (the list has no room for some)
  for (int i = gwarp; i < p.rows; i += gwarps) {
    int lo, hi;
    dropped(i, lo, hi);
    int at = slab[i];
    for (int e0 = lo; e0 < hi; e0 += 32) {
      int page = -1;
      const bool mine = e0 + lane < hi && claimed(i, e0 + lane, page);
      const unsigned who = __ballot_sync(0xffffffffu, mine);
      if (mine) {
        const int to = head0 - freed + at + __popc(who & ((1u << lane) - 1u));
        if (!bad_head && to >= 0) p.free_pages[to] = page;
        p.shares[page] = 0;
      }
      at += __popc(who);
    }
  }
  for (int r = gtid; r < p.rows; r += gthreads) {
    const int page = tail_page(fork_row(p, r));
    if (in_pool(page) && __ldcg(&p.shares[page]) < 0) atomicMin(&p.shares[page], kForkTail + r);
  }
  cluster.sync();
  // 6: every CTA ranks all rows; slab[r] is the page that row r's last entry gets
  // (-1: as it is; -2: none, the row loses its last page)
  int copies = 0;
  for (int r0 = 0; r0 < p.rows; r0 += kForkThreads) {
    const int r = r0 + tid;
    bool copy = false, lost = false;
    if (r < p.rows) {
      const ForkRow f = fork_row(p, r);
      const int page = tail_page(f);
      if (in_pool(page))
        copy = __ldcg(&p.shares[page]) != kForkTail + r;
      else
        lost = f.kept % kPage != 0;
    }
    int total;
    const int at = copies + block_scan(copy, warps, total);
    copies += total;
    if (r < p.rows) {
      int to = -1;
      if (copy) {
        to = -2;
        if (!bad_head && at < p.num_free - head1) {
          const int page = __ldcg(&p.free_pages[head1 + at]);
          if (in_pool(page)) to = page;
        }
      }
      if (lost) to = -2;
      if (to == -2 && cta == 0) report();
      slab[r] = to;
    }
    __syncthreads();
  }
  cluster.sync();
  // 7
  for (int r = gtid; r < p.rows; r += gthreads) {
    const ForkRow f = fork_row(p, r);
    const int page = tail_page(f), to = slab[r];
    p.new_lengths[r] = to == -2 ? f.kept - f.kept % kPage : f.kept;
    p.sources[r] = to >= 0 ? page : -1;
    p.targets[r] = to >= 0 ? to : -1;
    p.counts[r] = to >= 0 ? f.kept % kPage : 0;
    if (to == -1 && in_pool(page)) p.shares[page] = 0;  // the one that keeps it
  }
  if (gtid == 0)
    *p.free_head_out = bad_head ? head0 : min(head1 + copies, p.num_free);
  for (int r = tid; r < p.rows; r += kForkThreads) {
    const ForkRow f = fork_row(p, r);
    children[r] = f.parent;
    least[r] = 2 * f.pages + (f.kept % kPage != 0);  // pages, and whether the last is in part use
  }
  cluster.sync();  // the last entries of the parents were read above
  int* cells = slab + p.rows;
  const int columns = p.slab_columns;
  for (int c0 = cta * columns; c0 < p.width; c0 += ctas * columns) {
    const int n = min(columns, p.width - c0);
    for (int k = tid; k < p.rows * columns; k += kForkThreads) {
      const int r = k / columns, c = k % columns;
      if (c < n) cells[k] = p.table[(size_t)r * p.width + c0 + c];
    }
    __syncthreads();
    for (int k = tid; k < p.rows * columns; k += kForkThreads) {
      const int r = k / columns, c = k % columns, e = c0 + c;
      const int parent = children[r], pages = least[r] >> 1, to = slab[r];
      if (c >= n || e >= pages) continue;
      const bool tail = (least[r] & 1) != 0 && e == pages - 1;
      if (tail && to >= 0)
        p.table[(size_t)r * p.width + e] = to;
      else if (parent != r && !(tail && to == -2))
        p.table[(size_t)r * p.width + e] = cells[parent * columns + c];
    }
    __syncthreads();
  }
  cluster.sync();
}

cudaError_t launch_fork_rows(const ForkParams& params, cudaStream_t stream) {
  ForkParams p = params;
  // shared memory: three words a row and the slab
  const int limit = 200 * 1024;
  p.slab_columns = 8;
  while (p.slab_columns > 1 && (3 + p.slab_columns) * 4ll * p.rows > limit) p.slab_columns /= 2;
  const size_t smem = (size_t)(3 + p.slab_columns) * 4 * p.rows;
  static std::atomic<bool> configured[64];
  cudaError_t e = allow_smem(fork_rows_kernel, limit, configured);
  if (e != cudaSuccess) return e;
  const int64_t entries = (int64_t)p.rows * p.width;
  int ctas = 1;
  while (ctas < 8 && entries > 8192ll * ctas) ctas *= 2;
  return launch_cluster(fork_rows_kernel, ctas, smem, stream, p);
}

// ------------------------------------------------------------------ copy_pages

// A warp copies 4 KB pieces of (copy, pool, kv head) tiles, 8 x 16 bytes a lane
// in flight.  Bound by HBM for copies past L2.
constexpr int kCopyThreads = 256;
constexpr int kCopyPiece = 4096;

template <int D>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const CopyParams p) {
  pdl_wait();
  pdl_allow_dependents();
  constexpr int kPieces = kPage * D * 2 / kCopyPiece;  // of a tile
  const int lane = threadIdx.x & 31;
  const int64_t per_copy = (int64_t)p.pools * p.hkv * kPieces, all = per_copy * p.copies;
  const int64_t warps = (int64_t)gridDim.x * (kCopyThreads / 32);
  for (int64_t w = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); w < all;
       w += warps) {
    const int i = (int)(w / per_copy);
    int at = (int)(w % per_copy);
    const int piece = at % kPieces;
    at /= kPieces;
    const int h = at % p.hkv, pool = at / p.hkv;
    const int from = p.sources[i], to = p.targets[i];
    const int count = p.counts ? p.counts[i] : kPage;
    if (from < 0 || to < 0) continue;
    if (from >= p.num_pages || to >= p.num_pages || count < 0 || count > kPage) {
      if (lane == 0 && w % per_copy == 0) record_error(p.err, PGD_EDEVICE_BOUNDS);
      continue;
    }
    const int bytes = min(count * D * 2 - piece * kCopyPiece, kCopyPiece);
    if (bytes <= 0) continue;
    uint8_t* const base = static_cast<uint8_t*>(p.pool[pool]) + piece * kCopyPiece;
    const uint8_t* src = base + tile_first_row(p.layout, from, h, p.hkv, p.num_pages, 1) * D * 2;
    uint8_t* dst = base + tile_first_row(p.layout, to, h, p.hkv, p.num_pages, 1) * D * 2;
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k * 512 + lane * 16 < bytes)
        v[k] = *reinterpret_cast<const uint4*>(src + k * 512 + lane * 16);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k * 512 + lane * 16 < bytes)
        *reinterpret_cast<uint4*>(dst + k * 512 + lane * 16) = v[k];
  }
}

cudaError_t launch_copy_pages(const CopyParams& p, int head_dim, int sm_count,
                              cudaStream_t stream) {
  const int64_t pieces = (int64_t)p.copies * p.pools * p.hkv * (kPage * head_dim * 2 / kCopyPiece);
  int64_t ctas = (pieces + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  if (ctas > 8ll * sm_count) ctas = 8ll * sm_count;
  if (ctas < 1) return cudaSuccess;
  return head_dim == 64 ? launch_pdl(copy_pages_kernel<64>, dim3((unsigned)ctas),
                                     dim3(kCopyThreads), 0, stream, p)
                        : launch_pdl(copy_pages_kernel<128>, dim3((unsigned)ctas),
                                     dim3(kCopyThreads), 0, stream, p);
}

// ------------------------------------------------------------------ compact_pages

// Two bitmaps over the pool -- pages listed as free, pages held by a row -- made
// with atomics in the workspace; every CTA of the one cluster then sums their
// words' bits into prefixes in shared memory (a prefix per `step` words), from
// which the rank of any page among the free or the held is one look-up.
//   moves: the k-th held page from the top goes to the k-th free page from the
//   bottom while the latter is lower.  Without a limit that is all held pages
//   past the first `held` places of the free and held pages together.
//   free list: free pages left and vacated ones, each at its rank.
constexpr int kCompactThreads = 1024;

__global__ void __launch_bounds__(kCompactThreads) compact_pages_kernel(CompactParams p) {
  extern __shared__ int smem[];
  __shared__ int warps[33];
  __shared__ int unlimited;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), cta = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gwarp = cta * (kCompactThreads / 32) + warp, gwarps = ctas * (kCompactThreads / 32);
  const int gtid = cta * kCompactThreads + tid, gthreads = ctas * kCompactThreads;
  const int words = (p.num_pages + 31) / 32, blocks = (words + p.step - 1) / p.step;
  uint32_t* free_bits = p.bits;
  uint32_t* held_bits = p.bits + words;
  uint32_t* bad = p.bits + 2 * words;
  int* free_at = smem;  // [blocks + 1] free pages before the block's words
  int* held_at = smem + blocks + 1;
  pdl_wait();
  pdl_allow_dependents();
  for (int w = gtid; w < 2 * words + 1; w += gthreads) p.bits[w] = 0;
  cluster.sync();
  const int head = p.free_head ? *p.free_head : 0;
  const bool bad_head = head < 0 || head > p.num_free;
  if (bad_head && gtid == 0) atomicOr(bad, 1u);
  for (int k = (bad_head ? p.num_free : head) + gtid; k < p.num_free; k += gthreads) {
    const int page = p.free_pages[k];
    if (page < 0 || page >= p.num_pages)
      atomicOr(bad, 1u);
    else if (atomicOr(&free_bits[page >> 5], 1u << (page & 31)) >> (page & 31) & 1u)
      atomicOr(bad, 1u);  // listed twice
  }
  auto pages_of = [&](int r) {
    const int n = p.lengths[r];
    return n >= 0 && n <= p.width * kPage ? (n + kPage - 1) / kPage : -1;
  };
  for (int r = gwarp; r < p.rows; r += gwarps) {
    const int n = pages_of(r);
    if (n < 0 && lane == 0) atomicOr(bad, 1u);
    for (int e = lane; e < n; e += 32) {
      const int page = p.table[(size_t)r * p.width + e];
      if (page < 0 || page >= p.num_pages)
        atomicOr(bad, 1u);
      else
        atomicOr(&held_bits[page >> 5], 1u << (page & 31));
    }
  }
  cluster.sync();

  // prefixes: thread t sums a run of blocks
  const int run = (blocks + kCompactThreads - 1) / kCompactThreads;
  const int b0 = min(tid * run, blocks), b1 = min(b0 + run, blocks);
  int nf = 0, nh = 0;
  bool both = false;
  for (int w = b0 * p.step; w < min(b1 * p.step, words); ++w) {
    const uint32_t f = __ldcg(&free_bits[w]), h = __ldcg(&held_bits[w]);
    nf += __popc(f);
    nh += __popc(h);
    both |= (f & h) != 0;
  }
  int free_total, held_total;
  int f_at = block_scan(nf, warps, free_total);
  __syncthreads();
  int h_at = block_scan(nh, warps, held_total);
  for (int b = b0; b < b1; ++b) {
    free_at[b] = f_at;
    held_at[b] = h_at;
    for (int w = b * p.step; w < min((b + 1) * p.step, words); ++w) {
      f_at += __popc(__ldcg(&free_bits[w]));
      h_at += __popc(__ldcg(&held_bits[w]));
    }
  }
  if (tid == 0) unlimited = 0;
  const bool wrong = __syncthreads_or(both) || __ldcg(bad) != 0;
  // held pages of the union's places past the first held_total
  for (int b = b0; b < b1; ++b) {
    int f = free_at[b], h = held_at[b];
    for (int w = b * p.step; w < min((b + 1) * p.step, words); ++w) {
      const uint32_t fw = __ldcg(&free_bits[w]), hw = __ldcg(&held_bits[w]), all = fw | hw;
      const int n = __popc(all);
      if (f + h < held_total && f + h + n >= held_total) {
        uint32_t rest = all;  // the word that holds the last of these places
        int h_in = 0;
        for (int k = f + h; k < held_total; ++k) {
          const uint32_t low = rest & -rest;
          h_in += (hw & low) != 0;
          rest ^= low;
        }
        unlimited = held_total - (h + h_in);
      }
      f += __popc(fw);
      h += __popc(hw);
    }
  }
  __syncthreads();
  const int moves = wrong ? 0 : min(unlimited, p.max_moves);
  if (wrong && gtid == 0) record_error(p.err, PGD_EDEVICE_BOUNDS);
  const int kept = held_total - moves;  // held pages of a lower rank stay
  auto rank = [&](const uint32_t* bits, const int* at, int page) {
    const int w = page >> 5, b = w / p.step;
    int n = at[b];
    for (int k = b * p.step; k < w; ++k) n += __popc(bits[k]);
    return n + __popc(bits[w] & ((1u << (page & 31)) - 1u));
  };

  // the moves: sources from the top, targets from the bottom
  for (int w = gtid; w < words; w += gthreads) {
    for (uint32_t m = free_bits[w]; m; m &= m - 1) {
      const int page = 32 * w + __ffs(m) - 1, k = rank(free_bits, free_at, page);
      if (k < moves) p.targets[k] = page;
    }
    for (uint32_t m = held_bits[w]; m; m &= m - 1) {
      const int page = 32 * w + __ffs(m) - 1, k = held_total - 1 - rank(held_bits, held_at, page);
      if (k < moves) p.sources[k] = page;
    }
  }
  for (int k = moves + gtid; k < p.max_moves; k += gthreads) p.sources[k] = p.targets[k] = -1;
  cluster.sync();

  // table, shares, list
  for (int64_t k = gtid; k < (int64_t)p.rows * p.width; k += gthreads) {
    const int r = (int)(k / p.width), e = (int)(k % p.width);
    int page = p.table[k];
    if (moves > 0 && e < pages_of(r)) {
      const int h = rank(held_bits, held_at, page);
      if (h >= kept) page = __ldcg(&p.targets[held_total - 1 - h]);
    }
    p.new_table[k] = page;
  }
  auto bit = [](const uint32_t* bits, int page) { return bits[page >> 5] >> (page & 31) & 1u; };
  for (int page = gtid; page < p.num_pages; page += gthreads) {
    const bool f = bit(free_bits, page), h = bit(held_bits, page);
    if (wrong) {
      p.new_shares[page] = p.shares[page];
      continue;
    }
    const int fr = rank(free_bits, free_at, page), hr = rank(held_bits, held_at, page);
    const int vacated = max(hr - kept, 0);  // pages moved out below this one
    if (f && fr >= moves) {
      p.new_free[head + fr - moves + vacated] = page;
      p.new_shares[page] = p.shares[page];
    } else if (h && hr >= kept) {
      p.new_free[head + fr - moves + vacated] = page;
      const int to = __ldcg(&p.targets[held_total - 1 - hr]);
      const int n = p.shares[page];  // (this thread alone touches the two)
      p.new_shares[to] = n;
      p.new_shares[page] = 0;
    } else if (!f) {
      p.new_shares[page] = p.shares[page];
    }
  }
  for (int k = gtid; k < (wrong ? p.num_free : head); k += gthreads)
    p.new_free[k] = p.free_pages[k];
  // the end of the pages in use: the highest held page left, or the highest target
  if (gtid == 0) {
    int end = moves > 0 ? __ldcg(&p.targets[moves - 1]) + 1 : 0;
    if (kept > 0) {
      int lo = 0, hi = blocks;  // the last block with fewer than kept before it
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (held_at[mid] < kept)
          lo = mid;
        else
          hi = mid;
      }
      int n = held_at[lo];
      for (int w = lo * p.step; w < min((lo + 1) * p.step, words); ++w) {
        for (uint32_t m = held_bits[w]; m; m &= m - 1)
          if (++n == kept) end = max(end, 32 * w + __ffs(m));
      }
    }
    *p.end = end;
  }
}

cudaError_t launch_compact_pages(const CompactParams& params, cudaStream_t stream) {
  CompactParams p = params;
  const int words = (p.num_pages + 31) / 32;
  p.step = 1;
  while ((words + p.step - 1) / p.step > 24 * 1024) p.step *= 2;
  const size_t smem = ((size_t)(words + p.step - 1) / p.step + 1) * 8;
  static std::atomic<bool> configured[64];
  cudaError_t e = allow_smem(compact_pages_kernel, 200 * 1024, configured);
  if (e != cudaSuccess) return e;
  const int64_t work = (int64_t)p.rows * p.width + p.num_pages;
  int ctas = 1;
  while (ctas < 8 && work > 8192ll * ctas) ctas *= 2;
  return launch_cluster(compact_pages_kernel, ctas, smem, stream, p);
}

}  // namespace pgd
