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

// One CTA of 1024 threads for every SM, all resident at once (they meet).
template <class Params>
cudaError_t launch_grid(void (*kernel)(Params), int ctas, size_t smem, cudaStream_t stream,
                        const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(1024);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Where the CTAs of such a launch meet: a count of arrivals, zero before the launch.
struct GridBarrier {
  unsigned int* count;
  unsigned int* err;
  unsigned int ctas, arrivals = 0;

  __device__ void arrive() {
    __syncthreads();
    arrivals += ctas;
    if (threadIdx.x == 0) {
      __threadfence();
      atomicAdd(count, 1u);
    }
  }
  // Until all have arrived as often as this CTA; false after the limit of every wait.
  __device__ bool wait() const {
    bool late = false;
    if (threadIdx.x == 0) {
      const unsigned long long t0 = global_ns();
      for (unsigned int it = 1;; ++it) {
        unsigned int n;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(count) : "memory");
        if (n >= arrivals) break;
        if ((it & 63u) == 0u && global_ns() - t0 > kWaitLimitNs) {
          record_error(err, PGD_EDEVICE_TIMEOUT);
          late = true;
          break;
        }
      }
    }
    return !__syncthreads_or(late);
  }
  __device__ bool meet() {
    arrive();
    return wait();
  }
};

// f(r, e, entry) for the entries lo(r) .. hi(r) - 1 of a table's rows r, shared out
// over `warps` warps of which this is number `warp`, N rows at a time (rows N w ..
// N w + N - 1 of every round are warp w's) and 256 / N entries of each, so that a thread
// has eight loads in flight.
template <int N, class Lo, class Hi, class F>
__device__ __forceinline__ void each_entry_of(const int32_t* table, int rows, int width, int warp,
                                              int warps, Lo lo, Hi hi, F f) {
  const int lane = threadIdx.x & 31;
  constexpr int kEach = 8 / N;  // loads of a row
  for (int r0 = N * warp; r0 < rows; r0 += N * warps) {
    int from[N], to[N], most = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      from[k] = r0 + k < rows ? lo(r0 + k) : 0;
      to[k] = r0 + k < rows ? hi(r0 + k) : 0;
      most = max(most, to[k] - from[k]);
    }
    for (int e0 = lane; e0 - lane < most; e0 += 32 * kEach) {
      int page[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int e = from[k / kEach] + e0 + 32 * (k % kEach);
        if (e < to[k / kEach]) page[k] = table[(size_t)(r0 + k / kEach) * width + e];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int e = from[k / kEach] + e0 + 32 * (k % kEach);
        if (e < to[k / kEach]) f(r0 + k / kEach, e, page[k]);
      }
    }
  }
}

// A warp takes one row at a time where there is a warp for every row, else four.
__device__ __forceinline__ int rows_at_a_time(int rows, int warps) { return rows <= warps ? 1 : 4; }
template <class Lo, class Hi, class F>
__device__ __forceinline__ void each_table_entry(const int32_t* table, int rows, int width,
                                                 int warp, int warps, Lo lo, Hi hi, F f) {
  if (rows_at_a_time(rows, warps) == 1)
    each_entry_of<1>(table, rows, width, warp, warps, lo, hi, f);
  else
    each_entry_of<4>(table, rows, width, warp, warps, lo, hi, f);
}

// ------------------------------------------------------------------ fork_rows

// Six steps over rows and entries, each of which needs what all of the one before left:
//   1  the pages' shares: c - 1 more for the entries of a parent of c children, one
//      less for each that a child cuts off, so a page that nobody holds any more is
//      left at -1
//   2  the first entry of such a page that no child takes (row-major) claims it: min
//      of -2^31 + entry
//   3  claims counted by row; meanwhile each row whose last page is in part use
//      leaves that page (one share less)
//   4  the claimed pages go to the list; a last page that all its holders left
//      (-1) is claimed by the lowest of them, which keeps it
//   5  the other rows take pages off the list, in row order
//   6  the rows are moved, a slab of columns at a time through shared memory
//      (a row may be its neighbour's parent and child at once)
// Shares in between stay above -2^30 (a row's claims and its leaving its last
// page count one each); claims of entries are below that, claims of last pages
// from there up, so that neither is taken for the other.
// Bound by latency: each step is a table load and an atomic or load in L2 for every
// entry, eight a thread in flight.  Up to kForkClusterEntries entries (of the table, in use
// or not: lengths are on the device) one cluster does all steps and meets at cluster barriers (1-2 us a step), with what the rows are
// in every CTA's shared memory.  Past that its eight SMs' rate of scattered accesses
// binds (0.3 a cycle each), and two launches over all SMs are faster, the second of CTAs
// that meet at a barrier in memory (1.3 us a step; a launch a step took 3.5, and the
// host as long as the GPU).  That one starts once every SM has room for a CTA of it: it
// waits for the CTAs of other streams' kernels that fill one.  Cluster against grid: 64 rows of 306 entries 21 : 24 us,
// 512 of 74 24 : 20, 1024 of 76 30 : 22, 4096 of 24 54 : 30.
constexpr int kForkThreads = 1024;
constexpr int kForkClaim = INT32_MIN, kForkTail = INT32_MIN / 2;
constexpr int64_t kForkClusterEntries = 26000;

// What a row is and becomes.  In shared memory, for a CTA that meets with others at
// every step:
struct ForkRows {
  int* kept_;       // positions it gets
  int* old_pages_;  // pages it had
  int* least_;      // fewest pages that a child of it takes
  int* aux;         // see the steps
  int16_t* parent_;  // -1: none
  uint16_t* children_;
  __device__ int parent(int r) const { return parent_[r]; }
  __device__ int kept(int r) const { return kept_[r]; }
  __device__ int old_pages(int r) const { return old_pages_[r]; }
  __device__ int children(int r) const { return children_[r]; }
  __device__ int least(int r) const { return least_[r]; }
};

// or from the arguments, with the first step's children and least pages in counts and
// new_lengths until the sixth writes those:
struct ForkInputs {
  const ForkParams& p;
  __device__ int length(int r) const {
    const int n = p.lengths[r];
    return n >= 0 && n <= p.width * kPage ? n : 0;
  }
  __device__ int parent(int r) const {
    const int q = p.parents[r];
    return q >= 0 && q < p.rows ? q : -1;
  }
  __device__ int kept(int r) const {
    const int q = parent(r), most = p.keep ? max(p.keep[r], 0) : INT32_MAX;
    return q < 0 ? 0 : min(length(q), most);
  }
  __device__ int old_pages(int r) const { return (length(r) + kPage - 1) / kPage; }
  __device__ int children(int r) const { return p.counts[r]; }
  __device__ int least(int r) const { return p.new_lengths[r]; }
};

// The steps, for CTA `cta` of `ctas`.
template <class Rows>
struct Fork {
  const ForkParams& p;
  const Rows& rows;
  int cta, ctas;

  // (neighbouring numbers in different CTAs)
  __device__ int warp() const { return (int)(threadIdx.x >> 5) * ctas + cta; }
  __device__ int warps() const { return ctas * (kForkThreads / 32); }
  __device__ int thread() const { return (int)threadIdx.x * ctas + cta; }
  __device__ int threads() const { return ctas * kForkThreads; }
  __device__ bool in_pool(int page) const { return page >= 0 && page < p.num_pages; }
  __device__ void report() const { record_error(p.err, PGD_EDEVICE_BOUNDS); }
  __device__ int pages(int r) const { return (rows.kept(r) + kPage - 1) / kPage; }
  __device__ int entry(int r, int e) const { return (int)((size_t)r * p.width + e); }
  // an old row loses its entries from here on (some child, if any, takes fewer)
  __device__ int lost_from(int r) const {
    const int children = rows.children(r), least = rows.least(r);
    return children == 0 ? 0 : min(least, rows.old_pages(r));
  }
  __device__ int tail_page(int r) const {  // -1: the last page is full, or there is none
    const int n = rows.kept(r);
    return n % kPage ? p.table[(size_t)rows.parent(r) * p.width + n / kPage] : -1;
  }
  __device__ bool claimed(int page, int r, int e) const {
    return in_pool(page) && __ldcg(&p.shares[page]) == kForkClaim + entry(r, e);
  }
  template <class Lo, class F>
  __device__ void each_entry(Lo lo, F f) const {
    each_table_entry(p.table, p.rows, p.width, warp(), warps(), lo,
                     [&](int r) { return rows.old_pages(r); }, f);
  }
  // the list's next page: before, and once the freed pages are back
  __device__ int head() const { return p.free_head ? *p.free_head : 0; }
  __device__ bool bad_head() const { return head() < 0 || head() > p.num_free; }

  // shares as if every entry that no child takes were given up (a row's children, all
  // told, hold its pages once each; the sums need no order)
  __device__ void adjust() const {
    auto add = [&](int page, int n) {
      if (in_pool(page))
        atomicAdd(&p.shares[page], p.undo ? -n : n);
      else
        report();
    };
    each_entry([&](int r) { return rows.children(r) == 1 ? rows.old_pages(r) : 0; },
               [&](int r, int, int page) { add(page, rows.children(r) - 1); });
    if (p.keep)  // rows that their parents' entries are cut for
      for (int r = warp(); r < p.rows; r += warps()) {
        const int q = rows.parent(r);
        if (q < 0) continue;
        for (int e = pages(r) + (threadIdx.x & 31); e < rows.old_pages(q); e += 32)
          add(p.table[(size_t)q * p.width + e], -1);
      }
  }
  __device__ void claim() const {
    each_entry([&](int r) { return lost_from(r); }, [&](int r, int e, int page) {
      if (!in_pool(page)) return;
      const int held = __ldcg(&p.shares[page]);
      if (held < 0) {
        if (held < -1 && held > kForkTail) report();  // given back more often than held
        atomicMin(&p.shares[page], kForkClaim + entry(r, e));
      }
    });
  }
  // the claims of a row to `counts` of it, zero before (and each row's of one warp)
  __device__ void count(int* counts) const {
    each_entry([&](int r) { return lost_from(r); }, [&](int r, int e, int page) {
      if (claimed(page, r, e)) atomicAdd(&counts[r], 1);
    });
  }
  // A row leaves `page`, its last one in part use: a share less, unless its shares say that
  // nobody is left to hold it (a claim stays as it is for all that look for it).
  __device__ void leave(int page) const {
    if (in_pool(page) &&
        (__ldcg(&p.shares[page]) < 0 || atomicSub(&p.shares[page], 1) < 0))
      report();
  }
  __device__ void leave_tails() const {
    for (int r = thread(); r < p.rows; r += threads()) leave(tail_page(r));
  }
  // row r's `n` claimed pages, the `at`-th of `freed` on, to the list (a warp; four
  // entries a lane at once: one at a time, rows of 126 entries took 5 us)
  __device__ void list(int r, int at, int n, int freed) const {
    const int lane = threadIdx.x & 31, hi = rows.old_pages(r), end = at + n;
    const int32_t* row = p.table + (size_t)r * p.width;
    for (int e0 = lost_from(r) + lane; at < end && e0 - lane < hi; e0 += 128) {
      int page[4];
      bool mine[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) page[k] = e0 + 32 * k < hi ? row[e0 + 32 * k] : -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) mine[k] = claimed(page[k], r, e0 + 32 * k);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const unsigned who = __ballot_sync(0xffffffffu, mine[k]);
        if (mine[k]) {
          const int to = head() - freed + at + __popc(who & ((1u << lane) - 1u));
          if (!bad_head() && to >= 0) p.free_pages[to] = page[k];
          p.shares[page[k]] = 0;
        }
        at += __popc(who);
      }
    }
  }
  // The lowest row to claim `page` keeps it, where all have left it and none gave it up.
  __device__ void claim_tail(int r, int page) const {
    if (!in_pool(page)) return;
    const int held = __ldcg(&p.shares[page]);
    if (held < 0 && held >= kForkTail) atomicMin(&p.shares[page], kForkTail + r);
  }
  __device__ void claim_tails() const {
    for (int r = thread(); r < p.rows; r += threads()) claim_tail(r, tail_page(r));
  }
  __device__ int listed_head(int freed) const {  // (a list may have no room for some)
    return bad_head() ? head() : max(head() - freed, 0);
  }
  // What becomes of row r's last page, `page` (-1: full or none): 1: a copy; -1: as it
  // is; -2: none, the row loses it.
  __device__ int last(int r, int page) const {
    if (in_pool(page)) return __ldcg(&p.shares[page]) != kForkTail + r ? 1 : -1;
    return rows.kept(r) % kPage != 0 ? -2 : -1;
  }
  // The page for the copy that `at` rows before want one too (-2: none).
  __device__ int copy_page(int at, int head1) const {
    if (bad_head() || at >= p.num_free - head1) return -2;
    const int page = __ldcg(&p.free_pages[head1 + at]);
    return in_pool(page) ? page : -2;
  }
  // Row r's outputs; to: the last page it gets, or as last (not 1).
  __device__ void write(int r, int to, int page, int kept) const {
    p.new_lengths[r] = to == -2 ? kept - kept % kPage : kept;
    p.sources[r] = to >= 0 ? page : -1;
    p.targets[r] = to >= 0 ? to : -1;
    p.counts[r] = to >= 0 ? kept % kPage : 0;
    if (to == -1 && in_pool(page)) p.shares[page] = 0;  // the one that keeps it
  }
  // Moves the rows: row r gets n_pages(r) pages of row parent(r), the last one to(r) (-1, -2
  // as last).  `cells`: rows << p.slab_shift words.
  template <class Parent, class Pages, class To>
  __device__ void move(int* cells, Parent parent, Pages n_pages, To to) const {
    const int shift = p.slab_shift, columns = 1 << shift, R = p.rows;
    for (int c0 = cta << shift; c0 < p.width; c0 += ctas << shift) {
      const int n = min(columns, p.width - c0);
#pragma unroll 4
      for (int k = threadIdx.x; k < R << shift; k += kForkThreads) {
        const int r = k >> shift, c = k & (columns - 1);
        if (c < n) cells[k] = p.table[(size_t)r * p.width + c0 + c];
      }
      __syncthreads();
      for (int k = threadIdx.x; k < R << shift; k += kForkThreads) {
        const int r = k >> shift, c = k & (columns - 1), e = c0 + c;
        const int q = parent(r), pages = n_pages(r), last = to(r);
        if (c >= n || e >= pages) continue;
        const bool tail = e == pages - 1 && last != -1;  // (-1 where the last page is full)
        const int page = cells[(q << shift) + c];
        if (!in_pool(page)) report();  // (adjust looks at entries that some row gives up)
        if (tail && last >= 0)
          p.table[(size_t)r * p.width + e] = last;
        else if (q != r && !tail)
          p.table[(size_t)r * p.width + e] = page;
      }
      __syncthreads();
    }
  }
};

// Children and least pages of all rows, by each CTA for itself: rows.aux and rows.least
// (the latter, like kept and old_pages, of all fields filled here).
__device__ void fork_count_children(const ForkParams& p, const ForkRows& rows, int* scratch,
                                    bool reports) {
  const int tid = threadIdx.x, R = p.rows;
#pragma unroll 4
  for (int r = tid; r < R; r += kForkThreads) {
    const int n = p.lengths[r], q = p.parents[r];
    const bool good = n >= 0 && n <= p.width * kPage;
    rows.old_pages_[r] = good ? (n + kPage - 1) / kPage : 0;
    rows.kept_[r] = good ? n : 0;  // for now, what a child has of it
    rows.parent_[r] = (int16_t)(q >= 0 && q < R ? q : -1);
    rows.least_[r] = INT32_MAX;
    rows.aux[r] = 0;
    if (reports && (!good || q < -1 || q >= R)) record_error(p.err, PGD_EDEVICE_BOUNDS);
  }
  __syncthreads();
#pragma unroll 4
  for (int r = tid; r < R; r += kForkThreads) {
    const int q = rows.parent_[r];
    int n = q < 0 ? 0 : rows.kept_[q];
    if (p.keep) n = min(n, max(p.keep[r], 0));
    scratch[r] = n;
    if (q >= 0) {
      atomicAdd(&rows.aux[q], 1);
      atomicMin(&rows.least_[q], (n + kPage - 1) / kPage);
    }
  }
  __syncthreads();
  for (int r = tid; r < R; r += kForkThreads) {
    rows.kept_[r] = scratch[r];
    rows.children_[r] = (uint16_t)rows.aux[r];
  }
  __syncthreads();
}

__device__ __forceinline__ ForkRows fork_rows_at(int* smem, int R) {
  ForkRows rows;
  rows.kept_ = smem;
  rows.old_pages_ = smem + R;
  rows.least_ = smem + 2 * R;
  rows.aux = smem + 3 * R;
  rows.parent_ = reinterpret_cast<int16_t*>(smem + 4 * R);
  rows.children_ = reinterpret_cast<uint16_t*>(rows.parent_ + R);
  return rows;  // five words a row
}

__global__ void __launch_bounds__(kForkThreads) fork_rows_kernel(ForkParams p) {
  extern __shared__ int smem[];
  __shared__ int warps[33];
  cg::cluster_group cluster = cg::this_cluster();
  const int R = p.rows, tid = threadIdx.x;
  const ForkRows rows = fork_rows_at(smem, R);
  int* cells = smem + 5 * R;
  const Fork<ForkRows> fork{p, rows, (int)cluster.block_rank(), (int)cluster.num_blocks()};
  pdl_wait();
  pdl_allow_dependents();
  if (fork.thread() == 0 && fork.bad_head()) fork.report();
  fork_count_children(p, rows, cells, fork.cta == 0);
  fork.adjust();
  cluster.sync();
  fork.claim();
  cluster.sync();
  for (int r = tid; r < R; r += kForkThreads) rows.aux[r] = 0;
  __syncthreads();
  fork.count(rows.aux);
  fork.leave_tails();
  __syncthreads();
  // (each_entry's rows of this CTA)
  const int n = rows_at_a_time(R, fork.warps());
  for (int r = tid; r < R; r += kForkThreads)
    if (r / n % fork.ctas == fork.cta) p.sources[r] = rows.aux[r];
  cluster.sync();
  int freed = 0;  // of all rows
  for (int r0 = 0; r0 < R; r0 += kForkThreads) {
    const int r = r0 + tid;
    int total;
    const int at = block_scan(r < R ? __ldcg(&p.sources[r]) : 0, warps, total);
    if (r < R) rows.aux[r] = freed + at;
    freed += total;
    __syncthreads();
  }
  if (fork.thread() == 0 && !fork.bad_head() && fork.head() < freed) fork.report();
  for (int r = fork.warp(); r < R; r += fork.warps()) {
    const int at = rows.aux[r], end = r + 1 < R ? rows.aux[r + 1] : freed;
    if (at < end) fork.list(r, at, end - at, freed);
  }
  fork.claim_tails();
  cluster.sync();
  const int head1 = fork.listed_head(freed);
  int copies = 0;
  for (int r0 = 0; r0 < R; r0 += kForkThreads) {  // (every CTA, all rows)
    const int r = r0 + tid;
    int to = r < R ? fork.last(r, fork.tail_page(r)) : -1, total;
    const int at = copies + block_scan(to == 1, warps, total);
    copies += total;
    if (to == 1) to = fork.copy_page(at, head1);
    if (to == -2 && fork.cta == 0) fork.report();
    if (r < R) rows.aux[r] = to;
    __syncthreads();
  }
  cluster.sync();
  for (int r = fork.thread(); r < R; r += fork.threads())
    fork.write(r, rows.aux[r], fork.tail_page(r), rows.kept(r));
  if (fork.thread() == 0)
    *p.free_head_out = fork.bad_head() ? head1 : min(head1 + copies, p.num_free);
  cluster.sync();  // the last entries of the parents were read above
  fork.move(
      cells, [&](int r) { return rows.parent(r); }, [&](int r) { return fork.pages(r); },
      [&](int r) { return rows.aux[r]; });
}

// Larger tables: the first step, which leaves the children and least pages (and zeros for
// claims and for the count of the barriers that follow) in the outputs (p.undo: takes it
// back, where the launch of the others is refused),
__global__ void __launch_bounds__(kForkThreads) fork_adjust_kernel(ForkParams p) {
  extern __shared__ int smem[];
  const int R = p.rows, tid = threadIdx.x;
  const ForkRows rows = fork_rows_at(smem, R);
  const Fork<ForkRows> fork{p, rows, (int)blockIdx.x, (int)gridDim.x};
  pdl_wait();
  pdl_allow_dependents();
  fork_count_children(p, rows, smem + 5 * R, fork.cta == 0);
  if (fork.cta == 0) {
    if (tid == 0) {
      if (fork.bad_head()) fork.report();
      *p.free_head_out = 0;
    }
    for (int r = tid; r < R; r += kForkThreads) {
      p.counts[r] = rows.children_[r];
      p.new_lengths[r] = rows.least_[r];
      p.sources[r] = 0;
    }
  }
  fork.adjust();
}

// and the others, on all SMs.  A thread sees to a row's last page (there is one for each).
__global__ void __launch_bounds__(kForkThreads, 1) fork_grid_kernel(ForkParams p) {
  extern __shared__ int smem[];
  __shared__ int sums[2][kForkThreads / 32];
  const int R = p.rows, tid = threadIdx.x, lane = tid & 31;
  const ForkInputs inputs{p};
  const Fork<ForkInputs> fork{p, inputs, (int)blockIdx.x, (int)gridDim.x};
  GridBarrier all{reinterpret_cast<unsigned int*>(p.free_head_out), p.err, gridDim.x};
  const int mine = fork.thread() < R ? fork.thread() : -1;
  const int tail = mine >= 0 ? fork.tail_page(mine) : -1;
  fork.claim();
  if (!all.meet()) return;
  fork.count(p.sources);
  fork.leave(tail);
  if (!all.meet()) return;
  // a run of rows a CTA: the claims before it, and in all
  const int lo = (int)((int64_t)R * fork.cta / fork.ctas);
  const int hi = (int)((int64_t)R * (fork.cta + 1) / fork.ctas);
  int before = 0, freed = 0;
#pragma unroll 4
  for (int r = tid; r < R; r += kForkThreads) {
    const int n = p.sources[r];
    freed += n;
    if (r < lo) before += n;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  freed = __reduce_add_sync(0xffffffffu, freed);
  if (lane == 0) {
    sums[0][tid >> 5] = before;
    sums[1][tid >> 5] = freed;
  }
  __syncthreads();
  before = __reduce_add_sync(0xffffffffu, sums[0][lane]);
  freed = __reduce_add_sync(0xffffffffu, sums[1][lane]);
  if (fork.thread() == 0 && !fork.bad_head() && fork.head() < freed) fork.report();
  for (int r = lo + (tid >> 5); r < hi; r += kForkThreads / 32) {
    const int n = p.sources[r];
    if (n == 0) continue;
    int at = 0;
    for (int k = lo + (tid & 31); k < r; k += 32) at += p.sources[k];
    fork.list(r, before + __reduce_add_sync(0xffffffffu, at), n, freed);
  }
  fork.claim_tail(mine, tail);
  if (!all.meet()) return;
  if (mine >= 0) {  // for all CTAs' sums
    p.targets[mine] = fork.last(mine, tail);
    p.counts[mine] = tail;
  }
  if (!all.meet()) return;
  const int head1 = fork.listed_head(freed);
  int* parent = smem;
  int* kept = smem + R;
  int* to = smem + 2 * R;
  // copies before a row: a run of rows a warp, one of every 32 a lane
  constexpr int kRun = kMaxForkRows / kForkThreads;
  const int run = (R + kForkThreads - 1) / kForkThreads, r0 = (tid >> 5) * 32 * run + lane;
  int last[kRun], before_run = 0;
#pragma unroll
  for (int k = 0; k < kRun; ++k)
    last[k] = k < run && r0 + 32 * k < R ? p.targets[r0 + 32 * k] : -1;
#pragma unroll
  for (int k = 0; k < kRun; ++k) before_run += __popc(__ballot_sync(0xffffffffu, last[k] == 1));
  if (lane == 0) sums[0][tid >> 5] = before_run;
  __syncthreads();
  const int in_run = sums[0][lane];
  const int copies = __reduce_add_sync(0xffffffffu, in_run);
  int at = __reduce_add_sync(0xffffffffu, lane < tid >> 5 ? in_run : 0);
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    const int r = r0 + 32 * k;
    const unsigned who = __ballot_sync(0xffffffffu, last[k] == 1);
    if (last[k] == 1) last[k] = fork.copy_page(at + __popc(who & ((1u << lane) - 1u)), head1);
    at += __popc(who);
    if (last[k] == -2 && fork.cta == 0) fork.report();
    if (k < run && r < R) {
      parent[r] = inputs.parent(r);
      kept[r] = inputs.kept(r);
      to[r] = last[k];
    }
  }
  all.arrive();
  fork.move(
      smem + 3 * R, [&](int r) { return parent[r]; },
      [&](int r) { return (kept[r] + kPage - 1) / kPage; }, [&](int r) { return to[r]; });
  // the outputs, once nobody needs what they held so far
  if (fork.cta != 0 || !all.wait()) return;
#pragma unroll 4
  for (int r = tid; r < R; r += kForkThreads) fork.write(r, to[r], p.counts[r], kept[r]);
  if (tid == 0) *p.free_head_out = fork.bad_head() ? head1 : min(head1 + copies, p.num_free);
}

cudaError_t launch_fork_rows(const ForkParams& params, int sm_count, cudaStream_t stream) {
  ForkParams p = params;
  const int64_t entries = (int64_t)p.rows * p.width;
  const int limit = 220 * 1024;
  // a slab as wide as there is room and use for, beside `words` a row
  auto slab = [&](int ctas, int words) {
    p.slab_shift = 0;
    while (p.slab_shift < 6 && ((int64_t)ctas << p.slab_shift) < p.width &&
           (words + (2ll << p.slab_shift)) * 4 * p.rows <= limit)
      ++p.slab_shift;
    return (words + (1ll << p.slab_shift)) * 4 * (size_t)p.rows;
  };
  auto cluster = [&]() {
    static std::atomic<bool> configured[64];
    const cudaError_t e = allow_smem(fork_rows_kernel, limit, configured);
    if (e != cudaSuccess) return e;
    int ctas = 1;
    while (ctas < 8 && entries > 2048ll * ctas) ctas *= 2;
    return launch_cluster(fork_rows_kernel, ctas, slab(ctas, 5), stream, p);
  };
  p.undo = 0;
  if (entries <= kForkClusterEntries) return cluster();
  static std::atomic<bool> configured[2][64];
  cudaError_t e = allow_smem(fork_adjust_kernel, limit, configured[0]);
  if (e == cudaSuccess) e = allow_smem(fork_grid_kernel, limit, configured[1]);
  auto adjust = [&]() {
    return launch_pdl(fork_adjust_kernel, dim3(sm_count), dim3(kForkThreads), 24 * (size_t)p.rows,
                      stream, p);
  };
  if (e == cudaSuccess) e = adjust();
  if (e != cudaSuccess) return e;
  const size_t smem = slab(sm_count, 3);
  if (launch_grid(fork_grid_kernel, sm_count, smem, stream, p) == cudaSuccess) return cudaSuccess;
  // Refused (a context of fewer SMs than the device's): the shares as they were, and all steps
  // by one cluster, whatever the size.  Where that is refused too, nothing has changed.
  (void)cudaGetLastError();
  p.undo = 1;
  e = adjust();
  p.undo = 0;
  return e == cudaSuccess ? cluster() : e;
}

// ------------------------------------------------------------------ copy_pages

// A warp copies 4 KB pieces of (copy, pool, kv head) tiles, 8 x 16 bytes a lane
// in flight: pieces, not copies, are shared out, so a few copies of many layers fill the
// SMs too (40 copies in 24 pools of 2 kv heads of 64: 4.1 us), and a page in part use costs
// its positions only.  Bound by HBM for copies past L2: 1101 pages of two layers (8 kv heads
// of 128) in 177 us, 6.5 TB/s, 0.98 of a plain copy's rate.
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
// with atomics in the workspace; then their words' bits are summed into prefixes (one
// per `step` words), from which the rank of any page among the free or the held is one
// look-up.
//   moves: the k-th held page from the top goes to the k-th free page from the
//   bottom while the latter is lower.  Without a limit that is all held pages
//   past the first `held` places of the free and held pages together.
//   free list: free pages left and vacated ones, each at its rank.
// Bound by latency and the rate of scattered accesses in L2, as fork_rows: one cluster
// for small pools and tables; past that all SMs at once, after a launch that clears the bitmaps.
// Every CTA sums all bits for itself (2 bits a page out of L2), which is less than handing
// sums over.  Cluster against grid: 34 000 entries and pages 15 : 16 us, 70 000 20 : 17.5,
// 128 000 28 : 19.5, 490 000 63 : 25.
constexpr int kCompactThreads = 1024;
constexpr int64_t kCompactClusterWork = 48000;  // entries and pages

// What the bitmaps' sums come to.
struct CompactSums {
  int held_total, moves;
  bool wrong;
};

// Before the larger: bitmaps, flag and the count of the barriers.
__global__ void __launch_bounds__(kCompactThreads) compact_clear_kernel(CompactParams p) {
  pdl_wait();
  pdl_allow_dependents();
  const int words = (p.num_pages + 31) / 32;
  for (int w = blockIdx.x * kCompactThreads + threadIdx.x; w < 2 * words + 2;
       w += gridDim.x * kCompactThreads)
    p.bits[w] = 0;
}

template <bool GRID>
__global__ void __launch_bounds__(kCompactThreads, 1) compact_pages_kernel(CompactParams p) {
  extern __shared__ int smem[];
  __shared__ int warps[33];
  __shared__ int unlimited;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = GRID ? (int)gridDim.x : (int)cluster.num_blocks();
  const int cta = GRID ? (int)blockIdx.x : (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gwarp = warp * ctas + cta, gwarps = ctas * (kCompactThreads / 32);
  const int gtid = cta * kCompactThreads + tid, gthreads = ctas * kCompactThreads;
  const int words = (p.num_pages + 31) / 32, blocks = (words + p.step - 1) / p.step;
  uint32_t* free_bits = p.bits;
  uint32_t* held_bits = p.bits + words;
  uint32_t* bad = p.bits + 2 * words;
  GridBarrier all{bad + 1, p.err, gridDim.x};
  auto step_done = [&]() {
    if constexpr (GRID) return all.meet();
    cluster.sync();
    return true;
  };
  int* free_at = smem;  // [blocks] pages before the block's words
  int* held_at = smem + blocks;
  pdl_wait();
  pdl_allow_dependents();
  const int head = p.free_head ? *p.free_head : 0;
  const bool bad_head = head < 0 || head > p.num_free;
  auto pages_of = [&](int r) {
    const int n = p.lengths[r];
    return n >= 0 && n <= p.width * kPage ? (n + kPage - 1) / kPage : -1;
  };
  auto in_pool = [&](int page) { return page >= 0 && page < p.num_pages; };
  // set bits before word w
  auto word_rank = [&](const uint32_t* bits, const int* at, int w) {
    if (p.step == 1) return at[w];
    const int b = w / p.step;
    int n = at[b];
    for (int k = b * p.step; k < w; ++k) n += __popc(bits[k]);
    return n;
  };
  if constexpr (!GRID) {
    for (int w = gtid; w < 2 * words + 1; w += gthreads) p.bits[w] = 0;
    step_done();
  }
  {
    if (bad_head && gtid == 0) atomicOr(bad, 1u);
#pragma unroll 4
    for (int k = (bad_head ? p.num_free : head) + gtid; k < p.num_free; k += gthreads) {
      const int page = p.free_pages[k];
      if (!in_pool(page))
        atomicOr(bad, 1u);
      else if (atomicOr(&free_bits[page >> 5], 1u << (page & 31)) >> (page & 31) & 1u)
        atomicOr(bad, 1u);  // listed twice
    }
    each_table_entry(
        p.table, p.rows, p.width, gwarp, gwarps, [](int) { return 0; },
        [&](int r) {
          const int n = pages_of(r);
          if (n < 0) atomicOr(bad, 1u);
          return n;
        },
        [&](int, int, int page) {
          if (in_pool(page))
            atomicOr(&held_bits[page >> 5], 1u << (page & 31));
          else
            atomicOr(bad, 1u);
        });
    if (!step_done()) return;
  }

  CompactSums sum;
  {
    // prefixes: thread t sums a run of blocks
    const int run = (blocks + kCompactThreads - 1) / kCompactThreads;
    const int b0 = min(tid * run, blocks), b1 = min(b0 + run, blocks);
    int nf = 0, nh = 0;
    bool both = false;
#pragma unroll 8
    for (int w = b0 * p.step; w < min(b1 * p.step, words); ++w) {
      const uint32_t f = __ldcg(&free_bits[w]), h = __ldcg(&held_bits[w]);
      nf += __popc(f);
      nh += __popc(h);
      both |= (f & h) != 0;
    }
    int free_total;
    const int f_at = block_scan(nf, warps, free_total);
    __syncthreads();
    const int h_at = block_scan(nh, warps, sum.held_total);
    if (tid == 0) unlimited = 0;
    sum.wrong = __syncthreads_or(both) || __ldcg(bad) != 0;
    // without a limit the held pages past the first held_total places of the union move
    int f = f_at, h = h_at;
    for (int b = b0; b < b1; ++b) {
      free_at[b] = f;
      held_at[b] = h;
#pragma unroll 4
      for (int w = b * p.step; w < min((b + 1) * p.step, words); ++w) {
        const uint32_t fw = free_bits[w], hw = held_bits[w], all = fw | hw;
        if (f + h < sum.held_total && f + h + __popc(all) >= sum.held_total) {
          uint32_t rest = all;  // the word that holds the last of these places
          int h_in = 0;
          for (int k = f + h; k < sum.held_total; ++k) {
            const uint32_t low = rest & -rest;
            h_in += (hw & low) != 0;
            rest ^= low;
          }
          unlimited = sum.held_total - (h + h_in);
        }
        f += __popc(fw);
        h += __popc(hw);
      }
    }
    __syncthreads();
    sum.moves = sum.wrong ? 0 : min(unlimited, p.max_moves);
    if (sum.wrong && gtid == 0) record_error(p.err, PGD_EDEVICE_BOUNDS);
    // the moves: sources from the top, targets from the bottom
    const int moves = sum.moves;
    for (int w = tid * ctas + cta; moves > 0 && w < words; w += gthreads) {
      const uint32_t fw = free_bits[w], hw = held_bits[w];
      int k = word_rank(free_bits, free_at, w);
      for (uint32_t m = fw; m && k < moves; m &= m - 1, ++k) p.targets[k] = 32 * w + __ffs(m) - 1;
      k = sum.held_total - word_rank(held_bits, held_at, w);  // held pages from this word up
      for (uint32_t m = hw; m && k - __popc(m) < moves; m &= m - 1)
        if (--k < moves) p.sources[k] = 32 * w + __ffs(m) - 1;
    }
    for (int k = moves + gtid; k < p.max_moves; k += gthreads) p.sources[k] = p.targets[k] = -1;
    if (!step_done()) return;
  }

  {
    const int moves = sum.moves, kept = sum.held_total - moves;  // held pages of a lower rank stay
    const bool wrong = sum.wrong;
    // the held pages from `lowest` up have moved, to the free ones up to `highest`
    const int lowest = moves > 0 ? __ldcg(&p.sources[moves - 1]) : INT32_MAX;
    const int highest = moves > 0 ? __ldcg(&p.targets[moves - 1]) : -1;
    each_table_entry(
        p.table, p.rows, p.width, gwarp, gwarps, [](int) { return 0; },
        [&](int) { return p.width; },
        [&](int r, int e, int page) {
          if (page >= lowest && page < p.num_pages && e < pages_of(r)) {
            const int w = page >> 5;
            const int k = sum.held_total - 1 - word_rank(held_bits, held_at, w) -
                          __popc(held_bits[w] & ((1u << (page & 31)) - 1u));
            page = __ldcg(&p.targets[k]);
          }
          p.new_table[(size_t)r * p.width + e] = page;
        });
    // shares, and the list: free pages left and vacated ones, a word a warp at a time
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
    for (int w = gwarp; w < words; w += gwarps) {
      const int page = 32 * w + lane;
      const uint32_t fw = free_bits[w], hw = held_bits[w];
      const bool vacated = !wrong && (hw >> lane & 1u) && page >= lowest;
      const bool left = (fw >> lane & 1u) && page > highest;
      const uint32_t listed = __ballot_sync(0xffffffffu, vacated || left);
      if (!wrong && listed) {
        const int at = max(word_rank(free_bits, free_at, w) - moves, 0) +
                       max(word_rank(held_bits, held_at, w) - kept, 0);
        if (listed >> lane & 1u) p.new_free[head + at + __popc(listed & below)] = page;
      }
      const bool taken = !wrong && (fw >> lane & 1u) && page <= highest;
      if (page < p.num_pages && !vacated && !taken) p.new_shares[page] = p.shares[page];
    }
    for (int k = gtid; k < moves; k += gthreads) {  // (nobody else touches the two)
      const int from = __ldcg(&p.sources[k]), to = __ldcg(&p.targets[k]);
      const int n = p.shares[from];
      p.new_shares[to] = n;
      p.new_shares[from] = 0;
    }
    for (int k = gtid; k < (wrong ? p.num_free : head); k += gthreads)
      p.new_free[k] = p.free_pages[k];
    // the end of the pages in use: the highest held page left, or the highest target
    if (gtid == 0) {
      int end = highest + 1;
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
        for (int w = lo * p.step; w < min((lo + 1) * p.step, words); ++w)
          for (uint32_t m = held_bits[w]; m; m &= m - 1)
            if (++n == kept) end = max(end, 32 * w + __ffs(m));
      }
      *p.end = end;
    }
  }
}

size_t compact_workspace_bytes(int num_pages) {
  const size_t words = ((size_t)num_pages + 31) / 32;
  return (2 * words + 2) * 4;  // bitmaps, flag, count of the barriers
}

cudaError_t launch_compact_pages(const CompactParams& params, int sm_count, cudaStream_t stream) {
  CompactParams p = params;
  const int words = (p.num_pages + 31) / 32;
  p.step = 1;
  while ((words + p.step - 1) / p.step > kMaxCompactPrefixes) p.step *= 2;
  const size_t smem = (size_t)((words + p.step - 1) / p.step) * 8;
  const int64_t work = (int64_t)p.rows * p.width + p.num_pages;
  static std::atomic<bool> configured[2][64];
  auto cluster = [&]() {
    const cudaError_t e = allow_smem(compact_pages_kernel<false>, 200 * 1024, configured[0]);
    if (e != cudaSuccess) return e;
    int ctas = 1;
    while (ctas < 8 && work > 2048ll * ctas) ctas *= 2;
    return launch_cluster(compact_pages_kernel<false>, ctas, smem, stream, p);
  };
  if (work <= kCompactClusterWork) return cluster();
  cudaError_t e = allow_smem(compact_pages_kernel<true>, 200 * 1024, configured[1]);
  if (e == cudaSuccess)
    e = launch_pdl(compact_clear_kernel, dim3(32), dim3(kCompactThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  e = launch_grid(compact_pages_kernel<true>, sm_count, smem, stream, p);
  if (e == cudaSuccess) return e;
  (void)cudaGetLastError();  // refused, as in launch_fork_rows
  return cluster();
}

}  // namespace pgd
