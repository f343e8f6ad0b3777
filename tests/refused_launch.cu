// page_ops.cu with launches that a test can refuse, as a context of few SMs does, or leave out
// altogether: a list of what would have been launched remains.  Built by test_refused_launch.py.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstring>
#include <utility>

namespace {

int g_refused;    // 1: cooperative launches, 2: clusters of several CTAs
bool g_dry;       // nothing is launched
char g_done[256];  // a letter a launch: g (cooperative), c (a cluster), k (any other)

template <class... Expected, class... Actual>
cudaError_t test_launch(const cudaLaunchConfig_t* cfg, void (*kernel)(Expected...),
                        Actual&&... args) {
  char kind = 'k';
  for (unsigned i = 0; i < cfg->numAttrs; ++i) {
    const cudaLaunchAttribute& a = cfg->attrs[i];
    if (a.id == cudaLaunchAttributeCooperative && a.val.cooperative) kind = 'g';
    if (a.id == cudaLaunchAttributeClusterDimension && a.val.clusterDim.x > 1) kind = 'c';
  }
  if (kind == 'g' && (g_refused & 1)) return cudaErrorCooperativeLaunchTooLarge;
  if (kind == 'c' && (g_refused & 2)) return cudaErrorLaunchOutOfResources;
  const size_t n = strlen(g_done);
  if (n + 1 < sizeof(g_done)) g_done[n] = kind;
  return g_dry ? cudaSuccess
               : cudaLaunchKernelEx(cfg, kernel, std::forward<Actual>(args)...);
}

// (a device of its own without launches: what is set once a device is not set on the real one)
cudaError_t test_device(int* dev) {
  if (!g_dry) return cudaGetDevice(dev);
  *dev = 63;
  return cudaSuccess;
}

template <class Kernel>
cudaError_t test_attribute(Kernel kernel, cudaFuncAttribute attr, int value) {
  return g_dry ? cudaSuccess : cudaFuncSetAttribute(kernel, attr, value);
}

}  // namespace

#define cudaLaunchKernelEx test_launch
#define cudaGetDevice test_device
#define cudaFuncSetAttribute test_attribute
#include "page_ops.cu"

#define API extern "C" __attribute__((visibility("default")))

API void refuse(int refused, int dry) {
  g_refused = refused;
  g_dry = dry != 0;
  memset(g_done, 0, sizeof(g_done));
}

API const char* launched() { return g_done; }

API int fork_rows(int rows, int width, int num_pages, int num_free, int sm_count, int32_t* table,
                  const int32_t* lengths, const int32_t* parents, int32_t* shares,
                  int32_t* free_pages, const int32_t* free_head, int32_t* new_lengths,
                  int32_t* sources, int32_t* targets, int32_t* counts, int32_t* free_head_out,
                  unsigned int* err) {
  pgd::ForkParams p = {};
  p.rows = rows;
  p.width = width;
  p.num_pages = num_pages;
  p.num_free = num_free;
  p.table = table;
  p.lengths = lengths;
  p.parents = parents;
  p.shares = shares;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.new_lengths = new_lengths;
  p.sources = sources;
  p.targets = targets;
  p.counts = counts;
  p.free_head_out = free_head_out;
  p.err = err;
  return pgd::launch_fork_rows(p, sm_count, nullptr);
}

API int compact_pages(int rows, int width, int num_pages, int num_free, int max_moves, int sm_count,
                      const int32_t* table, const int32_t* lengths, const int32_t* shares,
                      const int32_t* free_pages, const int32_t* free_head, int32_t* new_table,
                      int32_t* new_shares, int32_t* new_free, int32_t* sources, int32_t* targets,
                      int32_t* end, uint32_t* workspace, unsigned int* err) {
  pgd::CompactParams p = {};
  p.rows = rows;
  p.width = width;
  p.num_pages = num_pages;
  p.num_free = num_free;
  p.max_moves = max_moves;
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
  p.bits = workspace;
  p.err = err;
  return pgd::launch_compact_pages(p, sm_count, nullptr);
}
