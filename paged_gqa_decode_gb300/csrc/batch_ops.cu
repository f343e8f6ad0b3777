// The step's set-up on the GPU: pages, slots and positions from request
// lengths, and rotary positions fused with the paged append.
#include "pgd_device.cuh"
#include "pgd_ext_internal.h"

namespace pgd {

// ------------------------------------------------------------------ assign_pages

// have = ceil(cached / 64), need = ceil((cached + new) / 64); with exclusive
// sums over the requests, request r's new pages are free[head + sum(need -
// have) ..] and its tokens take the places sum(new) .. of the pass.
//
// One launch.  Every CTA walks all requests in chunks of kChunk and scans both
// counts itself (8 bytes a request out of L2: cheaper than a second launch or
// a hand-over between CTAs), keeping the chunk's exclusive sums in shared
// memory; then it does its share of the chunk -- a contiguous range of the
// pass's places, of the new pages and of the requests -- and finds the request
// of a place or page by binary search.  The places are shared out once for the
// whole pass, so consecutive threads write consecutive tokens.  Sums are 64-bit
// (the lengths are the caller's; only their clipped values are stored).
// Bound by latency: 64 requests of a token each take 5.8 us, 500 with 27 008
// tokens 6.5 us, 4099 with 131 072 tokens 10.7 us (1.7 MB, 0.25 us of bytes).
constexpr int kAssignThreads = 1024;
constexpr int kAssignItems = 4;
constexpr int kAssignChunk = kAssignThreads * kAssignItems;

struct AssignRequest {
  int cached, fresh, have, extra;  // new tokens, pages in use, pages to add
  bool valid;                      // lengths in range (an invalid request counts for nothing)
};

__device__ __forceinline__ AssignRequest assign_request(const AssignParams& p, int r) {
  AssignRequest q;
  q.cached = p.cached[r];
  q.fresh = p.new_tokens[r];
  q.valid = q.cached >= 0 && q.fresh >= 0 &&
            (int64_t)q.cached + q.fresh <= (int64_t)p.maxp * kPage;
  if (!q.valid) q.fresh = 0;
  // (no overflow: a valid request's positions fit its table row, below 2^31)
  q.have = q.valid ? (int)(((int64_t)q.cached + kPage - 1) / kPage) : 0;
  q.extra = q.valid ? (int)(((int64_t)q.cached + q.fresh + kPage - 1) / kPage) - q.have : 0;
  return q;
}

// Whether the request's pages and places fit: `start` and `page` are its
// exclusive sums, `room` the pages left in the list.
__device__ __forceinline__ bool assign_served(const AssignParams& p, const AssignRequest& q,
                                              int64_t start, int64_t page, int64_t room) {
  return q.valid && (q.fresh == 0 || start + q.fresh <= p.tokens) &&
         (q.extra == 0 || page + q.extra <= room);
}

// Last index r of the n sorted sums (n >= 1) with sums[r] <= x (sums[0] <= x).
__device__ __forceinline__ int assign_find(const int* sums, int n, int x) {
  int lo = 0, hi = n;  // sums[lo] <= x < sums[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int clip32(int64_t v) {
  return v < (int64_t)INT32_MAX ? (int)v : INT32_MAX;
}

__global__ void __launch_bounds__(kAssignThreads) assign_pages_kernel(const AssignParams p) {
  __shared__ int tok_at[kAssignChunk], page_at[kAssignChunk];  // exclusive sums, clipped
  __shared__ int64_t warp_tok[32], warp_page[32];
  __shared__ int taken_max;
  pdl_wait();
  pdl_allow_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (tid == 0) taken_max = 0;
  const int head0 = p.free_head ? *p.free_head : 0;
  const bool bad_head = head0 < 0 || head0 > p.num_free;
  const int64_t room = bad_head ? 0 : p.num_free - head0;
  if (bad_head && cta == 0 && tid == 0) record_error(p.err, PGD_EDEVICE_BOUNDS);
  // this CTA's places of the pass
  const int64_t t_lo = (int64_t)p.tokens * cta / ctas, t_hi = (int64_t)p.tokens * (cta + 1) / ctas;

  int64_t tok_base = 0, page_base = 0;  // sums over the chunks before
  for (int base = 0; base < p.requests; base += kAssignChunk) {
    const int n = min(kAssignChunk, p.requests - base);
    // each thread's kAssignItems consecutive requests, then the scan
    int64_t tok = 0, page = 0;
    int fresh[kAssignItems], extra[kAssignItems];
#pragma unroll
    for (int k = 0; k < kAssignItems; ++k) {
      const int j = tid * kAssignItems + k;
      fresh[k] = extra[k] = 0;
      if (j < n) {
        const AssignRequest q = assign_request(p, base + j);
        fresh[k] = q.fresh;
        extra[k] = q.extra;
      }
      tok += fresh[k];
      page += extra[k];
    }
    int64_t tok_in = tok, page_in = page;  // inclusive sums over the warp, then the CTA
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, tok_in, o);
      const int64_t b = __shfl_up_sync(0xffffffffu, page_in, o);
      if (lane >= o) {
        tok_in += a;
        page_in += b;
      }
    }
    if (lane == 31) {
      warp_tok[warp] = tok_in;
      warp_page[warp] = page_in;
    }
    __syncthreads();
    if (warp == 0) {
      int64_t a = warp_tok[lane], b = warp_page[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, o);
        const int64_t y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
          a += x;
          b += y;
        }
      }
      warp_tok[lane] = a;
      warp_page[lane] = b;
    }
    __syncthreads();
    const int64_t chunk_tok = warp_tok[31], chunk_page = warp_page[31];
    int64_t t = tok_base + tok_in - tok + (warp ? warp_tok[warp - 1] : 0);
    int64_t g = page_base + page_in - page + (warp ? warp_page[warp - 1] : 0);
#pragma unroll
    for (int k = 0; k < kAssignItems; ++k) {
      const int j = tid * kAssignItems + k;
      if (j < n) {
        tok_at[j] = clip32(t);
        page_at[j] = clip32(g);
      }
      t += fresh[k];
      g += extra[k];
    }
    __syncthreads();

    // this CTA's share of the chunk's requests: starts, lengths, errors
    const int r_lo = (int)((int64_t)n * cta / ctas), r_hi = (int)((int64_t)n * (cta + 1) / ctas);
    for (int j = r_lo + tid; j < r_hi; j += kAssignThreads) {
      const AssignRequest q = assign_request(p, base + j);
      const bool served = assign_served(p, q, tok_at[j], page_at[j], room);
      p.starts[base + j] = min(tok_at[j], p.tokens);
      p.lengths[base + j] = served ? q.cached + q.fresh : q.cached;
      if (!served) record_error(p.err, PGD_EDEVICE_BOUNDS);
    }
    // CTA 0: the pages taken up to the chunk's last served request
    if (cta == 0) {
      for (int j = tid; j < n; j += kAssignThreads) {
        const AssignRequest q = assign_request(p, base + j);
        if (q.extra > 0 && assign_served(p, q, tok_at[j], page_at[j], room))
          atomicMax(&taken_max, page_at[j] + q.extra);
      }
    }
    // its share of the chunk's new pages, into the table
    const int64_t pages = min(chunk_page, max((int64_t)0, room - page_base));
    for (int64_t i = pages * cta / ctas + tid; i < pages * (cta + 1) / ctas;
         i += kAssignThreads) {
      const int at = (int)(page_base + i);  // below room
      const int j = assign_find(page_at, n, at);
      const AssignRequest q = assign_request(p, base + j);
      if (!assign_served(p, q, tok_at[j], page_at[j], room)) continue;
      const int id = p.free_pages[head0 + at];
      p.table[(size_t)(base + j) * p.maxp + q.have + (at - page_at[j])] = id;
      if (id < 0 || id >= p.num_pages) record_error(p.err, PGD_EDEVICE_BOUNDS);
    }
    // its places of the pass that fall into the chunk
    const int64_t lo = max(t_lo, tok_base), hi = min(t_hi, tok_base + chunk_tok);
    for (int64_t i = lo + tid; i < hi; i += kAssignThreads) {
      const int at = (int)i;
      const int j = assign_find(tok_at, n, at);
      const AssignRequest q = assign_request(p, base + j);
      int row = 0, pos = -1, slot = -1;
      if (assign_served(p, q, tok_at[j], page_at[j], room)) {
        row = base + j;
        pos = q.cached + (at - tok_at[j]);
        const int k = pos / kPage;
        const int id = k < q.have ? p.table[(size_t)row * p.maxp + k]
                                  : p.free_pages[head0 + page_at[j] + (k - q.have)];
        if (id >= 0 && id < p.num_pages)
          slot = id * kPage + pos % kPage;
        else
          record_error(p.err, PGD_EDEVICE_BOUNDS);
      }
      p.rows[at] = row;
      p.positions[at] = pos;
      p.slots[at] = slot;
    }
    tok_base += chunk_tok;
    page_base += chunk_page;
    __syncthreads();  // the sums are replaced by the next chunk's
  }
  // padding
  for (int64_t i = max(t_lo, tok_base) + tid; i < t_hi; i += kAssignThreads) {
    p.rows[i] = 0;
    p.positions[i] = -1;
    p.slots[i] = -1;
  }
  if (cta == 0 && tid == 0) {
    p.starts[p.requests] = (int)min(tok_base, (int64_t)p.tokens);
    *p.free_head_out = head0 + taken_max;
  }
}

cudaError_t launch_assign_pages(const AssignParams& p, int sm_count, cudaStream_t stream) {
  const int64_t work = p.tokens > p.requests ? p.tokens : p.requests;
  int64_t ctas = (work + kAssignThreads - 1) / kAssignThreads;
  if (ctas > sm_count) ctas = sm_count;
  if (ctas < 1) ctas = 1;
  return launch_pdl(assign_pages_kernel, dim3((unsigned)ctas), dim3(kAssignThreads), 0, stream, p);
}

// ------------------------------------------------------------------ rotary_append

// Two fp32 values as a bf16x2 word (round to nearest even), `lo` in bits 0-15.
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One word of a rotated pair of words: two pairs across the halves of a head
// (x in wx, y in wy), or four adjacent pairs of a chunk.
__device__ __forceinline__ void turn_across(uint32_t& wx, uint32_t& wy, float c0, float s0,
                                            float c1, float s1) {
  const float x0 = bf16_lo(wx), x1 = bf16_hi(wx), y0 = bf16_lo(wy), y1 = bf16_hi(wy);
  wx = pack_pair(fmaf(x0, c0, -(y0 * s0)), fmaf(x1, c1, -(y1 * s1)));
  wy = pack_pair(fmaf(y0, c0, x0 * s0), fmaf(y1, c1, x1 * s1));
}
__device__ __forceinline__ void turn_adjacent(uint32_t* w, const float4& c, const float4& s) {
  const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float x = bf16_lo(w[k]), y = bf16_hi(w[k]);
    w[k] = pack_pair(fmaf(x, cs[k], -(y * sn[k])), fmaf(y, cs[k], x * sn[k]));
  }
}

// Pair (x, y) of frequency i at position n: (x c - y s, y c + x s) with c + i s
// = factor e^{2 pi i n f}, f in turns.  The phase is an integer product: n
// times the 64-bit fraction f, its overflow dropping whole turns exactly, so
// far positions lose nothing; its upper 32 bits, signed, are the angle in
// [-1/2, 1/2) turns that sincospi takes.
//
// One CTA per token.  Every head of q, k and v is D / 16 units of two 16-byte
// chunks: unit u of a rotated head holds the pairs of chunks u and u + rd / 16
// (rd the rotary_dim) -- the pairs across the halves, or eight adjacent pairs
// of the interleaved layout -- and the units past rd / 16 copy the rest of the
// head, as all of v's do.  A thread's units are a multiple of D / 16 apart, so
// it needs the same eight frequencies for all of them.  Bound by memory: a
// thread has its (nearly always only) unit in flight while the token's
// position, slot and angles are found.  4096 tokens of 32 / 8 heads of 128 take
// 19.5 us (101 MB, 5.1 TB/s; 25.5 us with the values loaded after the position),
// 16 001 out of a fused projection of 64 / 8 heads of 64 52.2 us (328 MB, 6.3 TB/s;
// 83.5 us so).
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(512, 4) rotary_append_kernel(const RotaryParams p) {
  constexpr int kUnits = D / 16;
  __shared__ __align__(16) float cos_t[64], sin_t[64];
  pdl_wait();
  pdl_allow_dependents();
  const int b = blockIdx.x;
  const int rot = p.rotary.rotary_dim / 16;  // rotating units of a head
  const int u = threadIdx.x % kUnits;
  const bool rotates = u < rot;
  const int ca = rotates ? u : 2 * u, cb = rotates ? u + rot : 2 * u + 1;  // the unit's chunks
  const int hq = p.q ? p.hq : 0;
  const int heads = hq + 2 * p.hkv;
  auto load = [&](int h, uint4& a, uint4& z) {
    const uint16_t* src = h < hq           ? p.q + (size_t)b * p.q_stride + h * D
                          : h < hq + p.hkv ? p.k_new + (size_t)b * p.k_stride + (h - hq) * D
                                           : p.v_new + (size_t)b * p.v_stride + (h - hq - p.hkv) * D;
    a = *reinterpret_cast<const uint4*>(src + 8 * ca);
    z = *reinterpret_cast<const uint4*>(src + 8 * cb);
  };
  // The first unit's values do not wait for the token's position.
  int h = threadIdx.x / kUnits;
  uint4 a, z;
  if (h < heads) load(h, a, z);

  const int n = p.positions[b];
  int page = -1, in_page = 0;
  bool skip = n < 0;  // left alone
  if (p.slots) {
    const int slot = p.slots[b];
    skip = skip || slot < 0;
    page = slot / kPage;
    in_page = slot % kPage;
  } else if (!skip) {
    const int row = p.row_of ? p.row_of[b] : b;
    if ((!p.row_of || (row >= 0 && row < p.table_rows)) && n / kPage < p.maxp)
      page = page_of(p.table, row, n / kPage, p.maxp);
    in_page = n % kPage;
  }
  if (skip) return;
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) record_error(p.err, PGD_EDEVICE_BOUNDS);
    return;
  }
  const int pairs = p.rotary.rotary_dim / 2;
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    const uint64_t phase = p.rotary.turns[i] * (uint64_t)(uint32_t)n;
    const float half_turns = (float)(int32_t)(phase >> 32) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    cos_t[i] = c * p.rotary.factor;
    sin_t[i] = s * p.rotary.factor;
  }
  __syncthreads();
  for (; h < heads; h += blockDim.x / kUnits) {
    if (h >= blockDim.x / kUnits) load(h, a, z);
    if (rotates && h < hq + p.hkv) {
      uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
      uint32_t* wz = reinterpret_cast<uint32_t*>(&z);
      if constexpr (kInterleaved) {
        const float4 c0 = *reinterpret_cast<const float4*>(cos_t + 4 * ca);
        const float4 s0 = *reinterpret_cast<const float4*>(sin_t + 4 * ca);
        const float4 c1 = *reinterpret_cast<const float4*>(cos_t + 4 * cb);
        const float4 s1 = *reinterpret_cast<const float4*>(sin_t + 4 * cb);
        turn_adjacent(wa, c0, s0);
        turn_adjacent(wz, c1, s1);
      } else {
#pragma unroll
        for (int w = 0; w < 4; w += 2) {
          const float4 c = *reinterpret_cast<const float4*>(cos_t + 8 * u + 2 * w);
          const float4 s = *reinterpret_cast<const float4*>(sin_t + 8 * u + 2 * w);
          turn_across(wa[w], wz[w], c.x, s.x, c.y, s.y);
          turn_across(wa[w + 1], wz[w + 1], c.z, s.z, c.w, s.w);
        }
      }
    }
    uint16_t* dst;
    if (h < hq) {
      dst = p.q_out + (size_t)b * p.q_out_stride + h * D;
    } else {
      const bool is_k = h < hq + p.hkv;
      const int g = h - hq - (is_k ? 0 : p.hkv);
      const int64_t row0 = tile_first_row(p.layout, page, g, p.hkv, p.num_pages, p.maxp);
      dst = (is_k ? p.k_pool : p.v_pool) + ((size_t)row0 + in_page) * D;
    }
    *reinterpret_cast<uint4*>(dst + 8 * ca) = a;
    *reinterpret_cast<uint4*>(dst + 8 * cb) = z;
  }
}

template <int D>
cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream) {
  const int units = ((p.q ? p.hq : 0) + 2 * p.hkv) * (D / 16);
  const int threads = units >= 512 ? 512 : (units + 31) / 32 * 32;
  return p.rotary.interleaved
             ? launch_pdl(rotary_append_kernel<D, true>, dim3(p.rows), dim3(threads), 0, stream, p)
             : launch_pdl(rotary_append_kernel<D, false>, dim3(p.rows), dim3(threads), 0, stream,
                          p);
}

cudaError_t launch_rotary_append(const RotaryParams& p, int head_dim, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  return head_dim == 64 ? launch_rotary<64>(p, stream) : launch_rotary<128>(p, stream);
}

}  // namespace pgd
