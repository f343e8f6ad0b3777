// How a kernel's attention scores differ from scale * q . k: the policies the
// decode and prefill kernels are built with.  PlainScore adds nothing (the
// kernels of pgd.h); ModScore adds a tanh cap, a distance bias, a first
// visible key per token and a bidirectional prefix (include/pgd_ext.h).
#pragma once

#include <math.h>

#include "pgd_device.cuh"
#include "pgd_internal.h"

namespace pgd {

struct PlainScore {
  using Params = DecodeParams;
  static constexpr bool kMod = false;
};

struct ModParams : DecodeParams {
  float cap_in;   // a = scale / softcap (0: no cap)
  float cap_out;  // softcap * log2(e): capped scores in log2 units
  // the polynomial forms of a capped score (cap_near below): coefficients of the
  // near form with the cap and the powers of a folded in, a^2, and the raw
  // scores up to which each form holds (-1: not used)
  float near_q[3], a2, limit_near, limit_mid;
  // tcgen05 prefill: a row's first reference (log2 units; -inf: its first page's
  // maximum), by how much a score may exceed the reference before it is raised, and
  // whether scores in the cap's near form never do
  float ref_log2, slack_log2, limit_near2;  // (limit_near's square, with its sign)
  bool near_fits;
  const float* slopes;       // [Hq] or nullptr
  const int32_t* first_key;  // [rows] or nullptr
  const int32_t* prefix_len; // [table_rows] or nullptr
};

struct ModScore {
  using Params = ModParams;
  static constexpr bool kMod = true;
};

// The positions token b sees, lo .. span.hi, of table row `row` (a valid one)
// at position n >= 0; lo > hi: none.
struct TokenSpan {
  int lo, hi;
};

__device__ __forceinline__ TokenSpan mod_span(const ModParams& p, int b, int row, int n) {
  TokenSpan s;
  s.hi = n;
  if (p.prefix_len) s.hi = max(n, max(p.prefix_len[row], 0) - 1);  // (-2^31 - 1 wraps)
  s.lo = p.window > 0 ? max(n - p.window + 1, 0) : 0;
  if (p.first_key) s.lo = max(s.lo, p.first_key[b]);
  return s;
}

// cap * tanh(x / cap) in log2 units for a raw score s = q . k, with t = a s, a =
// scale / cap, and the cap in log2 units.
//   |t| <= 1: cap t P(t^2), P(u) = tanh(x) / x at x^2 = u as a polynomial of
//   degree 5 in u, fitted here by a minimax exchange on [0, 1]: within 6.2e-7
//   of it, so a score capped at 50 is off by less than 3e-5.
//   |t| <= 0.3: the same with degree 2, fitted on [0, 0.09], within 1.2e-6.
//   beyond: cap (1 - 2 / (1 + 2^(2 t log2 e))), two special functions, within
//   2^-21 of the cap at any argument (also an infinite one).
// A warp takes the shortest form that all of its scores allow: nearly always
// the first or second, scores of trained models staying well inside their cap.
constexpr float kTanhMid = 1.f, kTanhNear = 0.3f;
constexpr float kMid0 = 0.9999994039535522f, kMid1 = -0.3332904279232025f,
                kMid2 = 0.13281433284282684f, kMid3 = -0.051605675369501114f,
                kMid4 = 0.016743114218115807f, kMid5 = -0.003067060373723507f;
constexpr float kNear0 = 0.9999988675117493f, kNear1 = -0.33310022950172424f,
                kNear2 = 0.12633946537971497f;

__device__ __forceinline__ float cap_mid(float s, float a, float cap_log2) {
  const float t = a * s, u = t * t;
  float q = fmaf(kMid5, u, kMid4);
  q = fmaf(q, u, kMid3);
  q = fmaf(q, u, kMid2);
  q = fmaf(q, u, kMid1);
  q = fmaf(q, u, kMid0);
  return (cap_log2 * t) * q;
}

__device__ __forceinline__ float cap_far(float s, float a, float cap_log2) {
  constexpr float kTwoLog2e = 2.8853900817779268f;
  const float e = exp2_approx(a * s * kTwoLog2e);  // inf: the quotient is 0
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return fmaf(-2.f * cap_log2, r, cap_log2);
}

}  // namespace pgd
