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
  float cap_in;   // scale / softcap (0: no cap)
  float cap_out;  // softcap * log2(e): capped scores in log2 units
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
  if (p.prefix_len) s.hi = max(n, p.prefix_len[row] - 1);
  s.lo = p.window > 0 ? max(n - p.window + 1, 0) : 0;
  if (p.first_key) s.lo = max(s.lo, p.first_key[b]);
  return s;
}

// cap * tanh(x / cap) in log2 units for a raw score s = q . k, with a = scale /
// cap and c = scale log2 e (so cap log2 e = c / a).
//   |a s| <= 1: c s P(u), u = (a s)^2, P(u) = tanh(x) / x as a polynomial of
//   degree 5 in u, fitted here by a minimax exchange on [0, 1]: within 6e-7 of
//   it, so a score capped at 50 is off by less than 3e-5.  No special function.
//   beyond: cap (1 - 2 / (1 + 2^(2 a s log2 e))), two special functions,
//   within 2^-22 of the cap at any argument (also an infinite one).
// A warp takes the first form when all of its scores allow it: nearly always,
// scores of trained models staying well inside their cap.
constexpr float kTanh0 = 0.9999994039535522f, kTanh1 = -0.3332904279232025f,
                kTanh2 = 0.13281433284282684f, kTanh3 = -0.051605675369501114f,
                kTanh4 = 0.016743114218115807f, kTanh5 = -0.003067060373723507f;

__device__ __forceinline__ float cap_near(float s, float a, float c) {
  const float t = a * s, u = t * t;
  float q = fmaf(kTanh5, u, kTanh4);
  q = fmaf(q, u, kTanh3);
  q = fmaf(q, u, kTanh2);
  q = fmaf(q, u, kTanh1);
  q = fmaf(q, u, kTanh0);
  return (c * s) * q;
}

__device__ __forceinline__ float2 cap_near2(float2 s, float a, float c) {
  const float2 t = __fmul2_rn(make_float2(a, a), s), u = __fmul2_rn(t, t);
  float2 q = __ffma2_rn(make_float2(kTanh5, kTanh5), u, make_float2(kTanh4, kTanh4));
  q = __ffma2_rn(q, u, make_float2(kTanh3, kTanh3));
  q = __ffma2_rn(q, u, make_float2(kTanh2, kTanh2));
  q = __ffma2_rn(q, u, make_float2(kTanh1, kTanh1));
  q = __ffma2_rn(q, u, make_float2(kTanh0, kTanh0));
  return __fmul2_rn(__fmul2_rn(make_float2(c, c), s), q);
}

__device__ __forceinline__ float cap_far(float s, float a, float cap_log2) {
  constexpr float kTwoLog2e = 2.8853900817779268f;
  const float e = exp2_approx(a * s * kTwoLog2e);  // inf: the quotient is 0
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return fmaf(-2.f * cap_log2, r, cap_log2);
}

}  // namespace pgd
