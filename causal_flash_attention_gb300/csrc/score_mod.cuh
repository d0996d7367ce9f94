// Score changes of the span entry points, shared by their kernels: key spans
// as bit masks, the tanh cap and the distance bias.
#pragma once

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

// Bits [0, x) of a word, for any x.
__device__ __forceinline__ uint32_t bits_below(int x) {
  return x <= 0 ? 0u : (x >= 32 ? 0xffffffffu : (1u << x) - 1u);
}

// Bits of [lo, hi) that fall into the 32 positions from `base`.
__device__ __forceinline__ uint32_t span_bits(int lo, int hi, int base) {
  return bits_below(hi - base) & ~bits_below(lo - base);
}

// Bit matrix transpose across a warp: bit l of lane r's word becomes bit r of
// lane l's. Five exchanges of ever smaller blocks (the recursive block
// transpose).
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x, int lane) {
  uint32_t m = 0x0000ffffu;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
    x = (lane & j) ? ((x & ~m) | ((y & ~m) >> j)) : ((x & m) | ((y & m) << j));
    m ^= m << (j >> 1);   // the next, half as wide, low-half mask
  }
  return x;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + e^(2u)) with e^(2u) = 2^(cap_in * s), s the unscaled score: tanh u =
// 1 - 2r and 1 - tanh^2 u = 4 r (1 - r). Both ends are exact limits (2^x
// overflows to infinity, r = 0; underflows to 0, r = 1). tanh.approx would take
// one special-function instruction instead of two, but its relative error of
// 2^-11 is as large as the rounding of P to 16 bits; this form is off by about
// 2^-21 of the cap.
__device__ __forceinline__ float cap_r(float s, float cap_in) {
  return rcp_approx(1.f + ex2(s * cap_in));
}

// The cap by a polynomial where the warp's scores allow it, u = s * scale / softcap:
// tanh u = u (a0 + a1 w + ...), w = u^2, minimax fits (by reweighted least squares) of
// degree 9 for |u| <= 3/4, off by 2.1e-7, 2.9e-7 in fp32, and of degree 5 for
// |u| <= 0.3, off by 1.7e-7, 2.1e-7 in fp32 (of tanh u itself by 2.8e-6 and 4.0e-6 at most,
// for small u). The greatest score counts masked keys too, so a row's last bits may
// depend on what stands beside it. No special function, which the softmax is
// short of; the coefficients come with the powers of scale / softcap and softcap *
// log2(e) multiplied in, so y = softcap log2(e) tanh u directly from the unscaled score.
template <int N>
struct CapPoly {
  uint64_t a[N];
  __device__ __forceinline__ explicit CapPoly(const float (&from)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = f2_pack(from[i], from[i]);
  }
  // capped score / score, of two at a time, in paired fp32 instructions
  __device__ __forceinline__ uint64_t factor(uint64_t s) const {
    const uint64_t w = f2_mul(s, s);
    uint64_t y = a[N - 1];
#pragma unroll
    for (int k = N - 2; k >= 0; --k) y = f2_fma(w, y, a[k]);
    return y;
  }
  __device__ __forceinline__ float one(float s) const {
    const uint64_t x = f2_pack(s, s);
    float y0, y1;
    f2_unpack(f2_mul(x, factor(x)), y0, y1);
    return y0;
  }
  // scores in place
  template <int M>
  __device__ __forceinline__ void operator()(float (&s)[M]) const {
#pragma unroll
    for (int i = 0; i < M; i += 2) {
      const uint64_t x = f2_pack(s[i], s[i + 1]);
      f2_unpack(f2_mul(x, factor(x)), s[i], s[i + 1]);
    }
  }
};
// Past that, by the exponential form.
__device__ __forceinline__ float cap_exact(float s, const ScoreMod& m) {
  return fmaf(-2.f * m.cap_log2, cap_r(s, m.cap_in), m.cap_log2);
}

// The greatest |score| of a warp's, for the choice of form (a NaN stays one in each).
template <int M>
__device__ __forceinline__ float warp_abs_max(const float (&s)[M]) {
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < M; i += 2) big = fmax3(big, fabsf(s[i]), fabsf(s[i + 1]));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
}

// A warp's unscaled scores to capped ones in the log2 domain.
template <int M>
__device__ __forceinline__ void cap_scores(float (&s)[M], float big, const ScoreMod& m) {
  if (big <= m.cap_limit_b) {
    CapPoly<3>(m.cap_b)(s);
  } else if (big <= m.cap_limit_a) {
    CapPoly<5>(m.cap_a)(s);
  } else {
#pragma unroll
    for (int i = 0; i < M; ++i) s[i] = cap_exact(s[i], m);
  }
}

}  // namespace fa
