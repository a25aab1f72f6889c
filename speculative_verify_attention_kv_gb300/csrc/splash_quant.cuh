// The cache's row quantiser as splash_qkv_append uses it. splash_kv_append divides
// every value: with fewer instructions around it, the quotients below gain little
// and lose where values are next to a border (32768 tokens of 4 heads of 256: fp32
// 70 us instead of 82, bf16 82 either way, rows of zeros 73 instead of 67, of zeros and
// NaN 88 instead of 67; 256 bf16 tokens 5.0 instead of 4.1).
//
// A row of D values is spread over LPR lanes of a warp (EPL = D / LPR
// consecutive values a lane): a = max |x| over the row's lanes, s = fl32(a/127),
// code = clamp(rne(fl32(x / s)), -127, 127), all zero where s == 0. Scale and
// quotient are correctly rounded fp32 divisions (no fast-math in the including
// translation units), rounding is half-to-even (cvt.rni).
#pragma once

#include "splash_common.cuh"

namespace splash {

// Two fp32 values and the operations on both (each rounded like the scalar one).
using F2 = unsigned long long;
__device__ inline F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ inline void split(F2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ inline F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ inline F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ inline F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The definition itself. Not inlined: few rows need it, and its divisions would
// fill the instruction cache.
static __device__ __noinline__ uint32_t code_exact(float x, float s) {
  return s != 0.f ? (uint32_t)max(-127, min(127, __float2int_rn(__fdiv_rn(x, s)))) : 0u;
}

// Codes of EPL values for scale s, four to a word. The quotient is first taken as
// x * fl(1/s), off by at most 127 * 2^-23 from x / s, and rounded by adding 1.5 *
// 2^23; fl32(x / s) itself is off by at most 127 * 2^-24. Together that is below
// 2.4e-5, so a value whose fraction is further than 4e-5 from a half has the
// same code either way. The others (of random fp32 values one in 12500) are divided,
// and so are products that are not finite (infinite and NaN values). Where s = 0, the
// reciprocal is taken as 0, and so are the codes: a row of zeros, or a lane that has
// no head.
template <int EPL>
__device__ inline void quantise(const float (&x)[EPL], float s, uint32_t (&packed)[(EPL + 3) / 4]) {
  constexpr float kRound = 12582912.f;
  const float inv = s != 0.f ? __frcp_rn(s) : 0.f;
  uint32_t c[EPL];
  bool sure = true;
#pragma unroll
  for (int i = 0; i < EPL; i += 2) {
    const F2 q = mul2(f2(x[i], x[i + 1]), f2(inv, inv)), t = add2(q, f2(kRound, kRound));
    // q - (t - 1.5 * 2^23): both differences are exact
    const F2 d = fma2(add2(t, f2(-kRound, -kRound)), f2(-1.f, -1.f), q);
    float t0, t1, d0, d1;
    split(t, t0, t1);
    split(d, d0, d1);
    sure = sure && fabsf(d0) <= 0.49996f && fabsf(d1) <= 0.49996f;
    c[i] = __float_as_uint(t0);
    c[i + 1] = __float_as_uint(t1);
  }
  if (!sure) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float q = __fmul_rn(x[i], inv), n = __fsub_rn(__fadd_rn(q, kRound), kRound);
      if (!(fabsf(__fsub_rn(q, n)) <= 0.49996f)) c[i] = code_exact(x[i], s);
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; i += 4) {
    const uint32_t lo = __byte_perm(c[i], c[i + 1], 0x0040);
    const uint32_t hi = EPL > 2 ? __byte_perm(c[i + (EPL > 2 ? 2 : 0)], c[i + (EPL > 2 ? 3 : 0)], 0x0040) : 0u;
    packed[i / 4] = __byte_perm(lo, hi, 0x5410);
  }
}

}  // namespace splash
