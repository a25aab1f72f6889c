// The cache's row quantiser, shared by the appends.
//
// A row of D values is spread over LPR lanes of a warp (EPL = D / LPR
// consecutive values a lane): a = max |x| over the row's lanes, s = fl32(a/127),
// code = clamp(rne(fl32(x / s)), -127, 127), all zero where s == 0. Scale and
// quotient are correctly rounded fp32 divisions (no fast-math in the including
// translation units), rounding is half-to-even (cvt.rni).
#pragma once

#include "splash_common.cuh"

namespace splash {

// Writes EPL codes as one store and, from the row's first lane, the scale.
// `a` is the row's absmax, already reduced over the row's lanes.
template <int EPL>
__device__ inline void store_codes(const float (&x)[EPL], float a, int8_t* codes_dst,
                                   float* scale_dst, bool first_lane) {
  const float s = __fdiv_rn(a, 127.0f);
  uint32_t packed[(EPL + 3) / 4] = {};
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    int c = 0;
    if (s != 0.f) {
      c = __float2int_rn(__fdiv_rn(x[i], s));
      c = max(-127, min(127, c));
    }
    packed[i / 4] |= (uint32_t)(c & 0xff) << (8 * (i % 4));
  }
  if constexpr (EPL == 2) {
    *reinterpret_cast<uint16_t*>(codes_dst) = (uint16_t)packed[0];
  } else if constexpr (EPL == 4) {
    *reinterpret_cast<uint32_t*>(codes_dst) = packed[0];
  } else {
    *reinterpret_cast<uint2*>(codes_dst) = make_uint2(packed[0], packed[1]);
  }
  if (first_lane) *scale_dst = s;
}

}  // namespace splash
