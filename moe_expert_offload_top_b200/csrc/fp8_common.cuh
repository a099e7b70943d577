// Device helpers of the fp8 kernels.
#pragma once
#include "common.cuh"

namespace ftk {

// Largest magnitude of a block, a NaN winning over every number (fmaxf would drop it).
FT_DEVICE float amax_nan(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}
// Scale of a block with largest magnitude amax: 448 is the largest e4m3 value; the floor
// 2^-126 keeps the inverse finite for a block of zeros.  A NaN stays one.
FT_DEVICE float fp8_scale(float amax) {
  const float s = amax / 448.0f;
  return s < 1.17549435e-38f ? 1.17549435e-38f : s;
}
// Two fp32 values -> two e4m3 codes (lo in the low byte): round to nearest even, saturating at +-448.
FT_DEVICE uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two fp32 values -> a bf16 pair (lo in the low half), round to nearest even, NaN kept.
FT_DEVICE uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight words to a 32-byte aligned address.
FT_DEVICE void st_sector(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// silu(a) = a / (1 + exp(-a)), to (9 + 2.4 |a|) 2^-24 of its value: __expf is good to 2 + 1.173 |a| ulp
// (the rounded product with log2 e), the sum to 2^-24, __fdividef to 2 ulp.  __fdividef gives 0
// for divisors above 2^126, and exp(-a) = inf does: below a = -87.3, where |silu(a)| < 1.1e-36,
// the result may be 0.  The loss of bits against expf and the IEEE quotient is less than the
// sums behind a have, and far below the step of the e4m3 code that h becomes; with those two the
// gate/up tiles took 12 % longer (664 against 593 us).
FT_DEVICE float silu_fast(float a) { return __fdividef(a, 1.0f + __expf(-a)); }

}  // namespace ftk
