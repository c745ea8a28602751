// The 8-bit row format: e4m3 codes with one power-of-two fp32 scale per 128
// consecutive columns of a row.
//
// scale = the smallest power of two s >= 2^-126 with amax / s <= 448 (the
// largest e4m3 value), code = e4m3(v / s), rounded to nearest even.  A floating
// format loses nothing to a power-of-two scale (its relative precision is the
// same everywhere in its normal range), and dividing by one is exact: a code
// carries one rounding, and every implementation finds the same one.
//
// An infinity makes its block's scale infinite and the block's codes 0 or NaN,
// so the whole block stands for NaN; a NaN does not take part in amax and stays
// the NaN of its own place.
#pragma once

#include "kernels.cuh"
#include "ptx.cuh"

namespace ql {

constexpr int kFp8Block = 128;  // columns per scale of a row; a weight has one per 128 x 128 block

// amax (>= 0, NaN ignored) -> scale and its reciprocal, both exact.
// amax = m 2^k with 1 <= m < 2 and 448 = 1.75 * 2^8, so the exponent is k - 8,
// plus one where m > 1.75 (the addition below carries into the exponent then).
QL_DEV void fp8_scale(float amax, float& scale, float& inv) {
  const uint32_t bits = __float_as_uint(amax);
  int e = static_cast<int>((bits + 0x1FFFFFu) >> 23) - 8;
  e = e < 1 ? 1 : e;
  const bool inf = bits == 0x7F800000u;
  scale = __uint_as_float(inf ? 0x7F800000u : static_cast<uint32_t>(e) << 23);
  inv = __uint_as_float(inf ? 0u : static_cast<uint32_t>(254 - e) << 23);
}
// Largest magnitude of the 16 lanes that hold one block of 128 columns (8 each).
QL_DEV float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
QL_DEV uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
QL_DEV uint2 e4m3x8(const float (&f)[8], float inv) {
  uint2 o;
  o.x = e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16);
  o.y = e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16);
  return o;
}
QL_DEV void unpack_bf16x8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
QL_DEV uint4 pack_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
QL_DEV float absmax8(const float (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}

}  // namespace ql
