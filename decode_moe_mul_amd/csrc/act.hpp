// Internal header: activations handled eight consecutive values to a lane (an
// "octet"), and their conversion to the output types the quantized products
// take.  Four neighbouring lanes hold one 32-value block, so a block's largest
// magnitude is two DPP steps away, a wave's loads and stores are contiguous,
// and no lane walks a block by itself.
//
// A block that holds a NaN or an infinity is marked as a whole: scale byte 255
// (E8M0's NaN) and zero codes, or d = NaN and zero int8 codes, so that every
// value read from it and every product with it is NaN.
#pragma once
#include "common.hpp"

namespace qmoe {

enum ActOut { kOutF32 = 0, kOutBF16 = 1, kOutQ8 = 2, kOutMx8 = 3, kOutMx4 = 4 };

QMOE_D uint32_t f32_to_bf16_bits(float v) {  // nearest even; NaN stays a NaN
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}
QMOE_D uint32_t pack_bf16(float lo, float hi) {
  return f32_to_bf16_bits(lo) | (f32_to_bf16_bits(hi) << 16);
}

// eight values from a 16-byte aligned place
template <bool BF>
QMOE_D void load8(const void* x, size_t at, float (&v)[8]) {
  if constexpr (BF) {
    const uint4 q = *(const uint4*)((const uint16_t*)x + at);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_bits_to_f32(w[j] & 0xFFFFu);
      v[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
    }
  } else {
    const float4 a = ((const float4*)((const float*)x + at))[0];
    const float4 b = ((const float4*)((const float*)x + at))[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

template <bool BF>
QMOE_D void store8(void* y, size_t at, const float (&v)[8]) {
  if constexpr (BF) {
    *(uint4*)((uint16_t*)y + at) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    float4* p = (float4*)((float*)y + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// The largest |v| of a 32-value block as fp32 bits, from its four lanes (all
// four must be active).  Bits of magnitudes compare as unsigned integers, and
// a NaN's are above infinity's, so it is not lost as fmaxf would lose it.
QMOE_D uint32_t block_max_bits(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
  m = max(m, dpp_u32<0xB1, 0xF>(0u, m));  // quad_perm [1, 0, 3, 2]
  m = max(m, dpp_u32<0x4E, 0xF>(0u, m));  // quad_perm [2, 3, 0, 1]
  return m;
}

// Eight values over their block's scale as MX codes, saturating: clamping first
// makes the conversions (nearest even) saturate.  `top`: the type's largest value.
// The sign bit is v < 0, also where v over the scale is below fp32's smallest
// number: of a multiply-add with 0 only the exact product is rounded, so that a
// negative v stays negative (at least as -0) and a negative zero becomes +0.  A
// product and a sum would make +0 of both.
template <int OUT>
QMOE_D uint2 mx_codes8(const float (&v)[8], float mul) {
  constexpr float top = OUT == kOutMx8 ? 448.f : 6.f;
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = __builtin_amdgcn_fmed3f(fmaf(v[i], mul, 0.f), -top, top);
  if constexpr (OUT == kOutMx8) {
    int w0 = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], w0, true);
    int w1 = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], 0, false);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], w1, true);
    return make_uint2((uint32_t)w0, (uint32_t)w1);
  } else {
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, t[0], t[1], 1.f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[2], t[3], 1.f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[4], t[5], 1.f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[6], t[7], 1.f, 3);
    return make_uint2(w, 0);
  }
}

// E8M0 byte of a block from its largest magnitude's bits: the exponent field
// less the element type's largest exponent (zero and fp32 subnormals: 0).
template <int OUT>
QMOE_D int mx_exponent(uint32_t max_bits) {
  return max((int)(max_bits >> 23) - (OUT == kOutMx8 ? 8 : 2), 0);
}
// 2^-(e - 127), an fp32 normal for every byte in 0..252
QMOE_D float mx_over(int e) { return __builtin_bit_cast(float, (uint32_t)(254 - e) << 23); }

template <int OUT>
QMOE_D void store_mx8(uint2 codes, int e, size_t at, void* out, void* scales) {
  if constexpr (OUT == kOutMx8) *(uint2*)((uint8_t*)out + at) = codes;
  else *(uint32_t*)((uint8_t*)out + (at >> 1)) = codes.x;
  if ((threadIdx.x & 3) == 0) ((uint8_t*)scales)[at >> 5] = (uint8_t)e;
}

// m / 127 rounded to nearest.  The fp64 product with 1 / 127 is within 2^-52 of the
// quotient, and no quotient is nearer than 2^-32 to a border between two fp32
// numbers: in halves of the quotient's last place, 127 times a border is an odd
// number below 2^32, and m an even one.  (Norm 8192 x 7168 to int8 97.8 us; with an
// fp32 division 98.9.)
QMOE_D float over_127(float m) { return (float)((double)m * (1.0 / 127.0)); }

// Eight int8 codes: the fp32 quotients v / d rounded half away from zero.  With
// the reciprocal of d rounded to nearest (one division), a quotient is the
// product, corrected once by its exact remainder: rounded to nearest by
// Markstein's theorem, and a third of eight divisions' work (norm 8192 x 7168 to
// int8 106 us with those).  Small d are scaled up first, exactly, to keep the
// remainder above the subnormals.
QMOE_D void q8_codes8(const float (&v)[8], float d, uint32_t (&w)[2]) {
  const float up = d < 0x1p-60f ? 0x1p90f : 1.f, ds = d * up, rd = 1.f / ds;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = v[i] * up, q1 = a * rd, q = fmaf(fmaf(-q1, ds, a), rd, q1);
    const float t = truncf(q);
    const float c = t + (fabsf(q - t) >= 0.5f ? copysignf(1.f, q) : 0.f);
    w[i >> 2] |= ((uint32_t)(int)__builtin_amdgcn_fmed3f(c, -127.f, 127.f) & 0xFFu)
                 << (8 * (i & 3));
  }
}

// Store one octet of row-major [R, K] values at flat index `at` (a multiple
// of 8) in the output type.  Every lane of the block's four calls this.
//  * MX: codes of v / 2^E, E from the block's largest magnitude; scaling by a
//    power of two is exact but for values that vanish beside the block's largest.
//  * int8: d = max / 127 (fp32), q = the quotient v / d (fp32) rounded half away
//    from zero: qquantize_act_q8's rule.
template <int OUT>
QMOE_D void store_act8(const float (&v)[8], size_t at, void* out, void* scales) {
  if constexpr (OUT == kOutF32 || OUT == kOutBF16) {
    store8<OUT == kOutBF16>(out, at, v);
  } else {
    const uint32_t m = block_max_bits(v);
    const bool bad = m >= 0x7F800000u;
    const bool first = (threadIdx.x & 3) == 0;
    if constexpr (OUT == kOutQ8) {
      const float d = over_127(__builtin_bit_cast(float, m));
      uint32_t w[2] = {0, 0};
      q8_codes8(v, d, w);
      if (!(d > 0.f) || bad) w[0] = w[1] = 0;
      *(uint2*)((int8_t*)out + at) = make_uint2(w[0], w[1]);
      if (first) ((float*)scales)[at >> 5] = bad ? __builtin_nanf("") : d;
    } else {
      const int e = mx_exponent<OUT>(m);
      const uint2 c = mx_codes8<OUT>(v, mx_over(e));
      store_mx8<OUT>(bad ? make_uint2(0, 0) : c, bad ? 255 : e, at, out, scales);
    }
  }
}

}  // namespace qmoe
