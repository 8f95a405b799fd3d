// Activations between products: the MXFP4 quantizer and its read-back, and
// SwiGLU delivered in the type the down product takes.  All three read and
// write every value once, eight consecutive values to a lane (act.hpp).
//  * qquantize_act_mxfp4: per 32 values along K, E = floor(log2 max|x|) - 2,
//    stored as E + 127 (at least 0); codes = the E2M1 values nearest to
//    x / 2^E, ties to even, saturating at 6: the rule of the MXFP4 weights.
//  * qswiglu_act_*: v = fp32( gate / (1 + exp(-gate)) * up ), quantized.
#include <algorithm>

#include "act.hpp"

#pragma clang fp contract(off)

namespace qmoe {

template <bool XBF>
__global__ __launch_bounds__(256) void quantize_act_mxfp4_kernel(const void* x, size_t n8,
                                                                 void* codes, void* scales) {
  const size_t o = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (o >= n8) return;  // n8 is a multiple of 4: a block's four lanes leave together
  float v[8];
  load8<XBF>(x, o * 8, v);
  store_act8<kOutMx4>(v, o * 8, codes, scales);
}

template <bool YBF>
__global__ __launch_bounds__(256) void dequantize_act_mxfp4_kernel(const uint8_t* codes,
                                                                   const uint8_t* scales,
                                                                   size_t n8, void* y) {
  const size_t o = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (o >= n8) return;
  const uint32_t c = ((const uint32_t*)codes)[o];
  const float s = e8m0_to_f32(scales[o >> 2]);
  typedef float v2f __attribute__((ext_vector_type(2)));
  const v2f p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 0),
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 1),
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 2),
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 3)};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = p[i].x * s;
    v[2 * i + 1] = p[i].y * s;
  }
  store8<YBF>(y, o * 8, v);
}

// gate / (1 + exp(-gate)) * up in fp64, so that its one rounding to fp32 is
// the correct one but for values within 2^-40 of a border.  exp(z), z = -gate:
// z = n ln 2 + r, |r| <= ln 2 / 2, the Taylor series of exp(r) to r^13 / 13!
// (the next term is below 2^-56) and n added to the exponent.  z is kept in
// [-60, 700]: below, 1 + exp(z) is 1 in fp64; above, the quotient is 0 in fp32
// for every finite gate and up.
QMOE_D float swiglu1(float g, float u) {
  const double z = fmin(fmax(-(double)g, -60.0), 700.0);
  // adding 1.5 * 2^52 rounds to an integer, which the sum's low word holds
  const double sum = fma(z, 1.4426950408889634, 6755399441055744.0);
  const int32_t ni = (int32_t)(uint32_t)__builtin_bit_cast(uint64_t, sum);
  const double n = sum - 6755399441055744.0;
  double r = fma(n, -0x1.62e42fefa4000p-1, z);  // ln 2 to 40 bits: n times it is exact
  r = fma(n, 0x1.8432a1b0e2634p-43, r);               // and the rest (Cody and Waite's reduction)
  constexpr double c[14] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720,
                            1.0 / 5040, 1.0 / 40320, 1.0 / 362880, 1.0 / 3628800,
                            1.0 / 39916800, 1.0 / 479001600, 1.0 / 6227020800};
  double p = c[13];
#pragma unroll
  for (int i = 12; i >= 0; --i) p = fma(p, r, c[i]);
  const uint64_t bits = __builtin_bit_cast(uint64_t, p) + ((uint64_t)(uint32_t)ni << 52);
  const double den = 1.0 + __builtin_bit_cast(double, bits);
  // the hardware's reciprocal, within 2^-20, and two Newton steps: 2^-80 but
  // for their own rounding
  double y = __builtin_amdgcn_rcp(den);
  y = fma(fma(-den, y, 1.0), y, y);
  y = fma(fma(-den, y, 1.0), y, y);
  return (float)((double)g * (double)u * y);
}

// The same in fp32, within kGluErr of it (relative) for finite results of
// ordinary size and gate > -87: Cody and Waite's reduction in base 2, -gate log2 e
// = n + f with log2 e in two parts (f within 2^-25), the hardware's exp2 and
// reciprocal (an ulp, 2^-23, each) and four roundings (2^-24 each) come to less
// than 2^-20.9.
constexpr float kGluErr = 0x1p-20f;
QMOE_D float swiglu1_near(float g, float u) {
  const float n = __builtin_rintf(g * -1.44269502f);
  float f = fmaf(g, -1.44269502f, -n);
  f = fmaf(g, -1.92596303e-8f, f);
  const float den = 1.f + ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
  return g * u * __builtin_amdgcn_rcpf(den);
}

struct GluParams {
  const void* gate;
  const void* up;
  long long ld;  // values between rows of gate and up
  void* out;
  void* scales;
  uint32_t n8, K8;
};

// fp64 throughout is bound by its arithmetic: 48 us at 2048 x 14336 (bf16 to
// MXFP4; fp32 input 53).  An MX code, though, hardly ever depends on the last
// bits: the fp32 value's neighbours at +-kGluErr have the same exponent and
// code but for about one value in 10^5.  Where they differ, or the value is not
// an ordinary one, the block's four lanes compute theirs in fp64; the result is
// the fp64 one everywhere, in 30 us (4.5 TB/s; fp32 input 44).  int8 takes fp64
// throughout, 50-54 us (fp32 input 55-59): its scale carries every bit of the
// block's largest value.  Of the other 31 only those near a half would need it;
// no kernel here tells them apart.
template <int OUT, bool XBF>
__global__ __launch_bounds__(256) void swiglu_act_kernel(GluParams P) {
  const uint32_t o = blockIdx.x * 256 + threadIdx.x;
  if (o >= P.n8) return;
  const uint32_t row = o / P.K8, col = o - row * P.K8;
  const size_t at = (size_t)row * P.ld + (size_t)col * 8;
  float g[8], u[8], v[8];
  load8<XBF>(P.gate, at, g);
  load8<XBF>(P.up, at, u);
  if constexpr (OUT != kOutQ8) {
    float least = __builtin_inff(), gate = __builtin_inff(), lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = swiglu1_near(g[i], u[i]);
      least = fminf(least, fabsf(v[i]));
      gate = fminf(gate, g[i]);
      lo[i] = v[i] * (1.f - kGluErr);
      hi[i] = v[i] * (1.f + kGluErr);
    }
    const uint32_t m = block_max_bits(v);  // a NaN or infinity is above 2^100
    const float top = __builtin_bit_cast(float, m);
    const int e = mx_exponent<OUT>(__builtin_bit_cast(uint32_t, top * (1.f - kGluErr)));
    const int e_hi = mx_exponent<OUT>(__builtin_bit_cast(uint32_t, top * (1.f + kGluErr)));
    const uint2 c = mx_codes8<OUT>(lo, mx_over(e)), c_hi = mx_codes8<OUT>(hi, mx_over(e));
    uint32_t odd = !(top < 0x1p100f) || !(least > 0x1p-120f) || !(gate > -87.f) || e != e_hi ||
                   c.x != c_hi.x || c.y != c_hi.y;
    odd |= dpp_u32<0xB1, 0xF>(0u, odd);  // any of the block's lanes
    odd |= dpp_u32<0x4E, 0xF>(0u, odd);
    if (!odd) {
      store_mx8<OUT>(c, e, (size_t)o * 8, P.out, P.scales);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = swiglu1(g[i], u[i]);
  store_act8<OUT>(v, (size_t)o * 8, P.out, P.scales);
}

template <int OUT>
static int run_swiglu(const char* who, const void* gate, const void* up, int x_dtype,
                      long long ld, int R, int K, void* out, void* scales, void* stream) {
  if (R < 0 || K <= 0 || K % 32 || ld < K || ld % 8)
    return fail(QMOE_ERR_INVALID_ARG, "%s: R=%d K=%d ld=%lld (K %% 32 == 0, ld >= K, ld %% 8 == 0)",
                who, R, K, ld);
  if (x_dtype != QMOE_F32 && x_dtype != QMOE_BF16)
    return fail(QMOE_ERR_UNSUPPORTED, "%s: unknown x_dtype %d", who, x_dtype);
  const long long n8 = (long long)R * (K / 8);
  if (n8 > 0xFFFFFF00LL) return fail(QMOE_ERR_UNSUPPORTED, "%s: R * K beyond 2^35", who);
  if (R == 0) return QMOE_OK;
  if (!gate || !up || !out || !scales) return fail(QMOE_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!QMOE_ALIGNED(gate, 16) || !QMOE_ALIGNED(up, 16) || !QMOE_ALIGNED(out, 16) ||
      (OUT == kOutQ8 && !QMOE_ALIGNED(scales, 4)))
    return fail(QMOE_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  const GluParams P{gate, up, ld, out, scales, (uint32_t)n8, (uint32_t)(K / 8)};
  const dim3 grid((unsigned)((n8 + 255) / 256));
  hipStream_t s = (hipStream_t)stream;
  if (x_dtype == QMOE_BF16)
    return QMOE_LAUNCH("swiglu_act", (swiglu_act_kernel<OUT, true>), grid, 256, 0, s, P);
  return QMOE_LAUNCH("swiglu_act", (swiglu_act_kernel<OUT, false>), grid, 256, 0, s, P);
}

}  // namespace qmoe

using namespace qmoe;

extern "C" {

int qquantize_act_mxfp4(const void* x, int x_dtype, int R, int K, uint8_t* codes,
                        uint8_t* scales, void* stream) {
  if (R < 0 || K <= 0 || K % 32)
    return fail(QMOE_ERR_INVALID_ARG, "qquantize_act_mxfp4: R=%d K=%d (K %% 32 != 0)", R, K);
  if (x_dtype != QMOE_F32 && x_dtype != QMOE_BF16)
    return fail(QMOE_ERR_UNSUPPORTED, "qquantize_act_mxfp4: unknown x_dtype %d", x_dtype);
  const long long n8 = (long long)R * (K / 8);
  if (n8 > 0xFFFFFF00LL)
    return fail(QMOE_ERR_UNSUPPORTED, "qquantize_act_mxfp4: R * K beyond 2^35");
  if (R == 0) return QMOE_OK;
  if (!x || !codes || !scales)
    return fail(QMOE_ERR_INVALID_ARG, "qquantize_act_mxfp4: null pointer");
  if (!QMOE_ALIGNED(x, 16) || !QMOE_ALIGNED(codes, 16))
    return fail(QMOE_ERR_INVALID_ARG, "qquantize_act_mxfp4: misaligned x/codes");
  const dim3 grid((unsigned)((n8 + 255) / 256));
  hipStream_t s = (hipStream_t)stream;
  if (x_dtype == QMOE_BF16)
    return QMOE_LAUNCH("quantize_act_mxfp4", quantize_act_mxfp4_kernel<true>, grid, 256, 0, s, x,
                       (size_t)n8, codes, scales);
  return QMOE_LAUNCH("quantize_act_mxfp4", quantize_act_mxfp4_kernel<false>, grid, 256, 0, s, x,
                     (size_t)n8, codes, scales);
}

int qdequant_act_mxfp4(const uint8_t* codes, const uint8_t* scales, int R, int K, void* y,
                       int y_dtype, void* stream) {
  if (R < 0 || K <= 0 || K % 32)
    return fail(QMOE_ERR_INVALID_ARG, "qdequant_act_mxfp4: R=%d K=%d (K %% 32 != 0)", R, K);
  if (y_dtype != QMOE_F32 && y_dtype != QMOE_BF16)
    return fail(QMOE_ERR_UNSUPPORTED, "qdequant_act_mxfp4: unknown y_dtype %d", y_dtype);
  const long long n8 = (long long)R * (K / 8);
  if (n8 > 0xFFFFFF00LL)
    return fail(QMOE_ERR_UNSUPPORTED, "qdequant_act_mxfp4: R * K beyond 2^35");
  if (R == 0) return QMOE_OK;
  if (!codes || !scales || !y)
    return fail(QMOE_ERR_INVALID_ARG, "qdequant_act_mxfp4: null pointer");
  if (!QMOE_ALIGNED(codes, 16) || !QMOE_ALIGNED(y, 16))
    return fail(QMOE_ERR_INVALID_ARG, "qdequant_act_mxfp4: misaligned codes/y");
  const dim3 grid((unsigned)((n8 + 255) / 256));
  hipStream_t s = (hipStream_t)stream;
  if (y_dtype == QMOE_BF16)
    return QMOE_LAUNCH("dequantize_act_mxfp4", dequantize_act_mxfp4_kernel<true>, grid, 256, 0,
                       s, codes, scales, (size_t)n8, y);
  return QMOE_LAUNCH("dequantize_act_mxfp4", dequantize_act_mxfp4_kernel<false>, grid, 256, 0, s,
                     codes, scales, (size_t)n8, y);
}

int qswiglu_act_q8(const void* gate, const void* up, int x_dtype, long long ld, int R, int K,
                   int8_t* q, float* d, void* stream) {
  return run_swiglu<kOutQ8>("qswiglu_act_q8", gate, up, x_dtype, ld, R, K, q, d, stream);
}

int qswiglu_act_mxfp8(const void* gate, const void* up, int x_dtype, long long ld, int R, int K,
                      uint8_t* codes, uint8_t* scales, void* stream) {
  return run_swiglu<kOutMx8>("qswiglu_act_mxfp8", gate, up, x_dtype, ld, R, K, codes, scales,
                             stream);
}

int qswiglu_act_mxfp4(const void* gate, const void* up, int x_dtype, long long ld, int R, int K,
                      uint8_t* codes, uint8_t* scales, void* stream) {
  return run_swiglu<kOutMx4>("qswiglu_act_mxfp4", gate, up, x_dtype, ld, R, K, codes, scales,
                             stream);
}

}  // extern "C"
