// RMS norm of rows with the residual's addition, delivered in the type the
// next product takes: fp32, bf16, int8 with block scales, MXFP8 or MXFP4.
//
//   h = x + res (the fp32 sum, rounded to res' type; h = x without res)
//   y = fp32( h * w / sqrt(mean(h^2) + eps) )
//
// The codes are those that the activation quantizers would give for y, so y
// itself has to be right to its last bit: a block exponent or a code changes
// wherever y crosses a border, and an fp32 sum taken in another order moves y
// by several units.  The sum of squares (a square of fp32 is exact in fp64),
// the root and the product are therefore fp64, rounded once to fp32.  The sum
// takes at most 31 + 6 + 16 roundings (a thread's terms, the wave, the waves), the
// mean and eps two, of which the root leaves half; with the root's own, the
// reciprocal's and the last product's (h * w is exact) y is within 2^-47 of the
// definition before it is rounded to fp32.  fp64 multiply-adds run at the rate of
// fp32 ones on this part, and the kernel stays bound by memory: 8192 x 7168 bf16 to
// MXFP8, 413 MB, in 89-92 us (4.5 TB/s; a 1 GiB copy moves 5.1).
#include <algorithm>

#include "act.hpp"

#pragma clang fp contract(off)

namespace qmoe {

struct NormParams {
  const void* x;
  const void* res;   // NULL: no addition
  void* res_out;     // may be res itself: a lane reads its values before it writes them
  const float* w;
  void* out;
  void* scales;
  double eps;
  int R, K;
};

// Sum over aligned groups of `lanes` lanes (a power of two; a wave or more: the
// wave's).
QMOE_D double lanes_sum(double v, int lanes) {
  if (lanes >= 64) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  } else {
    for (int off = lanes >> 1; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  }
  return v;
}

// tpr threads share a row (a power of two, a block's four at least), NPT octets each:
// octet o of the row belongs to thread o mod tpr.  A block takes
// blockDim.x / tpr rows at a time and goes on to later ones.  w is requested
// with the row where a thread has one or two octets (one wait for memory, few
// rows); with more it is read from the near caches after the sum, which leaves
// the registers to rows in flight.
template <int OUT, int NPT, bool XBF, int RES>
__global__ __launch_bounds__(1024) void norm_kernel(NormParams P, int tpr) {
  __shared__ double part[16];
  const int K8 = P.K >> 3;
  const int t = threadIdx.x & (tpr - 1), lrow = threadIdx.x / tpr;
  const int rows = blockDim.x / tpr;
  const int waves = tpr >> 6, wave0 = (threadIdx.x >> 6) & ~(waves - 1);  // used with two or more
  constexpr bool early = NPT <= 2;
  // uniform over the block: every thread meets the barriers the same number of times
  for (long long r0 = (long long)blockIdx.x * rows; r0 < P.R; r0 += (long long)gridDim.x * rows) {
    const bool live = r0 + lrow < P.R;
    const size_t base = (size_t)(r0 + lrow) * P.K;
    float h[NPT][8], s[NPT][8], w[early ? NPT : 1][8];
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      const int o = t + j * tpr;
      if (live && o < K8) {
        load8<XBF>(P.x, base + (size_t)o * 8, h[j]);
        if constexpr (RES != 0) load8<RES == 2>(P.res, base + (size_t)o * 8, s[j]);
        if constexpr (early) load8<false>(P.w, (size_t)o * 8, w[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = s[j][i] = 0.f;
      }
    }
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      const int o = t + j * tpr;
      if constexpr (RES != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[j][i] += s[j][i];
          if constexpr (RES == 2) h[j][i] = bf16_bits_to_f32(f32_to_bf16_bits(h[j][i]));
        }
        if (P.res_out && live && o < K8) store8<RES == 2>(P.res_out, base + (size_t)o * 8, h[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fma((double)h[j][i], (double)h[j][i], sum);
    }
    sum = lanes_sum(sum, tpr);
    if (waves > 1) {
      __syncthreads();  // the last row's sums have been read
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
      __syncthreads();
      sum = 0.0;
      for (int i = 0; i < waves; ++i) sum += part[wave0 + i];
    }
    const double scale = 1.0 / sqrt(sum / P.K + P.eps);
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      const int o = t + j * tpr;
      if (live && o < K8) {
        if constexpr (!early) load8<false>(P.w, (size_t)o * 8, w[0]);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (float)((double)h[j][i] * (double)w[early ? j : 0][i] * scale);
        store_act8<OUT>(y, base + (size_t)o * 8, P.out, P.scales);
      }
    }
  }
}

template <int OUT, int NPT, bool XBF>
static int launch_norm3(const char* name, int res, dim3 g, int block, hipStream_t s,
                        const NormParams& P, int tpr) {
  if (res == 0) return QMOE_LAUNCH(name, (norm_kernel<OUT, NPT, XBF, 0>), g, block, 0, s, P, tpr);
  if (res == 1) return QMOE_LAUNCH(name, (norm_kernel<OUT, NPT, XBF, 1>), g, block, 0, s, P, tpr);
  return QMOE_LAUNCH(name, (norm_kernel<OUT, NPT, XBF, 2>), g, block, 0, s, P, tpr);
}
template <int OUT, int NPT>
static int launch_norm2(const char* name, bool xbf, int res, dim3 g, int block, hipStream_t s,
                        const NormParams& P, int tpr) {
  return xbf ? launch_norm3<OUT, NPT, true>(name, res, g, block, s, P, tpr)
             : launch_norm3<OUT, NPT, false>(name, res, g, block, s, P, tpr);
}

template <int OUT>
static int run_norm(const char* who, const void* x, int x_dtype, const void* res, void* res_out,
                    int res_dtype, const float* w, double eps, int R, int K, void* out,
                    void* scales, void* stream) {
  constexpr int unit = OUT == kOutF32 || OUT == kOutBF16 ? 8 : 32;
  if (R < 0 || K <= 0 || K % unit || K > 32768)
    return fail(QMOE_ERR_INVALID_ARG, "%s: R=%d K=%d (K %% %d == 0, K <= 32768)", who, R, K, unit);
  if ((x_dtype != QMOE_F32 && x_dtype != QMOE_BF16) ||
      (res && res_dtype != QMOE_F32 && res_dtype != QMOE_BF16))
    return fail(QMOE_ERR_UNSUPPORTED, "%s: unknown x_dtype %d or res_dtype %d", who, x_dtype,
                res_dtype);
  if (!(eps >= 0.0)) return fail(QMOE_ERR_INVALID_ARG, "%s: eps must be at least 0", who);
  if (!res && res_out) return fail(QMOE_ERR_INVALID_ARG, "%s: res_out without res", who);
  if (R == 0) return QMOE_OK;
  constexpr bool quant = unit == 32;
  if (!x || !w || !out || (quant && !scales))
    return fail(QMOE_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!QMOE_ALIGNED(x, 16) || !QMOE_ALIGNED(w, 16) || !QMOE_ALIGNED(out, 16) ||
      !QMOE_ALIGNED(res, 16) || !QMOE_ALIGNED(res_out, 16) ||
      (OUT == kOutQ8 && !QMOE_ALIGNED(scales, 4)))
    return fail(QMOE_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  const int K8 = K >> 3, cus = std::max(1, cu_count());
  // Octets per thread.  Rows up to 4096 take one: 2048 x 2048 fp32 to MXFP8 12.3
  // us, with four 13.7; 1 x 4096 3.3 and 4.1.  Longer rows take two while there
  // are few of them (16 x 7168 bf16 4.2; one 4.5, four 5.3) and four once they
  // fill the part (8192 x 7168 92, two 95, one 97; 1024 x 7168 13.8, 14.9, 14.9):
  // fewer barriers and sums per byte.  Rows below 512 share a wave: 8192 x 256 5.5
  // us, with a wave to each 7.2.
  int npt = K8 <= 512 ? 1 : R <= 2 * cus ? 2 : 4, tpr = 4;
  while (tpr < 1024 && tpr * npt < K8) tpr *= 2;
  while (tpr * npt < K8) npt *= 2;  // longer rows than 1024 threads hold: more per thread
  const int block = std::max(tpr, 256), rows = block / tpr;
  const long long need = ((long long)R + rows - 1) / rows;
  const dim3 grid((unsigned)std::min<long long>(need, (long long)cus * (2048 / block)));
  const NormParams P{x, res, res_out, w, out, scales, eps, R, K};
  const bool xbf = x_dtype == QMOE_BF16;
  const int rk = !res ? 0 : res_dtype == QMOE_F32 ? 1 : 2;
  hipStream_t s = (hipStream_t)stream;
  if (npt == 1) return launch_norm2<OUT, 1>("norm", xbf, rk, grid, block, s, P, tpr);
  if (npt == 2) return launch_norm2<OUT, 2>("norm", xbf, rk, grid, block, s, P, tpr);
  return launch_norm2<OUT, 4>("norm", xbf, rk, grid, block, s, P, tpr);
}

}  // namespace qmoe

using namespace qmoe;

extern "C" {

int qnorm(const void* x, int x_dtype, const void* res, void* res_out, int res_dtype,
          const float* w, double eps, int R, int K, void* y, int y_dtype, void* stream) {
  if (y_dtype == QMOE_F32)
    return run_norm<kOutF32>("qnorm", x, x_dtype, res, res_out, res_dtype, w, eps, R, K, y,
                             nullptr, stream);
  if (y_dtype == QMOE_BF16)
    return run_norm<kOutBF16>("qnorm", x, x_dtype, res, res_out, res_dtype, w, eps, R, K, y,
                              nullptr, stream);
  return fail(QMOE_ERR_UNSUPPORTED, "qnorm: unknown y_dtype %d", y_dtype);
}

int qnorm_act_q8(const void* x, int x_dtype, const void* res, void* res_out, int res_dtype,
                 const float* w, double eps, int R, int K, int8_t* q, float* d, void* stream) {
  return run_norm<kOutQ8>("qnorm_act_q8", x, x_dtype, res, res_out, res_dtype, w, eps, R, K, q,
                          d, stream);
}

int qnorm_act_mxfp8(const void* x, int x_dtype, const void* res, void* res_out, int res_dtype,
                    const float* w, double eps, int R, int K, uint8_t* codes, uint8_t* scales,
                    void* stream) {
  return run_norm<kOutMx8>("qnorm_act_mxfp8", x, x_dtype, res, res_out, res_dtype, w, eps, R, K,
                           codes, scales, stream);
}

int qnorm_act_mxfp4(const void* x, int x_dtype, const void* res, void* res_out, int res_dtype,
                    const float* w, double eps, int R, int K, uint8_t* codes, uint8_t* scales,
                    void* stream) {
  return run_norm<kOutMx4>("qnorm_act_mxfp4", x, x_dtype, res, res_out, res_dtype, w, eps, R, K,
                           codes, scales, stream);
}

}  // extern "C"
