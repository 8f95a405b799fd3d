// MXFP4 weights x MXFP4 activations on the block-scaled matrix cores, plain
// (qgemm_mxfp4_mxfp4) and with bias, activation and residual (qlinear_mxfp4).
//
//   y[r, n] = act( sum_k w[n, k] x[r, k] + bias[n] ) + res[r, n]
//
// Both operands are E2M1 codes with one E8M0 scale per 32 values along K, used
// as stored: every product of two codes is exact, the matrix op applies both
// scales and accumulates in fp32.
#include "mxcall.hpp"

#pragma clang fp contract(off)

namespace qmoe {

// Which kernel: as measured at K = 4096 (us).
//   rows   1 x 4096: 4.3, 16 x 4096: 5.1; 32 x 64: 6.6
//   32 x 64, four teams  128 x 4096: 6.9;  64 x 64: 8.5;  64 x 128: 11
//   64 x 64, four teams  64 x 14336: 10.7; 32 x 64: 15.0; 64 x 128: 14.8
//   64 x 128, two teams  512 x 4096: 11.4; 64 x 64: 14.3; 128 x 128: 13.0
//   128 x 128, two teams 256 x 14336: 15.2; 64 x 128: 20.9; 256 x 256: 28.6
//   128 x 128, two to a unit  2048 x 4096: 25.4; two teams: 30.0; 256 x 256: 30.2
//   256 x 256  2048 x 14336: 70; 128 x 128: 86
// The rule has no term for K.  Against the best of the six for R from 40 to 2048
// and N from 2048 to 14336 its choice takes at most 5 % longer at K = 4096, 6 % at
// 1024, 9 % at 14336 (700 x 4096: 40.2 and 36.9), and at 256, where the teams'
// tiles are short of steps, 22 % (700 x 14336: 13.4 and 11.0).
template <int WR, int WC, int TM, int TN, int KS>
using T4 = Tile<WR, WC, TM, TN, KS, false>;

static int run(const ProductCall& c, hipStream_t s) {
  const int st = check_product(c);
  if (st) return st == kNothing ? QMOE_OK : st;
  const MxProduct P = mx_product(c);
  const int cus = std::max(1, cu_count());
  if (P.R <= 16 && P.N <= 32 * cus) return launch_rows<false, false, 1>("mxfp4_rows", P, s);
  static constexpr Choice choices[] = {
      choice<T4<1, 2, 1, 1, 4>, false>(1, 7.f),  choice<T4<2, 2, 1, 1, 4>, false>(1, 9.5f),
      choice<T4<2, 2, 1, 2, 2>, false>(1, 11.f), choice<T4<2, 2, 2, 2, 2>, false>(1, 15.f),
      choice<T4<2, 2, 2, 2, 1>, false>(2, 25.f), choice<T4<2, 2, 4, 4, 1>, false>(1, 33.f)};
  return launch_choice(choices, c.who, "mxfp4_tile", P, s);
}

}  // namespace qmoe

using namespace qmoe;

extern "C" {

int qgemm_mxfp4_mxfp4(const void* W, int N, int K, const uint8_t* codes, const uint8_t* scales,
                      int R, void* y, int y_dtype, void* stream) {
  const ProductCall c{"qgemm_mxfp4_mxfp4", QMOE_MXFP4, W, nullptr, false, N, K, codes, scales, R,
                      nullptr, nullptr, QMOE_ACT_NONE, nullptr, 0, y, nullptr,
                      plain_dtype(y_dtype)};
  return run(c, (hipStream_t)stream);
}

int qlinear_mxfp4(const void* W, int N, int K, const uint8_t* codes, const uint8_t* scales, int R,
                  const float* bias, int act, const void* res, int res_dtype, void* y,
                  int y_dtype, void* stream) {
  const ProductCall c{"qlinear_mxfp4", QMOE_MXFP4, W, nullptr, false, N, K, codes, scales, R,
                      bias, nullptr, act, res, res_dtype, y, nullptr,
                      plain_dtype(y_dtype)};
  return run(c, (hipStream_t)stream);
}

}  // extern "C"
