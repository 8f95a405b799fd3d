// MXFP4 weights x MXFP8 activations with bias, activation and residual
// (qlinear_mxfp8).
//
//   y[r, n] = act( sum_k w[n, k] x[r, k] + bias[n] ) + res[r, n]
//
// E2M1 codes against E4M3 codes, one E8M0 scale per 32 values along K on either
// side, used as stored: every product of two codes is exact, the matrix op applies
// both scales and accumulates in fp32.  It is issued twice, for the small and the large
// codes, because one op drops what lies far below its largest product (split_e4m3): twice
// the matrix work, 2048 x 4096 x 4096 from 39 to 62 us.
#include "mxcall.hpp"

#pragma clang fp contract(off)

namespace qmoe {

template <int WR, int WC, int TM, int TN, int KS>
using T8 = Tile<WR, WC, TM, TN, KS, true>;

// Which kernel: as measured at K = 4096 with bf16 results (us; fp32 takes up to 3 % more).
//   rows  1 x 4096: 3.8
//   32 x 64, four teams    128 x 4096: 8.6; 64 x 64: 11.7; 64 x 128: 14.5
//   64 x 64, three teams   333 x 2050 (K = 7200): 20.4; 32 x 64: 26.9; 64 x 128: 26.2
//   64 x 128, two teams    700 x 4096: 30.3; 64 x 64: 35.3
//   128 x 128              700 x 4096: 27.1; 2048 x 4096: 61.6, 64 x 128: 71.4;
//                          2048 x 14336: 208, 64 x 128: 243
// 128 x 256 takes two of 128 x 128's rounds and more (2048 x 4096 4 %, 2048 x 14336
// 15 %): it is not here.
// (An activation row has 256 bytes a step: LDS holds no two of the largest tile.)
// Against the best of the four for R from 40 to 2048, N from 2048 to 14336 and K from
// 1024 to 14336 (51 sizes) the choice takes at most 7 % longer.
static int run(const ProductCall& c, hipStream_t s) {
  const int st = check_product(c);
  if (st) return st == kNothing ? QMOE_OK : st;
  const MxProduct P = mx_product(c);
  const int cus = std::max(1, cu_count());
  if (P.R <= 16 && P.N <= 32 * cus) return launch_rows<true, false, 1>("mxfp8_rows", P, s);
  static constexpr Choice choices[] = {
      choice<T8<1, 2, 1, 1, 4>, false>(1, 9.f), choice<T8<2, 2, 1, 1, 3>, false>(1, 13.2f),
      choice<T8<2, 2, 1, 2, 2>, false>(1, 16.3f), choice<T8<2, 2, 2, 2, 1>, false>(1, 29.f)};
  return launch_choice(choices, c.who, "mxfp8_tile", P, s);
}

}  // namespace qmoe

using namespace qmoe;

extern "C" int qlinear_mxfp8(const void* W, int N, int K, const uint8_t* codes,
                             const uint8_t* scales, int R, const float* bias, int act,
                             const void* res, int res_dtype, void* y, int y_dtype,
                             void* stream) {
  const ProductCall c{"qlinear_mxfp8", QMOE_MXFP4, W, nullptr, false, N, K, codes, scales, R,
                      bias, nullptr, act, res, res_dtype, y, nullptr, plain_dtype(y_dtype)};
  return run(c, (hipStream_t)stream);
}
