// The gated pair of products of MXFP4 weights with MXFP8 activations (qglu_mxfp8,
// qglu_mxfp8_act).
//
//   v[r, n] = act( sum_k wg[n, k] x[r, k] + bg[n] ) * ( sum_k wu[n, k] x[r, k] + bu[n] )
//
// One pass over the activations for both weights; gate and up meet in the registers
// that hold their sums and never go to memory.  v leaves in fp32, bf16 or as MXFP8
// activations of the next product: the fp32 v, quantized.
#include "mxcall.hpp"

#pragma clang fp contract(off)

namespace qmoe {

template <int WR, int WC, int TM, int TN, int KS>
using T8 = Tile<WR, WC, TM, TN, KS, true>;

// Which kernel: as measured at K = 4096 with bf16 results (us; N counts the pair's
// columns; every product is two matrix ops, as in qlinear_mxfp8).
//   32 x 64, three teams  64 x 2048 (K = 7168): 17.1; 64 x 64: 22.0; 128 x 64: 42.2
//   64 x 64, two teams    333 x 2048 (K = 7168): 24.4; 32 x 64: 35.8; 128 x 64: 42.3
//   128 x 64              700 x 2048 (K = 7168): 44.3; 64 x 64: 48.6
//                         2048 x 14336: 422, 64 x 64: 478; quantized 421, fp32 428
// 128 x 128 takes two of 128 x 64's rounds (3 % more at 2048 x 14336): it is not here.
// Against the best of the three for R from 40 to 2048, N from 2048 to 14336 and K from
// 1024 to 14336 (51 sizes) the choice takes at most 6 % longer.
static int run(const ProductCall& c, hipStream_t s) {
  const int st = check_product(c);
  if (st) return st == kNothing ? QMOE_OK : st;
  const MxProduct P = mx_product(c);
  const int cus = std::max(1, cu_count());
  if (P.R <= 16 && P.N <= 32 * cus)
    return P.e.out > kOutBF16 ? launch_rows<true, true, 2>("mxfp8_glu_rows", P, s)
                              : launch_rows<true, true, 1>("mxfp8_glu_rows", P, s);
  static constexpr Choice choices[] = {choice<T8<1, 2, 1, 2, 3>, true>(1, 12.f),
                                       choice<T8<2, 2, 1, 2, 2>, true>(1, 16.3f),
                                       choice<T8<2, 2, 2, 2, 1>, true>(1, 29.3f)};
  return launch_choice(choices, c.who, "mxfp8_glu_tile", P, s);
}

}  // namespace qmoe

using namespace qmoe;

extern "C" {

int qglu_mxfp8(const void* Wg, const void* Wu, int N, int K, const uint8_t* codes,
               const uint8_t* scales, int R, const float* bias_gate, const float* bias_up, int act,
               void* y, int y_dtype, void* stream) {
  const ProductCall c{"qglu_mxfp8", QMOE_MXFP4, Wg, Wu, true, N, K, codes, scales, R, bias_gate,
                      bias_up, act, nullptr, 0, y, nullptr, plain_dtype(y_dtype)};
  return run(c, (hipStream_t)stream);
}

int qglu_mxfp8_act(const void* Wg, const void* Wu, int N, int K, const uint8_t* codes,
                   const uint8_t* scales, int R, const float* bias_gate, const float* bias_up,
                   int act, uint8_t* out_codes, uint8_t* out_scales, void* stream) {
  const ProductCall c{"qglu_mxfp8_act", QMOE_MXFP4, Wg, Wu, true, N, K, codes, scales, R,
                      bias_gate, bias_up, act, nullptr, 0, out_codes, out_scales, kQuantized};
  return run(c, (hipStream_t)stream);
}

}  // extern "C"
