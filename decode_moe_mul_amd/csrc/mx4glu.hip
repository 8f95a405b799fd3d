// The gated pair of products of MXFP4 weights with MXFP4 activations (qglu_mxfp4,
// qglu_mxfp4_act).
//
//   v[r, n] = act( sum_k wg[n, k] x[r, k] + bg[n] ) * ( sum_k wu[n, k] x[r, k] + bu[n] )
//
// One pass over the activations for both weights; gate and up meet in the registers
// that hold their sums and never go to memory.  v leaves in fp32, bf16 or as MXFP4
// activations of the next product: the fp32 v, quantized.
#include "mxcall.hpp"

#pragma clang fp contract(off)

namespace qmoe {

template <int WR, int WC, int TM, int TN, int KS>
using T4 = Tile<WR, WC, TM, TN, KS, false>;

// Which kernel: as measured at K = 4096 (us; N counts the pair's columns).
//   rows  1 x 14336: 13.7, 16 x 14336: 16.3; 32 x 64: 14.3; 64 x 64: 13.7 (62 MB of
//     weights; a streaming read of as many takes 12)
//   32 x 64, three teams  40 x 4096: 8.1; 64 x 64: 8.5; 128 x 64: 11.1
//   64 x 64, two teams    128 x 4096: 9.0; 32 x 64: 9.1; 128 x 64: 11.4
//   128 x 64, two teams   700 x 2048 (K = 7168): 20.4; 64 x 64: 31; two to a unit: 23.5
//   128 x 64, two to a unit  2048 x 14336: 147; two teams: 202; 256 x 128: 149-158
// The largest tile is chosen where it saves a round.  Against the best of the five for R
// from 40 to 2048, N from 2048 to 14336 and K of 4096 and 14336 (33 sizes) the choice
// takes at most 5 % longer; at K = 1024, where the largest tile is short of steps, 28 %
// at most (2048 x 14336: 80 and 62).
static int run(const ProductCall& c, hipStream_t s) {
  const int st = check_product(c);
  if (st) return st == kNothing ? QMOE_OK : st;
  const MxProduct P = mx_product(c);
  const int cus = std::max(1, cu_count());
  if (P.R <= 16 && P.N <= 32 * cus)
    return P.e.out > kOutBF16 ? launch_rows<false, true, 2>("mxfp4_glu_rows", P, s)
                              : launch_rows<false, true, 1>("mxfp4_glu_rows", P, s);
  static constexpr Choice choices[] = {
      choice<T4<1, 2, 1, 2, 3>, true>(1, 9.2f), choice<T4<2, 2, 1, 2, 2>, true>(1, 9.5f),
      choice<T4<2, 2, 2, 2, 2>, true>(1, 12.5f), choice<T4<2, 2, 2, 2, 1>, true>(2, 21.f, 14.f),
      choice<T4<2, 2, 4, 4, 1>, true>(1, 36.f)};
  return launch_choice(choices, c.who, "mxfp4_glu_tile", P, s);
}

}  // namespace qmoe

using namespace qmoe;

extern "C" {

int qglu_mxfp4(const void* Wg, const void* Wu, int N, int K, const uint8_t* codes,
               const uint8_t* scales, int R, const float* bias_gate, const float* bias_up, int act,
               void* y, int y_dtype, void* stream) {
  const ProductCall c{"qglu_mxfp4", QMOE_MXFP4, Wg, Wu, true, N, K, codes, scales, R, bias_gate,
                      bias_up, act, nullptr, 0, y, nullptr, plain_dtype(y_dtype)};
  return run(c, (hipStream_t)stream);
}

int qglu_mxfp4_act(const void* Wg, const void* Wu, int N, int K, const uint8_t* codes,
                   const uint8_t* scales, int R, const float* bias_gate, const float* bias_up,
                   int act, uint8_t* out_codes, uint8_t* out_scales, void* stream) {
  const ProductCall c{"qglu_mxfp4_act", QMOE_MXFP4, Wg, Wu, true, N, K, codes, scales, R,
                      bias_gate, bias_up, act, nullptr, 0, out_codes, out_scales, kQuantized};
  return run(c, (hipStream_t)stream);
}

}  // extern "C"
