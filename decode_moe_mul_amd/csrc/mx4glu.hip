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

static int run(const ProductCall& c, hipStream_t s) {
  const int st = check_product(c);
  if (st) return st == kNothing ? QMOE_OK : st;
  const MxProduct P = mx_product(c);
  const int cus = std::max(1, cu_count());
  if (P.R <= 16 && P.N <= 32 * cus)
    return P.e.out > kOutBF16 ? launch_rows<false, true, 2>("mxfp4_glu_rows", P, s)
                              : launch_rows<false, true, 1>("mxfp4_glu_rows", P, s);
  static constexpr Choice choices[] = {
      choice<T4<1, 2, 1, 2, 2>, true>(1, 10.f), choice<T4<2, 2, 1, 2, 2>, true>(1, 11.f),
      choice<T4<2, 2, 2, 2, 2>, true>(1, 15.f), choice<T4<2, 2, 2, 2, 1>, true>(2, 25.f),
      choice<T4<2, 2, 4, 4, 1>, true>(1, 33.f)};
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
