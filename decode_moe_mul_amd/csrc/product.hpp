// Internal header: the host side that the products with an epilogue share, their
// argument checks first of all.
#pragma once
#include "epilogue.hpp"

namespace qmoe {

struct ProductCall {
  const char* who;
  int fmt;                 // of the weights
  const void *W, *W2;      // W2: up, where there are two products
  bool pair;
  int N, K;
  const void *codes, *scales;
  int R;
  const float *bias, *bias2;
  int act;
  const void* res;
  int res_dtype;
  void *y, *y_scales;
  int y_dtype;             // qmoe_dtype; of quantized outputs kQuantized
};
constexpr int kQuantized = 1 << 20;  // no qmoe_dtype
// a caller's y_dtype, which must not pass for the marker
static inline int plain_dtype(int d) { return d == kQuantized ? -1 : d; }
constexpr int kNothing = 1;  // nothing to compute: the call is done

// QMOE_OK, a negative status, or kNothing
static inline int check_product(const ProductCall& c) {
  const bool quant = c.y_dtype == kQuantized, q8 = c.fmt == QMOE_Q8_0;
  if (c.N < 0 || c.R < 0 || c.K <= 0 || c.K % 32 || c.K > 65536 || (quant && c.N % 32))
    return fail(QMOE_ERR_INVALID_ARG, "%s: N=%d R=%d K=%d (K %% 32 == 0, K <= 65536%s)", c.who, c.N,
                c.R, c.K, quant ? ", N % 32 == 0" : "");
  if (!quant && c.y_dtype != QMOE_F32 && c.y_dtype != QMOE_BF16)
    return fail(QMOE_ERR_UNSUPPORTED, "%s: unknown y_dtype %d", c.who, c.y_dtype);
  if (c.res && c.res_dtype != QMOE_F32 && c.res_dtype != QMOE_BF16)
    return fail(QMOE_ERR_UNSUPPORTED, "%s: unknown res_dtype %d", c.who, c.res_dtype);
  if (c.act < QMOE_ACT_NONE || c.act > QMOE_ACT_RELU2)
    return fail(QMOE_ERR_UNSUPPORTED, "%s: unknown activation %d", c.who, c.act);
  if (c.N > 1 << 30 || c.R > 1 << 30)  // tile positions past the last row stay below 2^31
    return fail(QMOE_ERR_UNSUPPORTED, "%s: N=%d R=%d beyond 2^30", c.who, c.N, c.R);
  if (c.N == 0 || c.R == 0) return kNothing;
  if (!c.W || (c.pair && !c.W2) || !c.codes || !c.scales || !c.y || (quant && !c.y_scales))
    return fail(QMOE_ERR_INVALID_ARG, "%s: null pointer", c.who);
  if (!QMOE_ALIGNED(c.W, 256) || !QMOE_ALIGNED(c.W2, 256) || !QMOE_ALIGNED(c.codes, 16) ||
      !QMOE_ALIGNED(c.y, 16) || !QMOE_ALIGNED(c.res, 16) || !QMOE_ALIGNED(c.bias, 4) ||
      !QMOE_ALIGNED(c.bias2, 4) ||
      (q8 && (!QMOE_ALIGNED(c.scales, 4) || !QMOE_ALIGNED(c.y_scales, 4))))
    return fail(QMOE_ERR_INVALID_ARG, "%s: misaligned pointer", c.who);
  if (c.res && c.res == c.y && c.res_dtype != c.y_dtype)
    return fail(QMOE_ERR_INVALID_ARG, "%s: y is res, but of another type", c.who);
  return QMOE_OK;
}

static inline Epilogue epilogue_of(const ProductCall& c) {
  const int out = c.y_dtype == QMOE_F32    ? kOutF32
                  : c.y_dtype == QMOE_BF16 ? kOutBF16
                  : c.fmt == QMOE_Q8_0     ? kOutQ8
                                           : kOutMx4;  // which MX type, the kernel knows
  return {c.bias, c.bias2, c.res, c.y, c.y_scales, c.act, out, c.res && c.res_dtype == QMOE_BF16};
}

}  // namespace qmoe
