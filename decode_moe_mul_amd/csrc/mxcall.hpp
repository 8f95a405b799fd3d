// Internal header: the kernel arguments of a checked MX product.
#pragma once
#include "mxrows.hpp"
#include "product.hpp"

namespace qmoe {

static inline MxProduct mx_product(const ProductCall& c) {
  const Layout L = layout_of(QMOE_MXFP4, c.N, c.K);
  const uint8_t *w = (const uint8_t*)c.W, *w2 = (const uint8_t*)(c.pair ? c.W2 : c.W);
  return {w + L.off[0],
          w + L.off[1],
          w2 + L.off[0],
          w2 + L.off[1],
          (const uint8_t*)c.codes,
          (const uint8_t*)c.scales,
          c.N,
          c.K,
          c.R,
          epilogue_of(c)};
}

}  // namespace qmoe
