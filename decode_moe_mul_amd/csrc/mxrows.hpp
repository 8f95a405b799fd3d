// Internal header: products of MXFP4 weights with up to 16 rows of MXFP4 or MXFP8
// activations; one product, or the two of a gated pair.
//
// A block computes 16 NB weight rows (of each of the products) x all activation
// rows with 16x16x128 ops; its waves split K in turns of 512 values, and their
// sums meet in LDS in wave order.  Operands go from memory to registers, a whole
// turn's loads together: with few rows the call is a read of the weights, and what
// counts is how many of them are on their way.
//
// Lane 16 g + i of step j takes block 4 j + g of the turn from weight row i, so
// that a load reads 64 consecutive bytes of each of 16 rows.  (Four consecutive
// blocks to a lane would put its scales into one word, but a load then touches four
// times as many cache sectors: 1 x 4096 x 4096 takes 4.6 us instead of 4.3.)  Its
// part of an MXFP8 row is values 16 g .. + 15 and 64 + 16 g .. + 15 of the step's
// 128.  The lane's scale of step j is byte g of the row's j-th scale word.
#pragma once
#include <algorithm>
#include <type_traits>

#include "mxtile.hpp"

#pragma clang fp contract(off)

namespace qmoe {

template <bool XF8>
QMOE_D v4f_t mx_mma16(uint4 w, uint32_t sw, uint4 x, uint4 xhi, uint32_t sx, v4f_t c) {
  const v8i_t wv = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
  if constexpr (XF8) {
    const auto op = [&](uint4 lo, uint4 hi, v4f_t sum) {
      const v8i_t xv = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
                        (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, xv, sum, 4, 0, 0, (int)sw, 0,
                                                              (int)sx);
    };
    uint4 bl, bh, sl, sh;  // as in the tiles: two ops, and no product is cut
    split_e4m3(x, bl, sl);
    split_e4m3(xhi, bh, sh);
    return op(bl, bh, op(sl, sh, c));
  } else {
    const v8i_t xv = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, xv, c, 4, 4, 0, (int)sw, 0,
                                                            (int)sx);
  }
}

template <bool F8>
struct Frag {  // one lane's part of a turn of one row
  uint4 q[4], hi[F8 ? 4 : 1];
  uint32_t s[4];
};
// `row` counts the plane's blocks before the row; blocks from nb on (past the
// row's end) are zeros.
template <bool F8, bool TAIL>
QMOE_D void load_frag(const uint8_t* q, const uint8_t* s, size_t row, int b0, int g, int nb,
                      Frag<F8>& f) {
  if constexpr (TAIL) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f.s[j] = b0 + 4 * j + g < nb ? s[row + b0 + 4 * j + g] : 0;
  } else {
    uint32_t w[4];  // no alignment: a row has K / 32 bytes
    __builtin_memcpy(w, s + row + b0, 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.s[j] = w[j] >> (8 * g);
  }
  const auto piece = [&](int chunk, int block) {  // 16 bytes of the row's codes
    const bool past = TAIL && block >= nb;
    return past ? make_uint4(0, 0, 0, 0) : *(const uint4*)(q + row * (F8 ? 32 : 16) + chunk * 16);
  };
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int b = b0 + 4 * j;
    if constexpr (F8) {
      f.q[j] = piece(2 * b + g, b + (g >> 1));
      f.hi[j] = piece(2 * b + 4 + g, b + 2 + (g >> 1));
    } else {
      f.q[j] = piece(b + g, b + g);
    }
  }
}

// A wave per turn where there are that many: 1 x 4096 x 14336 takes 8.3 us, with
// 8 waves 9.6.  Four rows of tiles (a gated pair in its quantized form) hold more
// registers than 16 waves leave.
template <bool GLU, int NB>
constexpr int rows_waves() { return GLU && NB == 2 ? 8 : 16; }

template <bool XF8, bool GLU, int NB>
__global__ __launch_bounds__(64 * (rows_waves<GLU, NB>())) void mx_rows_kernel(MxProduct P) {
  constexpr int A = (GLU ? 2 : 1) * NB;  // 16 x 16 sums: gate's (or all), then up's
  __shared__ v4f_t sums[rows_waves<GLU, NB>()][A][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int nb = P.K >> 5, turns = (nb + 15) >> 4, full = nb >> 4;
  const int n0 = blockIdx.x * 16 * NB;
  size_t wrow[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) wrow[b] = (size_t)min(n0 + 16 * b + i, P.N - 1) * nb;
  const size_t xrow = (size_t)min(i, P.R - 1) * nb;
  v4f_t acc[A];
#pragma unroll
  for (int a = 0; a < A; ++a) acc[a] = v4f_t{0.f, 0.f, 0.f, 0.f};
  const auto turn = [&](auto tail, int u) {
    constexpr bool TAIL = decltype(tail)::value;
    Frag<false> w[A];
    Frag<XF8> x;
#pragma unroll
    for (int a = 0; a < A; ++a)
      load_frag<false, TAIL>(a < NB ? P.wq : P.wq2, a < NB ? P.ws : P.ws2, wrow[a % NB], 16 * u,
                             g, nb, w[a]);
    load_frag<XF8, TAIL>(P.xq, P.xs, xrow, 16 * u, g, nb, x);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int a = 0; a < A; ++a)
        acc[a] = mx_mma16<XF8>(w[a].q[j], w[a].s[j], x.q[j], x.hi[XF8 ? j : 0], x.s[j], acc[a]);
  };
  int u = wave;
  for (; u < full; u += waves) turn(std::false_type{}, u);
  if (u < turns) turn(std::true_type{}, u);  // the last, partial turn
#pragma unroll
  for (int a = 0; a < A; ++a) sums[wave][a][lane] = acc[a];
  __syncthreads();
  if (wave > 0) return;
  for (int w = 1; w < waves; ++w)
#pragma unroll
    for (int a = 0; a < A; ++a) {
      const v4f_t v = sums[w][a][lane];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[a][j] += v[j];
    }
  // lane 16 g + i: weight rows 4 g .. + 3 of activation row i
  float v[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int n = n0 + 16 * b + 4 * g;
    float up[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[b][j] = acc[b][j], up[j] = GLU ? acc[A - NB + b][j] : 0.f;
    if constexpr (GLU) join4(P.e, v[b], up, n, P.N);
  }
  if constexpr (NB == 2)
    leave_block<XF8 ? kOutMx8 : kOutMx4>(P.e, v[0], v[1], i, P.R, n0, P.N, g);
  else if (i < P.R)
    leave4<GLU>(P.e, v[0], (size_t)i, n0 + 4 * g, P.N);
}

template <bool XF8, bool GLU, int NB>
static int launch_rows(const char* name, const MxProduct& P, hipStream_t s) {
  const dim3 grid((unsigned)((P.N + 16 * NB - 1) / (16 * NB)));
  const int waves = std::min(rows_waves<GLU, NB>(), (P.K / 32 + 15) / 16);
  return QMOE_LAUNCH(name, (mx_rows_kernel<XF8, GLU, NB>), grid, 64 * waves, 0, s, P);
}

}  // namespace qmoe
