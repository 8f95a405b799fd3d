// MXFP4 weights x MXFP4 activations on the block-scaled matrix cores.
//
//   y[r, n] = sum_k w[n, k] x[r, k]
//
// Both operands are E2M1 codes with one E8M0 scale per 32 values along K, used
// as stored: every product of two codes is exact, the matrix op applies both
// scales and accumulates in fp32.
//
// Operand order.  A 16x16x128 op takes, from lane 16 g + i, the 16 code bytes
// of one K block of row i, and that block's scale from a byte of a register
// that the op selects.  Which K block is called "block g of the step" is free
// as long as both operands agree, so four steps together cover 16 consecutive
// blocks with lane group g taking blocks 4 g .. 4 g + 3, one per step: its
// codes are then 64 consecutive bytes of the row and its four scales one
// 32-bit word, whose byte s serves step s without any repacking.
#include <algorithm>

#include "act.hpp"

#pragma clang fp contract(off)

namespace qmoe {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float v4f_t __attribute__((ext_vector_type(4)));

struct Mx4Params {
  const uint8_t* wq;  // codes [N][K/2]
  const uint8_t* ws;  // E8M0 [N][K/32]
  const uint8_t* xq;  // codes [R][K/2]
  const uint8_t* xs;  // E8M0 [R][K/32]
  void* y;            // [R][N]
  int N, K, R;
};

template <int STEP>
QMOE_D v4f_t mma4(uint4 a, uint32_t sa, uint4 b, uint32_t sb, v4f_t c) {
  const v8i_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, STEP, (int)sa, STEP,
                                                          (int)sb);
}

// One lane's part of 16 blocks: 4 blocks of codes and their scale word.
struct Frag {
  uint4 q[4];
  uint32_t s;
};
// Blocks b0 .. b0 + 3 of a row that starts at block `row` of the plane; blocks
// from nb on (past the row's end) are zeros.
QMOE_D uint32_t load_scales4(const uint8_t* p) {  // no alignment: a row has K / 32 bytes
  uint32_t v;
  __builtin_memcpy(&v, p, 4);
  return v;
}
template <bool TAIL>
QMOE_D void load_frag(const uint8_t* q, const uint8_t* s, size_t row, int b0, int nb, Frag& f) {
  if (!TAIL || b0 + 4 <= nb) {
    const uint4* p = (const uint4*)(q + (row + b0) * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.q[j] = p[j];
    f.s = load_scales4(s + row + b0);
  } else {
    f.s = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f.q[j] = make_uint4(0, 0, 0, 0);
      if (b0 + j < nb) {
        f.q[j] = *(const uint4*)(q + (row + b0 + j) * 16);
        f.s |= (uint32_t)s[row + b0 + j] << (8 * j);
      }
    }
  }
}

// ------------------------------------------------------ few rows ------
// A block computes 16 weight rows x 16 RT activation rows; its waves split K
// in turns of 16 blocks, and their sums meet in LDS in wave order.
template <int RT, bool YBF>
__global__ __launch_bounds__(512) void mxfp4_rows_kernel(Mx4Params P) {
  extern __shared__ __align__(16) float red[];  // [wave][RT][64 lanes][4]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int nb = P.K >> 5, turns = (nb + 15) >> 4, full = nb >> 4;
  const int n0 = blockIdx.x * 16, r0 = blockIdx.y * 16 * RT;
  const size_t wrow = (size_t)min(n0 + i, P.N - 1) * nb;
  size_t xrow[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) xrow[t] = (size_t)min(r0 + 16 * t + i, P.R - 1) * nb;
  v4f_t acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = v4f_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Frag& w, const Frag& x, v4f_t& c) {
    c = mma4<0>(w.q[0], w.s, x.q[0], x.s, c);
    c = mma4<1>(w.q[1], w.s, x.q[1], x.s, c);
    c = mma4<2>(w.q[2], w.s, x.q[2], x.s, c);
    c = mma4<3>(w.q[3], w.s, x.q[3], x.s, c);
  };
  int u = wave;
  for (; u < full; u += waves) {
    Frag w, x[RT];
    load_frag<false>(P.wq, P.ws, wrow, 16 * u + 4 * g, nb, w);
#pragma unroll
    for (int t = 0; t < RT; ++t) load_frag<false>(P.xq, P.xs, xrow[t], 16 * u + 4 * g, nb, x[t]);
#pragma unroll
    for (int t = 0; t < RT; ++t) multiply(w, x[t], acc[t]);
  }
  if (u < turns) {  // the last, partial turn
    Frag w, x;
    load_frag<true>(P.wq, P.ws, wrow, 16 * u + 4 * g, nb, w);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      load_frag<true>(P.xq, P.xs, xrow[t], 16 * u + 4 * g, nb, x);
      multiply(w, x, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < RT; ++t) *(v4f_t*)(red + ((wave * RT + t) * 64 + lane) * 4) = acc[t];
  __syncthreads();
  // lane 16 g + i of tile t holds rows n0 + 4 g .. + 3 of column i
  for (int o = threadIdx.x; o < RT * 64; o += blockDim.x) {
    const int t = o >> 6, l = o & 63;
    v4f_t s = *(const v4f_t*)(red + o * 4);
    for (int w = 1; w < waves; ++w) {
      const v4f_t v = *(const v4f_t*)(red + (w * RT * 64 + o) * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += v[j];
    }
    const int r = r0 + 16 * t + (l & 15), n = n0 + 4 * (l >> 4);
    if (r >= P.R) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (n + j >= P.N) break;
      const size_t at = (size_t)r * P.N + n + j;
      if constexpr (YBF) ((uint16_t*)P.y)[at] = (uint16_t)f32_to_bf16_bits(s[j]);
      else ((float*)P.y)[at] = s[j];
    }
  }
}

template <int RT>
static int launch_rows(const Mx4Params& P, bool ybf, hipStream_t s) {
  const dim3 grid((unsigned)((P.N + 15) / 16), (unsigned)((P.R + 16 * RT - 1) / (16 * RT)));
  const int turns = (P.K / 32 + 15) / 16;
  const int waves = std::min(8, turns);
  const size_t lds = (size_t)waves * RT * 64 * 16;
  if (ybf)
    return QMOE_LAUNCH("mxfp4_rows", (mxfp4_rows_kernel<RT, true>), grid, 64 * waves, lds, s, P);
  return QMOE_LAUNCH("mxfp4_rows", (mxfp4_rows_kernel<RT, false>), grid, 64 * waves, lds, s, P);
}

}  // namespace qmoe

using namespace qmoe;

extern "C" int qgemm_mxfp4_mxfp4(const void* W, int N, int K, const uint8_t* codes,
                                 const uint8_t* scales, int R, void* y, int y_dtype,
                                 void* stream) {
  if (N < 0 || R < 0 || K <= 0 || K % 32 || K > 65536)
    return fail(QMOE_ERR_INVALID_ARG,
                "qgemm_mxfp4_mxfp4: N=%d R=%d K=%d (K %% 32 == 0, K <= 65536)", N, R, K);
  if (y_dtype != QMOE_F32 && y_dtype != QMOE_BF16)
    return fail(QMOE_ERR_UNSUPPORTED, "qgemm_mxfp4_mxfp4: unknown y_dtype %d", y_dtype);
  if (N == 0 || R == 0) return QMOE_OK;
  if (!W || !codes || !scales || !y)
    return fail(QMOE_ERR_INVALID_ARG, "qgemm_mxfp4_mxfp4: null pointer");
  if (!QMOE_ALIGNED(W, 256) || !QMOE_ALIGNED(codes, 16) || !QMOE_ALIGNED(y, 16))
    return fail(QMOE_ERR_INVALID_ARG, "qgemm_mxfp4_mxfp4: misaligned W/codes/y");
  const Layout L = layout_of(QMOE_MXFP4, N, K);
  const Mx4Params P{(const uint8_t*)W + L.off[0], (const uint8_t*)W + L.off[1], codes, scales,
                    y, N, K, R};
  const bool ybf = y_dtype == QMOE_BF16;
  hipStream_t s = (hipStream_t)stream;
  if ((R + 63) / 64 > 65535)
    return fail(QMOE_ERR_UNSUPPORTED, "qgemm_mxfp4_mxfp4: R=%d too large", R);
  if (R <= 16) return launch_rows<1>(P, ybf, s);
  if (R <= 32) return launch_rows<2>(P, ybf, s);
  return launch_rows<4>(P, ybf, s);
}
