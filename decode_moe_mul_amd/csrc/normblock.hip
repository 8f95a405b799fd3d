// The norms around a block, with the block's gate and residual scale between them:
//
//   z = x * w_post / sqrt(mean(x^2) + eps_post)        (z = x without w_post)
//   h = res_scale * res + scale * gate * z             (rounded to fp32, then to res' type)
//   y = fp32( h * w / sqrt(mean(h^2) + eps) )
//
// x is what the block delivers, res the stream it joins, y what the next block's
// product takes (fp32, bf16, int8 with block scales, MXFP8 or MXFP4).  A call reads
// x, res and the weights and writes h and y, each once; the row stays in registers
// between the two norms.
//
// Codes change wherever y crosses a border, and h's own rounding decides y, so sums,
// roots and products are fp64, as in the single norm: the squares' sums take at most
// 32 + 6 + 16 roundings, which the root halves, and h at most seven more, which leaves
// h within 2^-47 of |res_scale res| + |scale gate z| of its definition before it is
// rounded to fp32, and y within 2^-47 of its own.  fp64 multiply-adds run at the rate of
// fp32 ones here.
#include <algorithm>

#include "act.hpp"

#pragma clang fp contract(off)

namespace qmoe {

struct NormBlockParams {
  const void* x;
  const float* w_post;  // NULL: no norm of x
  const void* gate;     // NULL: 1
  const void* res;
  void* res_out;        // NULL, or res itself: a lane reads its values before it writes them
  const float* w;
  void* out;
  void* scales;
  double eps_post, scale, res_scale, eps;
  int R, K, gate_bf, rows_per_gate;
};

// The sum of `v` over the `tpr` threads of a row; `part` is read by this call alone.
QMOE_D double row_sum(double v, int tpr, double* part) {
  if (tpr >= 64) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  } else {
    for (int off = tpr >> 1; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  }
  const int waves = tpr >> 6;
  if (waves > 1) {
    const int wave0 = (threadIdx.x >> 6) & ~(waves - 1);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < waves; ++i) v += part[wave0 + i];
  }
  return v;
}

// Eight values as they lie in memory.  `hide` keeps the compiler from carrying what
// it has computed of them (their fp64 values: twice to four times the registers)
// over a wait: of a row with four octets a thread that spilled 140 registers, and
// 8192 x 7168 took 479 us.
template <bool BF>
struct Octet {
  uint32_t w[BF ? 4 : 8];
  QMOE_D void load(const void* p, size_t at) {
    const uint4* q = (const uint4*)((const uint8_t*)p + at * (BF ? 2 : 4));
    *(uint4*)w = q[0];
    if constexpr (!BF) *(uint4*)(w + 4) = q[1];
  }
  QMOE_D void store(void* p, size_t at) const {
    uint4* q = (uint4*)((uint8_t*)p + at * (BF ? 2 : 4));
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (!BF) q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  QMOE_D float operator[](int i) const {
    if constexpr (!BF) return __builtin_bit_cast(float, w[i]);
    else if (i & 1) return __builtin_bit_cast(float, w[i >> 1] & 0xFFFF0000u);
    else return bf16_bits_to_f32(w[i >> 1] & 0xFFFFu);
  }
  QMOE_D void set(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < (BF ? 4 : 8); ++i) {
      if constexpr (BF) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      else w[i] = __builtin_bit_cast(uint32_t, v[i]);
    }
  }
  QMOE_D void zero() {
#pragma unroll
    for (int i = 0; i < (BF ? 4 : 8); ++i) w[i] = 0;
  }
  QMOE_D void hide() {
#pragma unroll
    for (int i = 0; i < (BF ? 4 : 8); ++i) asm volatile("" : "+v"(w[i]));
  }
};

// tpr threads share a row (a power of two, a block's four at least), NPT octets each:
// octet o of the row belongs to thread o mod tpr.  A block takes blockDim.x / tpr
// rows at a time and goes on to later ones.  Rows with one or two octets a thread
// request the weights and the gate with the row (one wait for memory, few rows);
// longer ones read them from the near caches when they are needed, which leaves the
// registers to rows in flight.
template <int OUT, int NPT, bool XBF, bool RBF>
__global__ __launch_bounds__(1024) void norm_block_kernel(NormBlockParams P, int tpr) {
  __shared__ double part[2][16];
  const int K8 = P.K >> 3;
  const int t = threadIdx.x & (tpr - 1), lrow = threadIdx.x / tpr;
  const int rows = blockDim.x / tpr;
  constexpr bool early = NPT <= 2;
  constexpr int NW = early ? NPT : 1;
  // uniform over the block: every thread meets the barriers the same number of times
  for (long long r0 = (long long)blockIdx.x * rows; r0 < P.R; r0 += (long long)gridDim.x * rows) {
    const bool live = r0 + lrow < P.R;
    const size_t base = (size_t)(r0 + lrow) * P.K;
    const size_t gbase =
        live && P.gate ? (size_t)((int)(r0 + lrow) / P.rows_per_gate) * P.K : 0;
    Octet<XBF> x[NPT];
    Octet<RBF> h[NPT];  // the residual, then h
    Octet<false> wp[NW], gt[NW], w[NW];
    const auto load_post = [&](int j, int o) {  // w_post and gate, where there are any
      if (P.w_post) wp[j].load(P.w_post, (size_t)o * 8);
      if (P.gate) {
        if (P.gate_bf) {
          Octet<true> g;
          g.load(P.gate, gbase + (size_t)o * 8);
          const float v[8] = {g[0], g[1], g[2], g[3], g[4], g[5], g[6], g[7]};
          gt[j].set(v);
        } else {
          gt[j].load(P.gate, gbase + (size_t)o * 8);
        }
      }
    };
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      const int o = t + j * tpr;
      if (live && o < K8) {
        x[j].load(P.x, base + (size_t)o * 8);
        h[j].load(P.res, base + (size_t)o * 8);
        if constexpr (early) {
          load_post(j, o);
          w[j].load(P.w, (size_t)o * 8);
        }
      } else {
        x[j].zero();
      }
    }
    double sc = P.scale;
    if (P.w_post) {
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < NPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma((double)x[j][i], (double)x[j][i], sum);
      // the second norm's barrier stands between this read of part[0] and the next write
      sum = row_sum(sum, tpr, part[0]);
      sc *= 1.0 / sqrt(sum / P.K + P.eps_post);
#pragma unroll
      for (int j = 0; j < NPT; ++j) x[j].hide();
    }
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      const int o = t + j * tpr;
      if (live && o < K8) {
        constexpr int J = early ? 1 : 0;
        if constexpr (!early) load_post(0, o);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          double z = (double)x[j][i];
          if (P.w_post) z *= (double)wp[j * J][i];
          z *= P.gate ? (double)gt[j * J][i] * sc : sc;
          v[i] = (float)fma(P.res_scale, (double)h[j][i], z);
        }
        h[j].set(v);
        if (P.res_out) h[j].store(P.res_out, base + (size_t)o * 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma((double)h[j][i], (double)h[j][i], sum);
        h[j].hide();
      }
    }
    if (!P.w_post && tpr > 64) __syncthreads();  // the last rows' sums have been read
    sum = row_sum(sum, tpr, part[1]);
    const double scale = 1.0 / sqrt(sum / P.K + P.eps);
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      const int o = t + j * tpr;
      if (live && o < K8) {
        if constexpr (!early) w[0].load(P.w, (size_t)o * 8);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[i] = (float)((double)h[j][i] * (double)w[early ? j : 0][i] * scale);
        store_act8<OUT>(y, base + (size_t)o * 8, P.out, P.scales);
      }
    }
  }
}

template <int OUT, int NPT>
static int launch_norm_block(bool xbf, bool rbf, dim3 g, int block, hipStream_t s,
                             const NormBlockParams& P, int tpr) {
  const char* name = "norm_block";
  if (xbf && rbf)
    return QMOE_LAUNCH(name, (norm_block_kernel<OUT, NPT, true, true>), g, block, 0, s, P, tpr);
  if (xbf)
    return QMOE_LAUNCH(name, (norm_block_kernel<OUT, NPT, true, false>), g, block, 0, s, P, tpr);
  if (rbf)
    return QMOE_LAUNCH(name, (norm_block_kernel<OUT, NPT, false, true>), g, block, 0, s, P, tpr);
  return QMOE_LAUNCH(name, (norm_block_kernel<OUT, NPT, false, false>), g, block, 0, s, P, tpr);
}

struct NormBlockCall {
  const void* x;
  int x_dtype;
  const float* w_post;
  double eps_post;
  const void* gate;
  int gate_dtype, gate_rows;
  double scale;
  const void* res;
  void* res_out;
  int res_dtype;
  double res_scale;
  const float* w;
  double eps;
  int R, K;
  void *out, *scales;
  void* stream;
};

template <int OUT>
static int run_norm_block(const char* who, const NormBlockCall& c) {
  constexpr int unit = OUT == kOutF32 || OUT == kOutBF16 ? 8 : 32;
  if (c.R < 0 || c.K <= 0 || c.K % unit || c.K > 32768)
    return fail(QMOE_ERR_INVALID_ARG, "%s: R=%d K=%d (K %% %d == 0, K <= 32768)", who, c.R, c.K,
                unit);
  const auto known = [](int d) { return d == QMOE_F32 || d == QMOE_BF16; };
  if (!known(c.x_dtype) || !known(c.res_dtype) || (c.gate && !known(c.gate_dtype)))
    return fail(QMOE_ERR_UNSUPPORTED, "%s: unknown x_dtype %d, res_dtype %d or gate_dtype %d", who,
                c.x_dtype, c.res_dtype, c.gate_dtype);
  if (!(c.eps >= 0.0) || (c.w_post && !(c.eps_post >= 0.0)))
    return fail(QMOE_ERR_INVALID_ARG, "%s: eps and eps_post must be at least 0", who);
  if (c.gate && (c.gate_rows < 1 || c.R % c.gate_rows))
    return fail(QMOE_ERR_INVALID_ARG, "%s: gate_rows=%d does not divide R=%d", who, c.gate_rows,
                c.R);
  if (c.R == 0) return QMOE_OK;
  if (!c.x || !c.res || !c.w || !c.out || (unit == 32 && !c.scales))
    return fail(QMOE_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!QMOE_ALIGNED(c.x, 16) || !QMOE_ALIGNED(c.w_post, 16) || !QMOE_ALIGNED(c.gate, 16) ||
      !QMOE_ALIGNED(c.res, 16) || !QMOE_ALIGNED(c.res_out, 16) || !QMOE_ALIGNED(c.w, 16) ||
      !QMOE_ALIGNED(c.out, 16) || (OUT == kOutQ8 && !QMOE_ALIGNED(c.scales, 4)))
    return fail(QMOE_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  const int K8 = c.K >> 3, cus = std::max(1, cu_count());
  const bool xbf = c.x_dtype == QMOE_BF16, rbf = c.res_dtype == QMOE_BF16;
  // Octets per thread.  Few rows: one up to 4096 values (1 x 4096 4.7 us, with two 5.3,
  // with four 8.1), two beyond (16 x 7168 6.2; one 6.9, four 7.3).  Once the rows fill
  // the part, fewer barriers and sums per byte pay, as far as the registers go: four of
  // bf16 (8192 x 7168 124 us; two 142, one 196; 8192 x 4096 61; two 68, one 79; eight
  // 140), two where fp32 is among them (8192 x 7168 166; four 185, one 215) and for rows
  // below 2048 values (8192 x 256 6.6; four 7.3, one 6.8).  Two rows of two octets to a
  // thread, which share the weights and the barriers, take 147 at 8192 x 7168.
  const bool many = c.R > 2 * cus;
  int npt = many ? (xbf && rbf && K8 >= 256 ? 4 : 2) : K8 <= 512 ? 1 : 2, tpr = 4;
  while (tpr < 1024 && tpr * npt < K8) tpr *= 2;
  while (tpr * npt < K8) npt *= 2;  // longer rows than 1024 threads hold: more per thread
  const int block = std::max(tpr, 256), rows = block / tpr;
  const long long need = ((long long)c.R + rows - 1) / rows;
  const dim3 grid((unsigned)std::min<long long>(need, (long long)cus * (2048 / block)));
  const NormBlockParams P{c.x,   c.w_post, c.gate,      c.res,   c.res_out,
                          c.w,   c.out,    c.scales,    c.eps_post, c.scale,
                          c.res_scale, c.eps, c.R, c.K, c.gate && c.gate_dtype == QMOE_BF16,
                          c.gate ? c.R / c.gate_rows : 1};
  hipStream_t s = (hipStream_t)c.stream;
  if (npt == 1) return launch_norm_block<OUT, 1>(xbf, rbf, grid, block, s, P, tpr);
  if (npt == 2) return launch_norm_block<OUT, 2>(xbf, rbf, grid, block, s, P, tpr);
  return launch_norm_block<OUT, 4>(xbf, rbf, grid, block, s, P, tpr);
}

}  // namespace qmoe

using namespace qmoe;

extern "C" {

#define NORM_BLOCK_ARGS                                                                          \
  const void *x, int x_dtype, const float *w_post, double eps_post, const void *gate,            \
      int gate_dtype, int gate_rows, double scale, const void *res, void *res_out,               \
      int res_dtype, double res_scale, const float *w, double eps, int R, int K
#define NORM_BLOCK_CALL(out, scales)                                                           \
  {x,         x_dtype,   w_post, eps_post, gate, gate_dtype, gate_rows, scale,  res, res_out, \
   res_dtype, res_scale, w,      eps,      R,    K,          out,       scales, stream}

int qnorm_block(NORM_BLOCK_ARGS, void* y, int y_dtype, void* stream) {
  const NormBlockCall c NORM_BLOCK_CALL(y, nullptr);
  if (y_dtype == QMOE_F32) return run_norm_block<kOutF32>("qnorm_block", c);
  if (y_dtype == QMOE_BF16) return run_norm_block<kOutBF16>("qnorm_block", c);
  return fail(QMOE_ERR_UNSUPPORTED, "qnorm_block: unknown y_dtype %d", y_dtype);
}

int qnorm_block_act_q8(NORM_BLOCK_ARGS, int8_t* q, float* d, void* stream) {
  const NormBlockCall c NORM_BLOCK_CALL(q, d);
  return run_norm_block<kOutQ8>("qnorm_block_act_q8", c);
}

int qnorm_block_act_mxfp8(NORM_BLOCK_ARGS, uint8_t* codes, uint8_t* scales, void* stream) {
  const NormBlockCall c NORM_BLOCK_CALL(codes, scales);
  return run_norm_block<kOutMx8>("qnorm_block_act_mxfp8", c);
}

int qnorm_block_act_mxfp4(NORM_BLOCK_ARGS, uint8_t* codes, uint8_t* scales, void* stream) {
  const NormBlockCall c NORM_BLOCK_CALL(codes, scales);
  return run_norm_block<kOutMx4>("qnorm_block_act_mxfp4", c);
}

}  // extern "C"
