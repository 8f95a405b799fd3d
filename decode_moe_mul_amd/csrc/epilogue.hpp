// Internal header: what a product does with its sums before they leave: bias,
// activation, the gated multiplication, residual.  All of it in fp32 on the fp32
// sums, rounded once to the output's type.
#pragma once
#include <type_traits>
#include <utility>

#include "act.hpp"

namespace qmoe {

template <int I>
using Int = std::integral_constant<int, I>;

// f(0), f(1), .. with indices that are constants in f's own code: what they pick
// among registers needs no loop to be unrolled first
template <class F, int... I>
QMOE_D void static_for_each(std::integer_sequence<int, I...>, F&& f) {
  (f(Int<I>{}), ...);
}
template <int N, class F>
QMOE_D void static_for(F&& f) {
  static_for_each(std::make_integer_sequence<int, N>{}, f);
}

struct Epilogue {
  const float* bias;   // [N] or NULL; of the gate where there are two products
  const float* bias2;  // [N] or NULL, of up
  const void* res;     // [R][N] or NULL; may be y itself (same type)
  void* y;             // [R][N] values, or codes
  void* scales;        // of a quantized output
  int act;             // qmoe_act
  int out;             // ActOut
  int res_bf;          // res is bf16
};

// exp through the hardware's exp2: the product with log2 e is rounded, so the
// relative error grows with |v|: |v| 2^-24 on top of exp2's own.  (Of normal values
// silu is off by 4.7e-8 in the mean square, gelu_tanh by 4.7e-8, as against 3.9e-8 and
// 4.2e-8 with torch's exp and division.  A Newton step on the reciprocal and the
// product's remainder in the exponent make it 4.5e-8 and 4.6e-8, and a pair of
// 2048 x 14336 x 4096 in MXFP4 169 to 172 us instead of 162.)
QMOE_D float exp_of(float v) { return __builtin_amdgcn_exp2f(v * 1.4426950408889634f); }
QMOE_D float recip(float v) { return __builtin_amdgcn_rcpf(v); }

// Phi(-|v|) of the normal distribution: half of erfc(z), z = |v| / sqrt 2, as
// t exp(-z^2) P(t), t = 1 / (1 + 0.4 z).  P of degree 8 is fitted to
// exp(z^2) erfc(z) / t over all z >= 0 (reweighted least squares; with the
// coefficients as they stand here its relative error is at most 1.6e-7),
// so the tail keeps its relative precision, which 1 + erf would lose.  15
// instructions; a library erfc takes 40 with a branch.
QMOE_D float normal_tail(float v) {
  const float t = recip(fmaf(fabsf(v), 0.28284271247f, 1.f));
  float p = 0.05025659129023552f;
  p = fmaf(p, t, -0.18288160860538483f);
  p = fmaf(p, t, 0.16905683279037476f);
  p = fmaf(p, t, -0.005586383864283562f);
  p = fmaf(p, t, 0.14142291247844696f);
  p = fmaf(p, t, 0.16854381561279297f);
  p = fmaf(p, t, 0.20784251391887665f);
  p = fmaf(p, t, 0.22566960752010345f);
  p = fmaf(p, t, 0.22567586600780487f);
  return 0.5f * p * t * __builtin_amdgcn_exp2f(v * v * -0.72134752044f);
}

// The activation on E values; `act` is uniform over the launch, so the switch
// is a scalar branch around straight-line code.  Infinities: silu, gelu and
// gelu_tanh give NaN at -infinity, as their formulas do; NaN stays NaN.
template <int E>
QMOE_D void activate(int act, float (&v)[E]) {
  switch (act) {
    case QMOE_ACT_SILU:  // v / (1 + exp(-v)); exp's infinity gives -0
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] *= recip(1.f + exp_of(-v[k]));
      break;
    case QMOE_ACT_GELU:  // v Phi(v)
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float q = normal_tail(v[k]);
        v[k] *= v[k] > 0.f ? 1.f - q : q;
      }
      break;
    case QMOE_ACT_GELU_TANH:  // v / 2 (1 + tanh u) = v / (1 + exp(-2 u))
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float u = fmaf(v[k] * v[k] * v[k], 0.0713548162726f, v[k] * 1.5957691216057308f);
        v[k] *= recip(1.f + exp_of(-u));
      }
      break;
    case QMOE_ACT_RELU:
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = v[k] < 0.f ? 0.f : v[k];
      break;
    case QMOE_ACT_RELU2:
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = v[k] < 0.f ? 0.f : v[k] * v[k];
      break;
    default:
      break;
  }
}

QMOE_D float res_at(const Epilogue& e, size_t at) {
  return e.res_bf ? bf16_bits_to_f32(((const uint16_t*)e.res)[at]) : ((const float*)e.res)[at];
}
QMOE_D void store_at(const Epilogue& e, size_t at, float v) {
  if (e.out == kOutBF16) ((uint16_t*)e.y)[at] = (uint16_t)f32_to_bf16_bits(v);
  else ((float*)e.y)[at] = v;
}

// Four consecutive columns n .. n + 3 of one row in a plain type, those that exist:
// bias (`b`, one product's), activation and residual, where the launch has them.
template <bool DONE>
QMOE_D void leave4(const Epilogue& e, float (&v)[4], size_t row, int n, int N) {
  if (n >= N) return;
  const size_t at = row * N + n;
  if constexpr (!DONE) {
    if (e.bias)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += e.bias[min(n + j, N - 1)];
    activate(e.act, v);
    if (e.res)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += res_at(e, row * N + min(n + j, N - 1));
  }
  if (N % 4 == 0) {
    if (e.out == kOutBF16)
      *(uint2*)((uint16_t*)e.y + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    else
      *(float4*)((float*)e.y + at) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < N) store_at(e, at + j, v[j]);
  }
}

// A gated pair's four columns n .. n + 3: v = act(v + bias) * (up + bias2).
QMOE_D void join4(const Epilogue& e, float (&v)[4], const float (&up)[4], int n, int N) {
  if (e.bias)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += e.bias[min(n + j, N - 1)];
  activate(e.act, v);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] *= up[j] + (e.bias2 ? e.bias2[min(n + j, N - 1)] : 0.f);
}

// Columns n0 .. + 31 of activation row i, quantized: lane 16 g + i of the wave holds
// columns 4 g .. + 3 (lo) and 16 + 4 g .. + 3 (hi).  Every lane calls this; N % 32 == 0.
template <int OUT>
QMOE_D void leave_block(const Epilogue& e, const float (&lo)[4], const float (&hi)[4], int i,
                        int R, int n0, int N, int g) {
  const float o[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  uint32_t m = 0;  // the largest magnitude's bits; a NaN's are above infinity's
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __builtin_bit_cast(uint32_t, o[k]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  const bool bad = m >= 0x7F800000u;
  if (i >= R) return;
  const size_t at = (size_t)i * N + n0;
  uint8_t* const y = (uint8_t*)e.y;
  if constexpr (OUT == kOutQ8) {
    const float d = over_127(__builtin_bit_cast(float, m));
    uint32_t w[2] = {0, 0};
    q8_codes8(o, d, w);
    if (!(d > 0.f) || bad) w[0] = w[1] = 0;
    *(uint32_t*)(y + at + 4 * g) = w[0];
    *(uint32_t*)(y + at + 16 + 4 * g) = w[1];
    if (g == 0) ((float*)e.scales)[at >> 5] = bad ? __builtin_nanf("") : d;
  } else {
    const int ex = mx_exponent<OUT>(m);
    uint2 c = mx_codes8<OUT>(o, mx_over(ex));
    if (bad) c = make_uint2(0, 0);
    if constexpr (OUT == kOutMx8) {
      *(uint32_t*)(y + at + 4 * g) = c.x;
      *(uint32_t*)(y + at + 16 + 4 * g) = c.y;
    } else {
      *(uint16_t*)(y + at / 2 + 2 * g) = (uint16_t)c.x;
      *(uint16_t*)(y + at / 2 + 8 + 2 * g) = (uint16_t)(c.x >> 16);
    }
    if (g == 0) ((uint8_t*)e.scales)[at >> 5] = (uint8_t)(bad ? 255 : ex);
  }
}

// How the sums of a tile's wave leave: through LDS, 32 rows of the wave's COLS
// columns at a time, so that a lane has eight consecutive columns of a row (of a
// pair, where every 64 columns are 32 of the gate and 32 of up, eight of either).
// Rows lie 8 words more than a multiple of 32 apart: the rows that one store of a
// wave's sums touches are on different banks.  The region is the wave's own.
//
// A tile's code here runs once, so what it costs is its fetching: the arithmetic
// stands in a loop that stays one (unrolled, every activation's code would be there
// as often as the wave has pieces), and each way of storing is a loop of its own, so
// that a tile runs through a short straight piece of them (with the choice inside the
// loop the largest tile's 17000 instructions took a call of 70 us to 95).
constexpr int leave_pitch(int cols) { return cols + 8; }

template <int COLS, bool GLU, int QUANT>  // QUANT: the ActOut of a quantized output
struct Leave {
  static constexpr int PITCH = leave_pitch(COLS), OC = GLU ? COLS / 2 : COLS;
  static constexpr int LR = OC / 8, Z = LR / 2, STEP = 64 / LR;  // lanes to a row, pieces to a lane
  enum Res { kNone, kBF16, kF32 };
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const Epilogue& e;
  float* region;
  float* p0;   // the lane's first piece
  int R, N, n0, lane;
  float b1[8], b2[8];

  static QMOE_D int lds_col(int col) { return GLU ? (col >> 5 << 6) + (col & 31) : col; }

  QMOE_D Leave(const Epilogue& ep, float* reg, int first, int R_, int N_, int lane_)
      : e(ep), region(reg), R(R_), N(N_), n0(first), lane(lane_) {
    const int col = (lane % LR) * 8;
    p0 = region + lane / LR * PITCH + lds_col(col);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int n = min(n0 + col + k, N - 1);
      b1[k] = e.bias ? e.bias[n] : 0.f;
      b2[k] = GLU && e.bias2 ? e.bias2[n] : 0.f;
    }
  }

  static QMOE_D void read8(const float* p, float (&v)[8]) {
    const float4 lo = ((const float4*)p)[0], hi = ((const float4*)p)[1];
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  }

  // Plain types: piece z of a lane is columns E l .. + E - 1 of a row, 16 bytes of y.
  // N % E == 0, so that a piece is there or not as one, and aligned.
  template <int OUT>
  struct Piece {
    static constexpr int E = OUT == kOutBF16 ? 8 : 4, LR = OC / E, Z = 32 * LR / 64;
  };
  template <Res RES, int OUT>
  struct Residual {  // of a lane's pieces of 32 rows, four columns to an element
    static constexpr int H = Piece<OUT>::E / 4;
    typename std::conditional<RES == kBF16, u32x2, u32x4>::type
        v[RES == kNone ? 1 : Piece<OUT>::Z * H];
  };
  // the residual of rows row0 .. + 31, all pieces at once: one wait for memory
  template <Res RES, int OUT>
  QMOE_D void load(int row0, Residual<RES, OUT>& r) const {
    using P = Piece<OUT>;
    if constexpr (RES != kNone) {
      const int c = min(n0 + lane % P::LR * P::E, N - P::E);
      static_for<P::Z>([&](auto z) {
        const size_t at = (size_t)min(row0 + lane / P::LR + z * (64 / P::LR), R - 1) * N + c;
        if constexpr (RES == kBF16 && P::E == 8) {
          const u32x4 q = *(const u32x4*)((const uint16_t*)e.res + at);
          r.v[2 * z] = u32x2{q[0], q[1]};
          r.v[2 * z + 1] = u32x2{q[2], q[3]};
        } else if constexpr (RES == kBF16) {
          r.v[z] = *(const u32x2*)((const uint16_t*)e.res + at);
        } else {
          const u32x4* p = (const u32x4*)((const float*)e.res + at);
          r.v[P::E / 4 * z] = p[0];
          if constexpr (P::E == 8) r.v[2 * z + 1] = p[1];
        }
      });
    }
  }
  template <Res RES, int OUT>
  QMOE_D void store_rows(int row0, const Residual<RES, OUT>& res) const {
    using P = Piece<OUT>;
    const int col = lane % P::LR * P::E;
    static_for<P::Z>([&](auto z) {
      const int lrow = lane / P::LR + z * (64 / P::LR), row = row0 + lrow;
      if (row < R && n0 + col < N) {
        const float4* p = (const float4*)(region + lrow * PITCH + lds_col(col));
        float v[P::E];
        static_for<P::E / 4>([&](auto h) {
          const float4 f = p[h];
          v[4 * h] = f.x; v[4 * h + 1] = f.y; v[4 * h + 2] = f.z; v[4 * h + 3] = f.w;
          const auto r = res.v[RES == kNone ? 0 : P::E / 4 * z + h];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (RES == kBF16) {
              const uint32_t w = r[k / 2];
              v[4 * h + k] += bf16_bits_to_f32(k & 1 ? w >> 16 : w & 0xFFFFu);
            } else if constexpr (RES == kF32) {
              v[4 * h + k] += __builtin_bit_cast(float, (uint32_t)r[k]);
            }
          }
        });
        const size_t at = (size_t)row * N + n0 + col;
        if constexpr (OUT == kOutBF16)
          *(uint4*)((uint16_t*)e.y + at) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                      pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        else
          *(float4*)((float*)e.y + at) = make_float4(v[0], v[1], v[2], v[3]);
      }
    });
  }
  // Quantized (N % 32 == 0): eight columns to a lane, and a block's four lanes are
  // there or not together.
  QMOE_D void store_codes(int row0) const {
    const int c0 = n0 + (lane % LR) * 8;
    static_for<Z>([&](auto z) {
      const int row = row0 + lane / LR + z * STEP;
      if (row < R && c0 < N) {
        float v[8];
        read8(p0 + z * STEP * PITCH, v);
        store_act8<QUANT>(v, (size_t)row * N + c0, e.y, e.scales);
      }
    });
  }
  // Any width: consecutive lanes take consecutive columns.
  template <Res RES, int OUT>
  QMOE_D void store_each(int row0) const {
#pragma unroll 4
    for (int o = lane; o < 32 * OC; o += 64) {
      const int row = o / OC, col = o % OC;
      if (row0 + row < R && n0 + col < N) {
        const size_t at = (size_t)(row0 + row) * N + n0 + col;
        float v = region[row * PITCH + lds_col(col)];
        if constexpr (RES == kBF16) v += bf16_bits_to_f32(((const uint16_t*)e.res)[at]);
        if constexpr (RES == kF32) v += ((const float*)e.res)[at];
        if constexpr (OUT == kOutBF16) ((uint16_t*)e.y)[at] = (uint16_t)f32_to_bf16_bits(v);
        else ((float*)e.y)[at] = v;
      }
    }
  }

  QMOE_D void math() const {
    if (!GLU && !e.bias && e.act == QMOE_ACT_NONE) return;
#pragma unroll 1
    for (int z = 0; z < Z; ++z) {
      float* const p = p0 + z * STEP * PITCH;
      float v[8];
      read8(p, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += b1[k];
      activate(e.act, v);
      if constexpr (GLU) {
        float u[8];
        read8(p + 32, u);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= u[k] + b2[k];
      }
      ((float4*)p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      ((float4*)p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }

  // One way of storing: rows row0 + 32 m .. + 31 for m < M; write(m) puts the wave's
  // sums of those rows into the region, which is this wave's own.  The next rows'
  // residual is on its way meanwhile.
  template <int M, Res RES, int OUT, class W>
  QMOE_D void way(int row0, W&& write) const {
    const bool wide = N % Piece<OUT>::E == 0;
    Residual<RES, OUT> res[2];
    if (wide) load<RES, OUT>(row0, res[0]);
    static_for<M>([&](auto m) {
      write(m);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if constexpr (m + 1 < M)
        if (wide) load<RES, OUT>(row0 + 32 * (m + 1), res[(m + 1) & 1]);
      math();
      if constexpr (OUT == QUANT) store_codes(row0 + 32 * m);
      else if (wide) store_rows<RES, OUT>(row0 + 32 * m, res[m & 1]);
      else store_each<RES, OUT>(row0 + 32 * m);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    });
  }
  template <int M, int OUT, class W>
  QMOE_D void ways(int row0, W&& write) const {
    if (GLU || !e.res) {
      way<M, kNone, OUT>(row0, write);
    } else if constexpr (!GLU) {
      if (e.res_bf) way<M, kBF16, OUT>(row0, write);
      else way<M, kF32, OUT>(row0, write);
    }
  }
  template <int M, class W>
  QMOE_D void all(int row0, W&& write) const {
    if constexpr (GLU)
      if (e.out > kOutBF16) return way<M, kNone, QUANT>(row0, write);
    if (e.out == kOutBF16) ways<M, kOutBF16>(row0, write);
    else ways<M, kOutF32>(row0, write);
  }
};

}  // namespace qmoe
