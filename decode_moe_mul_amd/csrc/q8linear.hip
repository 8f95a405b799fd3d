// Q8_0 weights x int8 activations with an epilogue: one product with bias,
// activation and residual (qlinear_q8), or the gated pair (qglu_q8, qglu_q8_act).
//
//   p[r, n] = sum_b (dw[n, b] d[r, b]) * sum_{k in b} qw[n, k] q[r, k]
//   y = act(p + bias) + res,  or  v = act(p_gate + bias_gate) * (p_up + bias_up)
//
// A 32-value block's integer sum is exact; its scaling and the sum over blocks are
// fp32.  That scaling is what bounds many rows: an output and block takes the sum made
// fp32, the product of the two scales and a multiply-add.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "copy.hpp"
#include "product.hpp"

#pragma clang fp contract(off)

namespace qmoe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

struct Q8Product {
  const int8_t* wq;    // [N][K]; of the gate where there are two products
  const uint16_t* wd;  // [N][K/32] fp16
  const int8_t* wq2;   // up's
  const uint16_t* wd2;
  const int8_t* xq;    // [R][K]
  const float* xd;     // [R][K/32]
  int N, K, R;
  Epilogue e;
};

QMOE_D i32x4_t i8_mma(i32x4_t a, i32x4_t b) {  // 16 x 16 x 64
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, i32x4_t{0, 0, 0, 0}, 0, 0, 0);
}

// ------------------------------------------------------ few rows ------
// A block computes 16 NB weight rows (of each product) x 16 activation rows; its waves
// split K in turns of 256 values (a pair: 128), and their sums meet in LDS in wave
// order.  Lane 16 g + i takes 16 bytes at 16 g of every 64 of weight row i and of
// activation row i, so that a load reads 64 consecutive bytes of 16 rows.  An op over
// 64 values mixes two blocks: it is done twice, with the activations of either block
// zeroed, which lanes 0..31 and 32..63 hold.
template <bool GLU, int NB>
constexpr int q8_waves() { return GLU && NB == 2 ? 8 : 16; }
// blocks of a turn: what 16 waves' registers hold of one product, of a pair half that
template <bool GLU>
constexpr int q8_turn() { return GLU ? 4 : 8; }

template <bool GLU, int NB>
__global__ __launch_bounds__(64 * (q8_waves<GLU, NB>())) void q8_rows_kernel(Q8Product P) {
  constexpr int A = (GLU ? 2 : 1) * NB, TURN = q8_turn<GLU>();
  __shared__ f32x4_t sums[q8_waves<GLU, NB>()][A][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int nb = P.K >> 5, turns = (nb + TURN - 1) / TURN, full = nb / TURN;
  const int across = (P.N + 16 * NB - 1) / (16 * NB);  // blocks to 16 activation rows
  const int n0 = (int)(blockIdx.x % across) * 16 * NB;
  const int r = (int)(blockIdx.x / across) * 16 + i;  // the lane's activation row
  size_t wrow[NB], drow[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    wrow[b] = (size_t)min(n0 + 16 * b + i, P.N - 1) * P.K;
#pragma unroll
    for (int j = 0; j < 4; ++j)  // the rows of the lane's results
      drow[b][j] = (size_t)min(n0 + 16 * b + 4 * g + j, P.N - 1) * nb;
  }
  const int xi = min(r, P.R - 1);
  const int8_t* const xq = P.xq + (size_t)xi * P.K;
  const float* const xd = P.xd + (size_t)xi * nb;
  f32x4_t acc[A];
#pragma unroll
  for (int a = 0; a < A; ++a) acc[a] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const auto turn = [&](auto tail, int u) {
    constexpr bool TAIL = decltype(tail)::value;
    constexpr int C = TURN / 2;
    const int b0 = u * TURN, left = nb - b0;  // blocks
    const i32x4_t zero = {0, 0, 0, 0};
    i32x4_t w[A][C], x[C];
    float d[TURN];
    uint16_t dw[A][4][TURN];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const bool past = TAIL && 2 * c + (g >> 1) >= left;
      const size_t at = (size_t)b0 * 32 + 64 * c + 16 * g;
#pragma unroll
      for (int a = 0; a < A; ++a)
        w[a][c] = past ? zero : *(const i32x4_t*)((a < NB ? P.wq : P.wq2) + wrow[a % NB] + at);
      x[c] = past ? zero : *(const i32x4_t*)(xq + at);
    }
    if constexpr (TAIL) {
#pragma unroll
      for (int b = 0; b < TURN; ++b) {
        d[b] = b < left ? xd[b0 + b] : 0.f;
#pragma unroll
        for (int a = 0; a < A; ++a)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            dw[a][j][b] = b < left ? (a < NB ? P.wd : P.wd2)[drow[a % NB][j] + b0 + b] : 0;
      }
    } else {  // no alignment but the types' own: a row has K / 32 scales
      __builtin_memcpy(d, xd + b0, sizeof d);
#pragma unroll
      for (int a = 0; a < A; ++a)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          __builtin_memcpy(dw[a][j], (a < NB ? P.wd : P.wd2) + drow[a % NB][j] + b0,
                           sizeof dw[a][j]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const i32x4_t half[2] = {g < 2 ? x[c] : zero, g < 2 ? zero : x[c]};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int a = 0; a < A; ++a) {
          const i32x4_t s = i8_mma(w[a][c], half[t]);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[a][j] = fmaf((float)s[j], f16_bits_to_f32(dw[a][j][2 * c + t]) * d[2 * c + t],
                             acc[a][j]);
        }
    }
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
      const f32x4_t v = sums[w][a][lane];
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
  if constexpr (NB == 2) leave_block<kOutQ8>(P.e, v[0], v[1], r, P.R, n0, P.N, g);
  else if (r < P.R) leave4<GLU>(P.e, v[0], (size_t)r, n0 + 4 * g, P.N);
}

static long long rows_blocks(const Q8Product& P, int cols) {
  return (long long)((P.N + cols - 1) / cols) * ((P.R + 15) / 16);
}
template <bool GLU, int NB>
static int launch_rows(const Q8Product& P, hipStream_t s) {
  const dim3 grid((unsigned)(rows_blocks(P, 16 * NB)));
  const int waves = std::min(q8_waves<GLU, NB>(), (P.K / 32 + q8_turn<GLU>() - 1) / q8_turn<GLU>());
  return QMOE_LAUNCH("q8_rows", (q8_rows_kernel<GLU, NB>), grid, 64 * waves, 0, s, P);
}

// ------------------------------------------------------ many rows ------
// A block computes BM = 32 WR TM activation rows x BN = 32 WC TN weight rows with
// WR x WC waves of TM x TN 32x32x32 ops, one to a 32-value block.  The products of a
// block's scales, dw[n] d[r] for 32 x 32 outputs, are a matrix product too, with one
// term: a 32x32x2 op in fp32 gives them rounded once, in the registers of the integer
// sums.  Those start from the bits of 1.5 2^23, so that a subtraction makes them fp32.
// That leaves the vector unit two operations an output and block.  700 x 2048 x 7168
// pairs take 110 us: with 16 x 16 ops and three vector operations 153, with these ops
// one after the other 112-147.  The fp32 op takes 64 cycles of the vector unit's own (a
// probe: it and 16 multiply-adds take the sum of both, the integer op hides behind
// them), about 211 a pair of ops in all; the scales as a bf16 op of their parts, which
// does overlap, gained 2 %, because waits for copies and barriers are 38 % of a wave
// (the loop over steps says which).
//
// K advances 128 values (four blocks) a step.  Codes go from memory to LDS without
// passing registers, whole 128-byte lines, into one of two buffers, a step ahead;
// scales pass through registers (their rows have any alignment) and lie as fp32, four to
// a row.  The 16-byte chunk c of tile row q lies at chunk c ^ ((q >> 1) & 7), so that the
// rows one operand read touches spread over the banks.  Rows past the ends repeat the
// last one and are never stored; blocks past K's end repeat the row's last one with
// scale 0.
//
// KS teams of WR x WC waves split K where there are too few tiles to fill the part,
// as in the MX tiles; a gated pair's weight rows are 32 of the gate, 32 of up.
template <int WR_, int WC_, int TM_, int TN_, int KS_>
struct Q8Tile {
  static constexpr int WR = WR_, WC = WC_, TM = TM_, TN = TN_, KS = KS_;
  static constexpr int BM = 32 * WR * TM, BN = 32 * WC * TN, ROWS = BM + BN, NW = WR * WC;
  static constexpr int TEAM = 64 * NW, THREADS = TEAM * KS;
  static constexpr int CODES = ROWS * 128, BUF = CODES + ROWS * 16;  // bytes
  static constexpr int JA = BM / 8 / NW, J = ROWS / 8 / NW;          // copies per wave and step
  static constexpr int SC = (ROWS + TEAM - 1) / TEAM;  // rows whose scales a thread loads
  static_assert(NW % 2 == 0 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && TN % 2 == 0, "");
  static constexpr int COLS = 32 * TN, PITCH = leave_pitch(COLS), OUT = NW * 32 * PITCH * 4;
  static constexpr int SUMS = TM * TN * 16 * TEAM * 4;
  static constexpr size_t LDS = std::max(KS * 2 * BUF, OUT + (KS - 1) * SUMS);
  static_assert(LDS <= 160 << 10, "");
};

// (Two waves to a SIMD leave a wave 256 registers, all of which the vector unit reads;
// with 512 the compiler puts the ops' results where it does not and copies each.)
template <class T, bool GLU>
__global__ __launch_bounds__(T::THREADS, T::THREADS > 256 ? 1 : 2) void q8_tile_kernel(
    Q8Product P, int tiles_m, int tiles_n) {
  constexpr int TM = T::TM, TN = T::TN, M = TM * TN;
  extern __shared__ __align__(16) uint8_t smem[];
  const int team = T::KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / T::TEAM);
  const int tid = threadIdx.x % T::TEAM, lane = tid & 63, i = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // a run of tiles to each XCD, down the rows first, as in the MX tiles
  const int T_ = tiles_m * tiles_n, per = T_ >> 3, extra = T_ & 7;
  const int xcd = blockIdx.x & 7;
  const int tile = xcd * per + min(xcd, extra) + (blockIdx.x >> 3);
  const int r0 = (tile % tiles_m) * T::BM, n0 = (tile / tiles_m) * (GLU ? T::BN / 2 : T::BN);
  const int nb = P.K >> 5, all = (nb + 3) >> 2;
  const int loops = (all + T::KS - 1) / T::KS;  // steps of a team, the last one's fewer
  const int first = team * loops, steps = min(max(all - first, 0), loops);
  uint8_t* const mem = smem + team * 2 * T::BUF;
  const int8_t* const abase = P.xq + (size_t)r0 * P.K;
  const int8_t* const bbase = P.wq + (size_t)n0 * P.K;
  const int8_t* const bbase2 = GLU ? P.wq2 + (size_t)n0 * P.K : nullptr;
  const int arows = P.R - r0 - 1, brows = P.N - n0 - 1;  // last valid row of the tile
  const auto weight = [](int q) { return GLU ? (q >> 6 << 5) + (q & 31) : q; };

  // Copy j of the wave fills 8 rows of the tile.
  const int rem = nb - 4 * (all - 1);  // blocks of K's last step, 1..4
  const int chunk = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);  // NW is even: for every j
  const uint32_t over = 32u * (uint32_t)max((chunk >> 1) - (rem - 1), 0);
  uint32_t off[T::J];
#pragma unroll
  for (int j = 0; j < T::J; ++j) {
    const int q = 8 * (wave + T::NW * (j < T::JA ? j : j - T::JA)) + (lane >> 3);
    const int row = j < T::JA ? min(q, arows) : min(weight(q), brows);
    off[j] = (uint32_t)row * (uint32_t)P.K + 16u * (uint32_t)chunk;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)mem;
  const auto copy = [&](int st, int j) {
    const int k = min(first + st, all - 1);  // past the team's steps: unused
    const int8_t* base = j < T::JA ? abase : bbase;
    if (GLU && j >= T::JA && ((wave + T::NW * (j - T::JA)) >> 2 & 1)) base = bbase2;
    copy_to_lds(lds0 + (st & 1) * T::BUF + (wave + T::NW * j) * 1024,
                uniform((const uint8_t*)base + (size_t)k * 128),
                off[j] - (k + 1 == all ? over : 0));
  };
  f32x4_t sreg[T::SC];
  const auto load_scales = [&](int st) {
    const int b0 = 4 * min(first + st, all - 1);
    const bool whole = b0 + 4 <= nb;
    static_for<T::SC>([&](auto j) {
      const int q = min(tid + j * T::TEAM, T::ROWS - 1), qb = q - T::BM;
      f32x4_t v = {0.f, 0.f, 0.f, 0.f};
      if (q < T::BM) {
        const float* d = P.xd + (size_t)(r0 + min(q, arows)) * nb + b0;
        if (whole) __builtin_memcpy(&v, d, 16);
        else
          for (int b = 0; b < nb - b0; ++b) v[b] = d[b];
      } else {
        const uint16_t* d = (GLU && (qb >> 5 & 1) ? P.wd2 : P.wd) +
                            (size_t)(n0 + min(weight(qb), brows)) * nb + b0;
        if (whole) {
          uint32_t w[2];
          __builtin_memcpy(w, d, 8);
          v = f32x4_t{f16_bits_to_f32(w[0] & 0xFFFFu), f16_bits_to_f32(w[0] >> 16),
                      f16_bits_to_f32(w[1] & 0xFFFFu), f16_bits_to_f32(w[1] >> 16)};
        } else {
          for (int b = 0; b < nb - b0; ++b) v[b] = f16_bits_to_f32(d[b]);
        }
      }
      sreg[j] = v;
    });
  };
  const auto store_scales = [&](int st) {
    static_for<T::SC>([&](auto j) {
      const int q = tid + j * T::TEAM;
      if (T::ROWS % T::TEAM == 0 || q < T::ROWS)
        *(f32x4_t*)(mem + (st & 1) * T::BUF + T::CODES + q * 16) = sreg[j];
    });
  };
  const int wm = (wave / T::WC) * 32 * TM, wn = (wave % T::WC) * 32 * TN;
  const auto row_of = [&](int r) {
    return r < TM ? wm + 32 * r + i : T::BM + wn + 32 * (r - TM) + i;
  };
  f32x16_t acc[TM][TN];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[m][n][j] = 0.f;
  // A step's 4 M pairs of ops in turn: the next pair is issued before the vector unit
  // takes the last one's results, and a block's operands are read a block ahead.
  i32x16_t bias;  // 1.5 2^23 as fp32: a sum below 2^22 added to its bits is added to it
#pragma unroll
  for (int j = 0; j < 16; ++j) bias[j] = 0x4B400000;
  const auto compute = [&](int st) {
    const uint8_t* const buf = mem + (st & 1) * T::BUF;
    f32x4_t sc[TM + TN];
    i32x4_t q[2][TM + TN];
    f32x16_t sum[2], mul[2];
    const auto read = [&](auto b) {
      static_for<TM + TN>([&](auto r) {
        q[b & 1][r] =
            *(const i32x4_t*)(buf + row_of(r) * 128 + 16 * ((2 * b + h) ^ ((i >> 1) & 7)));
      });
    };
    const auto sums = [&](auto t) {
      constexpr int b = t / M, m = t % M / TN, n = t % TN;
      sum[t & 1] = __builtin_bit_cast(f32x16_t, __builtin_amdgcn_mfma_i32_32x32x32_i8(
                       q[b & 1][m], q[b & 1][TM + n], bias, 0, 0, 0));
    };
    const auto muls = [&](auto t) {
      constexpr int b = t / M, m = t % M / TN, n = t % TN;
      f32x16_t zero;
#pragma unroll
      for (int j = 0; j < 16; ++j) zero[j] = 0.f;
      mul[t & 1] = __builtin_amdgcn_mfma_f32_32x32x2f32(sc[m][b], sc[TM + n][b], zero, 0, 0, 0);
    };
    read(Int<0>{});
    static_for<TM + TN>([&](auto r) {
      sc[r] = *(const f32x4_t*)(buf + T::CODES + row_of(r) * 16);
      // the op's second term is none: the upper lanes' scales are zero, on both sides,
      // since zero times a scale that is infinite would be NaN
      if (h) sc[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    });
    sums(Int<0>{});
    muls(Int<0>{});
    static_for<4 * M>([&](auto t) {
      constexpr int b = t / M, m = t % M / TN, n = t % TN;
      if constexpr (t % M == 0 && b < 3) read(Int<b + 1>{});
      if constexpr (t + 1 < 4 * M) sums(Int<t + 1>{});
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 16; ++j) sum[t & 1][j] -= 12582912.f;
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (t + 1 < 4 * M) muls(Int<t + 1>{});
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        acc[m][n][j] = fmaf(sum[t & 1][j], mul[t & 1][j], acc[m][n][j]);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // Buffer st & 1 holds step st.  A step asks for the next one's codes, stores that one's
  // scales and loads those of the one after it, then computes.  Vector loads return in
  // order and the compiler does not count the copies, so its waits for the scales (before
  // they are stored, before they are made fp32) are waits for the step's copies too: a
  // wave's arithmetic begins when they have come, and what runs meanwhile is the other
  // block on the unit, where there is one.  What is fetched past a team's steps repeats
  // the last one and is not used.
  static_for<T::J>([&](auto j) { copy(0, j); });
  load_scales(0);
  store_scales(0);
  load_scales(1);
  wait_copies();
  __syncthreads();
#pragma unroll 1
  for (int st = 0; st < loops; ++st) {
    static_for<T::J>([&](auto j) { copy(st + 1, j); });
    store_scales(st + 1);
    load_scales(st + 2);
    if (st < steps) compute(st);
    wait_copies();
    __syncthreads();
  }
  if constexpr (T::KS > 1) {
    float* const sums = (float*)(smem + T::OUT) + tid;
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (team > 0)
            sums[((team - 1) * M * 16 + (m * TN + n) * 16 + j) * T::TEAM] = acc[m][n][j];
    __syncthreads();
    if (team > 0) return;
#pragma unroll 1
    for (int t = 0; t < T::KS - 1; ++t)
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[m][n][j] += sums[(t * M * 16 + (m * TN + n) * 16 + j) * T::TEAM];
  }
  // Register 4 a + b of a 32 x 32 block is row 8 a + 4 h + b, column i.
  float* const out = (float*)smem + wave * 32 * T::PITCH;
  const Leave<T::COLS, GLU, kOutQ8> leave(P.e, out, n0 + (GLU ? wn / 2 : wn), P.R, P.N, lane);
  leave.template all<TM>(r0 + wm, [&](auto m) {
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int j = 0; j < 16; ++j)
        out[(8 * (j >> 2) + 4 * h + (j & 3)) * T::PITCH + 32 * n + i] =
            acc[decltype(m)::value][n][j];
  });
}

template <class T, bool GLU>
static int launch_q8(const Q8Product& P, hipStream_t s) {
  constexpr int cols = GLU ? T::BN / 2 : T::BN;
  const int tm = (P.R + T::BM - 1) / T::BM, tn = (P.N + cols - 1) / cols;
  // a kernel that takes more than 64 KB of LDS declares it, once per device
  static std::atomic<uint64_t> declared;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) dev = 64;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!bit || !(declared.load(std::memory_order_relaxed) & bit)) {
    (void)hipFuncSetAttribute((const void*)q8_tile_kernel<T, GLU>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, (int)T::LDS);
    declared.fetch_or(bit, std::memory_order_relaxed);
  }
  return QMOE_LAUNCH("q8_tile", (q8_tile_kernel<T, GLU>), dim3((unsigned)(tm * tn)), T::THREADS,
                     T::LDS, s, P, tm, tn);
}

struct Q8Choice {
  int bm, cols, threads, slots;
  float us, alone;
  int (*launch)(const Q8Product&, hipStream_t);
};
template <class T, bool GLU>
static constexpr Q8Choice q8_choice(int slots, float us, float alone) {
  return {T::BM, GLU ? T::BN / 2 : T::BN, T::THREADS, slots, us, alone, launch_q8<T, GLU>};
}

template <bool GLU>
static int run(const ProductCall& c, hipStream_t s) {
  const int st = check_product(c);
  if (st) return st == kNothing ? QMOE_OK : st;
  const Layout L = layout_of(QMOE_Q8_0, c.N, c.K);
  const uint8_t *w = (const uint8_t*)c.W, *w2 = (const uint8_t*)(GLU ? c.W2 : c.W);
  const Q8Product P{(const int8_t*)w + L.off[0], (const uint16_t*)(w + L.off[1]),
                    (const int8_t*)w2 + L.off[0], (const uint16_t*)(w2 + L.off[1]),
                    (const int8_t*)c.codes, (const float*)c.scales, c.N, c.K, c.R,
                    epilogue_of(c)};
  // Which kernel: as measured (us).  Both kinds go with K, so the choice does without it:
  // rounds of blocks times the time of one at K = 4096.
  //   rows  two blocks a unit 13, one 8, pairs 10.2 a block, quantized 19; a unit takes
  //     its blocks one after the other (from K = 4096 on 16 waves of 128 registers fill
  //     it).  49 x 535 (K = 3264) 7.1, with tiles 26.9; 64 x 4096 26.3, tiles 30.7;
  //     128 x 4096 50.4, tiles 30.8; 48 x 2048 (K = 14336) 37.8, tiles 105; pairs of
  //     64 x 2048 (K = 7168) 33.3, tiles 54.4; of 128 x 2048 64.7, tiles 55.0; 16 x 65536
  //     107, tiles 83
  //   32 x 128, three teams  a round of tiles 30
  //   64 x 128, two teams    37
  //   64 x 128               two to a unit 65, one 50
  //   128 x 128              two to a unit 109, one 75
  // Against the best for R from 8 to 2048, N from 2048 to 14336 and K from 1024 to 14336
  // (55 sizes, and as many of pairs) the choice takes at most 5 % longer but at 160 x 2048
  // (K = 1024: 10.8, rows 8.9; 14336: 107 and 93) and at pairs of 8 x 14336 (12.3, rows
  // 10.7; 145 and 119).
  const int cus = std::max(1, cu_count());
  const bool wide = GLU && P.e.out == kOutQ8;
  const long long blocks = rows_blocks(P, wide ? 32 : 16);
  const long long round = GLU ? cus : 2LL * cus, left = blocks % round;
  const float each = wide ? 19.f : GLU ? 10.2f : 13.f;
  float least = each * (float)(blocks / round) + (left == 0 ? 0.f : GLU || left > cus ? each : 8.f);
  static constexpr Q8Choice choices[] = {q8_choice<Q8Tile<1, 2, 1, 2, 3>, GLU>(1, 30.f, 30.f),
                                         q8_choice<Q8Tile<2, 2, 1, 2, 2>, GLU>(1, 37.f, 37.f),
                                         q8_choice<Q8Tile<2, 2, 1, 2, 1>, GLU>(2, 65.f, 50.f),
                                         q8_choice<Q8Tile<2, 2, 2, 2, 1>, GLU>(2, 109.f, 75.f)};
  const Q8Choice* best = nullptr;
  bool rows = blocks <= 0xFFFFFFFFLL / 1024;
  for (const Q8Choice& q : choices) {
    if (rows && P.R <= 4) break;  // a read of the weights: 1 x 65536 83 us, tiles 83
    const long long tiles = (long long)((P.R + q.bm - 1) / q.bm) * ((P.N + q.cols - 1) / q.cols);
    if (tiles > 0xFFFFFFFFLL / q.threads) continue;
    const long long at_once = (long long)q.slots * cus, last = tiles % at_once;
    const float us = q.us * (float)(tiles / at_once) +
                     (last == 0 ? 0.f : last <= cus ? q.alone : q.us);
    if ((!best && !rows) || us < least) best = &q, least = us, rows = false;
  }
  if (rows) {
    if constexpr (GLU)
      if (wide) return launch_rows<true, 2>(P, s);
    return launch_rows<GLU, 1>(P, s);
  }
  if (!best) return fail(QMOE_ERR_UNSUPPORTED, "%s: R=%d N=%d: too many tiles", c.who, c.R, c.N);
  return best->launch(P, s);
}

}  // namespace qmoe

using namespace qmoe;

extern "C" {

int qlinear_q8(const void* W, int N, int K, const int8_t* q, const float* d, int R,
               const float* bias, int act, const void* res, int res_dtype, void* y, int y_dtype,
               void* stream) {
  const ProductCall c{"qlinear_q8", QMOE_Q8_0, W, nullptr, false, N, K, q, d, R,
                      bias, nullptr, act, res, res_dtype, y, nullptr, plain_dtype(y_dtype)};
  return run<false>(c, (hipStream_t)stream);
}

int qglu_q8(const void* Wg, const void* Wu, int N, int K, const int8_t* q, const float* d, int R,
            const float* bias_gate, const float* bias_up, int act, void* y, int y_dtype,
            void* stream) {
  const ProductCall c{"qglu_q8", QMOE_Q8_0, Wg, Wu, true, N, K, q, d, R, bias_gate,
                      bias_up, act, nullptr, 0, y, nullptr, plain_dtype(y_dtype)};
  return run<true>(c, (hipStream_t)stream);
}

int qglu_q8_act(const void* Wg, const void* Wu, int N, int K, const int8_t* q, const float* d,
                int R, const float* bias_gate, const float* bias_up, int act, int8_t* out_q,
                float* out_d, void* stream) {
  const ProductCall c{"qglu_q8_act", QMOE_Q8_0, Wg, Wu, true, N, K, q, d, R,
                      bias_gate, bias_up, act, nullptr, 0, out_q, out_d, kQuantized};
  return run<true>(c, (hipStream_t)stream);
}

}  // extern "C"
