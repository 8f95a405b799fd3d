// Q8_0 weights x int8 activations with an epilogue: one product with bias,
// activation and residual (qlinear_q8), or the gated pair (qglu_q8, qglu_q8_act).
//
//   p[r, n] = sum_b (dw[n, b] d[r, b]) * sum_{k in b} qw[n, k] q[r, k]
//   y = act(p + bias) + res,  or  v = act(p_gate + bias_gate) * (p_up + bias_up)
//
// A 32-value block's integer sum is exact; its scaling and the sum over blocks are
// fp32.  That scaling is what bounds many rows: a conversion, a product of the two
// scales and a multiply-add for every output and block, 48 cycles of a SIMD beside
// the 16 that the matrix core takes for the block's 16 x 16 x 32 products.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "product.hpp"

#pragma clang fp contract(off)

namespace qmoe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

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
// A block computes 16 NB weight rows (of each product) x all activation rows, 16 at
// most; its waves split K in turns of 256 values (a pair: 128), and their sums meet in LDS in wave
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
  const int n0 = blockIdx.x * 16 * NB;
  size_t wrow[NB], drow[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    wrow[b] = (size_t)min(n0 + 16 * b + i, P.N - 1) * P.K;
#pragma unroll
    for (int j = 0; j < 4; ++j)  // the rows of the lane's results
      drow[b][j] = (size_t)min(n0 + 16 * b + 4 * g + j, P.N - 1) * nb;
  }
  const int xi = min(i, P.R - 1);
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
  if constexpr (NB == 2) leave_block<kOutQ8>(P.e, v[0], v[1], i, P.R, n0, P.N, g);
  else if (i < P.R) leave4<GLU>(P.e, v[0], (size_t)i, n0 + 4 * g, P.N);
}

template <bool GLU, int NB>
static int launch_rows(const Q8Product& P, hipStream_t s) {
  const dim3 grid((unsigned)((P.N + 16 * NB - 1) / (16 * NB)));
  const int waves = std::min(q8_waves<GLU, NB>(), (P.K / 32 + q8_turn<GLU>() - 1) / q8_turn<GLU>());
  return QMOE_LAUNCH("q8_rows", (q8_rows_kernel<GLU, NB>), grid, 64 * waves, 0, s, P);
}

// ------------------------------------------------------ many rows ------
// A block computes BM = 16 WR MI activation rows x BN = 64 WC weight rows with WR x WC
// waves of MI x 4 16x16 results.  K advances 64 values (two blocks) per step; a
// step's operand tiles are loaded once per block, 16 bytes a lane, one step ahead in
// registers, and written to one of two LDS buffers with 80-byte rows (64 + 16 of
// padding: the 16 rows one operand read touches fall on distinct banks).  Scales lie
// block-major behind them, so that the four rows of a result are one 16-byte read.
// Rows past the ends repeat the last one and are never stored; a block past K's end
// repeats the last one with scale 0.
//
// KS teams of WR x WC waves split K where there are too few tiles to fill the part,
// as in the MX tiles; a gated pair's weight rows are 32 of the gate, 32 of up.
template <int WR_, int WC_, int MI_, int KS_>
struct Q8Tile {
  static constexpr int WR = WR_, WC = WC_, MI = MI_, KS = KS_, NB = 4;
  static constexpr int BM = 16 * WR * MI, BN = 64 * WC, ROWS = BM + BN, NW = WR * WC;
  static constexpr int TEAM = 64 * NW, THREADS = TEAM * KS;
  static constexpr int ROW = 80, BUF = ROWS * (ROW + 8);  // bytes: codes, then two scales a row
  static constexpr int CH = ROWS * 4 / TEAM;              // 16-byte chunks per thread and step
  static constexpr int SC = (ROWS + TEAM - 1) / TEAM;     // rows whose scales a thread loads
  static_assert(MI % 2 == 0 && ROWS * 4 % TEAM == 0 && BM * 4 % TEAM == 0, "");
  static constexpr int PITCH = leave_pitch(64), OUT = NW * 32 * PITCH * 4;
  static constexpr int SUMS = MI * NB * 4 * TEAM * 4;
  static constexpr size_t LDS = std::max(KS * 2 * BUF, OUT + (KS - 1) * SUMS);
  static_assert(LDS <= 160 << 10, "");
};

template <class T, bool GLU>
__global__ __launch_bounds__(T::THREADS) void q8_tile_kernel(Q8Product P, int tiles_m) {
  constexpr int MI = T::MI, NB = T::NB;
  extern __shared__ __align__(16) uint8_t smem[];
  const int team = T::KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / T::TEAM);
  const int tid = threadIdx.x % T::TEAM, lane = tid & 63, li = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = (int)(blockIdx.x % tiles_m) * T::BM;
  const int n0 = (int)(blockIdx.x / tiles_m) * (GLU ? T::BN / 2 : T::BN);
  const int nb = P.K >> 5, all = (nb + 1) >> 1;
  const int loops = (all + T::KS - 1) / T::KS;  // steps of a team, the last one's fewer
  const int first = team * loops, steps = min(max(all - first, 0), loops);
  uint8_t* const mem = smem + team * 2 * T::BUF;
  const auto codes = [&](int buf) { return mem + buf * T::BUF; };
  const auto scales = [&](int buf) { return (float*)(mem + buf * T::BUF + T::ROWS * T::ROW); };
  const auto weight = [](int q) { return GLU ? (q >> 6 << 5) + (q & 31) : q; };
  const auto is_up = [](int q) { return GLU && (q >> 5 & 1); };

  // chunk c = tid + j TEAM: row c >> 2 of the tile (activations first), bytes 16 (c & 3)
  const int8_t* src[T::CH];
#pragma unroll
  for (int j = 0; j < T::CH; ++j) {
    const int q = (tid + j * T::TEAM) >> 2, qb = q - T::BM;
    src[j] = q < T::BM ? P.xq + (size_t)min(r0 + q, P.R - 1) * P.K
                       : (is_up(qb) ? P.wq2 : P.wq) + (size_t)min(n0 + weight(qb), P.N - 1) * P.K;
  }
  i32x4_t cr[T::CH];
  float sr[T::SC][2];
  const auto load = [&](int st) {
    const int b0 = 2 * min(first + st, all - 1), b1 = min(b0 + 1, nb - 1);
    const bool second = b0 + 1 < nb;
    const int ch = 16 * (tid & 3);  // TEAM is a multiple of 4
    const int k0 = ch < 32 ? b0 * 32 + ch : b1 * 32 + ch - 32;
    static_for<T::CH>([&](auto j) { cr[j] = *(const i32x4_t*)(src[j] + k0); });
    static_for<T::SC>([&](auto j) {
      const int q = min(tid + j * T::TEAM, T::ROWS - 1), qb = q - T::BM;
      if (q < T::BM) {
        const float* d = P.xd + (size_t)min(r0 + q, P.R - 1) * nb;
        sr[j][0] = d[b0];
        sr[j][1] = second ? d[b1] : 0.f;
      } else {
        const uint16_t* d =
            (is_up(qb) ? P.wd2 : P.wd) + (size_t)min(n0 + weight(qb), P.N - 1) * nb;
        sr[j][0] = f16_bits_to_f32(d[b0]);
        sr[j][1] = second ? f16_bits_to_f32(d[b1]) : 0.f;
      }
    });
  };
  const auto write = [&](int buf) {
    static_for<T::CH>([&](auto j) {
      const int c = tid + j * T::TEAM;
      *(i32x4_t*)(codes(buf) + (c >> 2) * T::ROW + 16 * (c & 3)) = cr[j];
    });
    static_for<T::SC>([&](auto j) {
      const int q = tid + j * T::TEAM;
      if (T::ROWS % T::TEAM == 0 || q < T::ROWS) {
        scales(buf)[q] = sr[j][0];
        scales(buf)[T::ROWS + q] = sr[j][1];
      }
    });
  };
  const int wm = (wave / T::WC) * 16 * MI, wn = (wave % T::WC) * 64;
  f32x4_t acc[MI][NB];
#pragma unroll
  for (int m = 0; m < MI; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[m][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const auto compute = [&](int buf) {
    // one block at a time: unrolling both keeps twice the operands live
#pragma unroll 1
    for (int kb = 0; kb < 2; ++kb) {
      // lane (li, g) supplies codes 8 g .. + 7 of the block of its row; the result
      // holds activation rows 4 g + j, weight row li
      long bq[NB], aq[MI];
      float bs[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int q = T::BM + wn + 16 * b + li;
        bq[b] = *(const long*)(codes(buf) + q * T::ROW + 32 * kb + 8 * g);
        bs[b] = scales(buf)[kb * T::ROWS + q];
      }
#pragma unroll
      for (int m = 0; m < MI; ++m)
        aq[m] = *(const long*)(codes(buf) + (wm + 16 * m + li) * T::ROW + 32 * kb + 8 * g);
      i32x4_t is[MI][NB];
#pragma unroll
      for (int m = 0; m < MI; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          is[m][b] = __builtin_amdgcn_mfma_i32_16x16x32_i8(aq[m], bq[b], i32x4_t{0, 0, 0, 0}, 0,
                                                          0, 0);
#pragma unroll
      for (int m = 0; m < MI; ++m) {
        const float4 a4 = *(const float4*)(scales(buf) + kb * T::ROWS + wm + 16 * m + 4 * g);
        const float as[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[m][b][j] = fmaf((float)is[m][b][j], as[j] * bs[b], acc[m][b][j]);
      }
    }
  };
  // buffer st & 1 holds step st; the next one is on its way in registers.  Loads past
  // the team's steps repeat the last one: their buffer is not used.
  load(0);
  write(0);
  __syncthreads();
  load(1);
  for (int st = 0; st < loops; ++st) {
    if (st < steps) compute(st & 1);
    write((st + 1) & 1);
    __syncthreads();
    load(st + 2);
  }
  if constexpr (T::KS > 1) {
    float* const sums = (float*)(smem + T::OUT) + tid;
#pragma unroll
    for (int m = 0; m < MI; ++m)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (team > 0)
            sums[((team - 1) * MI * NB * 4 + (m * NB + b) * 4 + j) * T::TEAM] = acc[m][b][j];
    __syncthreads();
    if (team > 0) return;
#pragma unroll 1
    for (int t = 0; t < T::KS - 1; ++t)
#pragma unroll
      for (int m = 0; m < MI; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[m][b][j] += sums[(t * MI * NB * 4 + (m * NB + b) * 4 + j) * T::TEAM];
  }
  float* const out = (float*)smem + wave * 32 * T::PITCH;
  const Leave<64, GLU, kOutQ8> leave(P.e, out, n0 + (GLU ? wn / 2 : wn), P.R, P.N, lane);
#pragma unroll
  for (int m = 0; m < MI; m += 2) {
    const int row0 = r0 + wm + 16 * m;
    const auto res = leave.residual(row0);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          out[(16 * t + 4 * g + j) * T::PITCH + 16 * b + li] = acc[m + t][b][j];
    leave.rows(row0, res);
  }
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
                     T::LDS, s, P, tm);
}

struct Q8Choice {
  int bm, cols, threads, slots;
  float us;
  int (*launch)(const Q8Product&, hipStream_t);
};
template <class T, bool GLU>
static constexpr Q8Choice q8_choice(int slots, float us) {
  return {T::BM, GLU ? T::BN / 2 : T::BN, T::THREADS, slots, us, launch_q8<T, GLU>};
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
  if (P.R <= 16) {
    if constexpr (GLU)
      if (P.e.out == kOutQ8) return launch_rows<true, 2>(P, s);
    return launch_rows<GLU, 1>(P, s);
  }
  // rounds of tiles times the time of one, as for the MX tiles
  static constexpr Q8Choice choices[] = {q8_choice<Q8Tile<1, 2, 2, 4>, GLU>(1, 30.f),
                                         q8_choice<Q8Tile<2, 2, 2, 2>, GLU>(1, 45.f),
                                         q8_choice<Q8Tile<2, 2, 4, 1>, GLU>(2, 130.f)};
  const int cus = std::max(1, cu_count());
  const Q8Choice* best = nullptr;
  float least = 0.f;
  for (const Q8Choice& q : choices) {
    const long long tiles = (long long)((P.R + q.bm - 1) / q.bm) * ((P.N + q.cols - 1) / q.cols);
    if (tiles > 0xFFFFFFFFLL / q.threads) continue;
    const long long at_once = (long long)q.slots * cus;
    const float us = q.us * (float)((tiles + at_once - 1) / at_once);
    if (!best || us < least) best = &q, least = us;
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
