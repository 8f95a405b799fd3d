// MXFP4 weights x MXFP4 activations on the block-scaled matrix cores.
//
//   y[r, n] = sum_k w[n, k] x[r, k]
//
// Both operands are E2M1 codes with one E8M0 scale per 32 values along K, used
// as stored: every product of two codes is exact, the matrix op applies both
// scales and accumulates in fp32.
#include <algorithm>
#include <atomic>
#include <type_traits>

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

QMOE_D v4f_t mma4(uint4 a, uint32_t sa, uint4 b, uint32_t sb, v4f_t c) {
  const v8i_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// ------------------------------------------------------ few rows ------
// A block computes 16 weight rows x all activation rows, 16 at most, with 16x16x128
// ops; its waves split K in turns of 512 values, and their sums meet in LDS in wave order.
// Operands go from memory to registers, a whole turn's loads together: with few
// rows the call is a read of the weights, and what counts is how many of them
// are on their way.
//
// Lane 16 g + i of step j takes block 4 j + g of the turn from row i, so that a
// load reads 64 consecutive bytes of each of 16 rows.  (Four consecutive blocks
// to a lane would put its scales into one word, but a load then touches four
// times as many cache sectors: 1 x 4096 x 4096 takes 4.6 us instead of 4.3.)  The
// lane's scale of step j is byte g of the row's j-th scale word.
struct Frag {  // one lane's part of a turn
  uint4 q[4];
  uint32_t s[4];
};
// `row` counts the plane's blocks before the row; blocks from nb on (past the
// row's end) are zeros.
template <bool TAIL>
QMOE_D void load_codes(const uint8_t* q, size_t row, int b, int nb, uint4& v) {
  if (TAIL && b >= nb) v = make_uint4(0, 0, 0, 0);
  else v = *(const uint4*)(q + (row + b) * 16);
}
template <bool TAIL>
QMOE_D void load_scales(const uint8_t* s, size_t row, int b0, int g, int nb, Frag& f) {
  if constexpr (TAIL) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f.s[j] = b0 + 4 * j + g < nb ? s[row + b0 + 4 * j + g] : 0;
  } else {
    uint32_t w[4];  // no alignment: a row has K / 32 bytes
    __builtin_memcpy(w, s + row + b0, 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.s[j] = w[j] >> (8 * g);
  }
}

// a wave per turn where there are that many: 1 x 4096 x 14336 takes 8.3 us, with
// 8 waves 9.6
constexpr int kRowsWaves = 16;

template <bool YBF>
__global__ __launch_bounds__(64 * kRowsWaves) void mxfp4_rows_kernel(Mx4Params P) {
  __shared__ v4f_t sums[kRowsWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int nb = P.K >> 5, turns = (nb + 15) >> 4, full = nb >> 4;
  const int n0 = blockIdx.x * 16;
  const size_t wrow = (size_t)min(n0 + i, P.N - 1) * nb, xrow = (size_t)min(i, P.R - 1) * nb;
  v4f_t acc = v4f_t{0.f, 0.f, 0.f, 0.f};
  const auto turn = [&](auto tail, int u) {
    constexpr bool TAIL = decltype(tail)::value;
    Frag w, x;
    load_scales<TAIL>(P.ws, wrow, 16 * u, g, nb, w);
    load_scales<TAIL>(P.xs, xrow, 16 * u, g, nb, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      load_codes<TAIL>(P.wq, wrow, 16 * u + 4 * j + g, nb, w.q[j]);
      load_codes<TAIL>(P.xq, xrow, 16 * u + 4 * j + g, nb, x.q[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = mma4(w.q[j], w.s[j], x.q[j], x.s[j], acc);
  };
  int u = wave;
  for (; u < full; u += waves) turn(std::false_type{}, u);
  if (u < turns) turn(std::true_type{}, u);  // the last, partial turn
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
  for (int w = 1; w < waves; ++w) {
    const v4f_t v = sums[w][lane];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += v[j];
  }
  // lane 16 g + i: weight rows 4 g .. + 3 of activation row i
  const int n = n0 + 4 * g;
  if (i >= P.R) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (n + j >= P.N) break;
    const size_t at = (size_t)i * P.N + n + j;
    if constexpr (YBF) ((uint16_t*)P.y)[at] = (uint16_t)f32_to_bf16_bits(acc[j]);
    else ((float*)P.y)[at] = acc[j];
  }
}

static int launch_rows(const Mx4Params& P, bool ybf, hipStream_t s) {
  const dim3 grid((unsigned)((P.N + 15) / 16));
  const int waves = std::min(kRowsWaves, (P.K / 32 + 15) / 16);
  if (ybf) return QMOE_LAUNCH("mxfp4_rows", mxfp4_rows_kernel<true>, grid, 64 * waves, 0, s, P);
  return QMOE_LAUNCH("mxfp4_rows", mxfp4_rows_kernel<false>, grid, 64 * waves, 0, s, P);
}

// ------------------------------------------------------ many rows ------
// A block computes BM = 32 WR TM activation rows x BN = 32 WC TN weight rows
// with WR x WC waves of TM x TN 32x32x64 ops.  A step is 256 values of K, 128
// code bytes of a row: four groups of ops, lane 32 h + i of group s taking block
// 2 s + h of row i.
//
// With the largest tile a SIMD holds one wave (its sums fill half the registers),
// so whatever that wave waits for, the matrix core waits for too; the smaller ones
// have two to four.  Everything else is therefore issued between matrix ops, in an
// order that the compiler keeps:
//  * codes go from memory to LDS without passing registers (16 bytes a lane,
//    1 KB of LDS, 8 rows of 128 bytes, each a whole cache line: half lines
//    doubled the requests to L2, which then set the pace), into one of two
//    buffers, a step ahead;
//  * the operands of a group are read from LDS during the group before it; the
//    step's barrier stands before its last group, when every wave holds the
//    rest of the step's operands, and frees the step's buffer;
//  * scales pass through registers (their rows have any alignment): 16 bytes a
//    row serve two steps, in one of two LDS buffers; a byte permute gives each
//    lane its four blocks of a step in one word, whose bytes the ops select.
// The 16-byte chunk c of tile row q lies at chunk c ^ ((q >> 1) & 7), chosen by
// which chunk of memory a lane fetches, so that the rows one operand read
// touches spread over the banks.  Rows past the ends repeat the last one and
// are never stored; blocks past K's end repeat the row's last one with scale
// bytes of 0, and 2^-127 from either side leaves nothing of their products.
//
// KS teams of WR x WC waves split K where there are too few tiles to fill the
// part: each takes a run of whole turns (two steps) with buffers of its own,
// and the first team adds the others' sums to its own in team order.
template <int WR_, int WC_, int TM_, int TN_, int KS_ = 1>
struct Tile {
  static constexpr int WR = WR_, WC = WC_, TM = TM_, TN = TN_, KS = KS_;
  static constexpr int BM = 32 * WR * TM, BN = 32 * WC * TN, ROWS = BM + BN, NW = WR * WC;
  static constexpr int TEAM = 64 * NW, THREADS = TEAM * KS;
  static constexpr int CODES = ROWS * 128, SCALES = ROWS * 16;  // bytes of one buffer
  static constexpr int TEAM_LDS = 2 * (CODES + SCALES);
  static constexpr int JA = BM / 8 / NW, J = ROWS / 8 / NW;     // copies per wave and step
  static constexpr int J1 = J / 2;                              // of them in the first part
  static constexpr int SR = (ROWS + TEAM - 1) / TEAM;           // scale rows per thread
  static_assert(NW % 2 == 0 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "");
  // leaving: 32 rows of a wave's columns, then the other teams' sums
  static constexpr int COLS = 32 * TN, PITCH = COLS + 8, OUT = NW * 32 * PITCH * 4;
  static constexpr int SUMS = TM * TN * 16 * TEAM * 4;
  static constexpr size_t LDS = std::max(KS * TEAM_LDS, OUT + (KS - 1) * SUMS);
  static_assert(LDS <= 160 << 10, "");
};

typedef float v16f_t __attribute__((ext_vector_type(16)));

template <int SEL>
QMOE_D v16f_t mma4_32(uint4 a, uint32_t sa, uint4 b, uint32_t sb, v16f_t c) {
  const v8i_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, SEL, (int)sa, SEL,
                                                         (int)sb);
}

// a block-uniform address in scalar registers
QMOE_D const uint8_t* uniform(const uint8_t* p) {
  const uint64_t a = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  return (const uint8_t*)((uint64_t)hi << 32 | lo);
}

// 16 bytes a lane from base + off to LDS address lds + 16 * lane.  It has no
// output register; its completion is counted with the vector loads, in order,
// and waited for by wait_copies before the barrier that hands the data over.
// The compiler does not count it: its own waits for vector loads can only be
// longer than needed.  m0 is declared as written, so that no value of the
// compiler's own is taken to survive there (its warning that m0 is one of its
// reserved registers is expected).
QMOE_D void copy_to_lds(uint32_t lds, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(off), "s"(base)
               : "m0", "memory");
}
QMOE_D void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <class T, bool YBF>
__global__ __launch_bounds__(T::THREADS) void mxfp4_tile_kernel(Mx4Params P, int tiles_m,
                                                                int tiles_n) {
  constexpr int TM = T::TM, TN = T::TN, M = TM * TN, NR = TM + TN;
  extern __shared__ __align__(16) uint8_t smem[];
  const int team = T::KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / T::TEAM);
  const int tid = threadIdx.x % T::TEAM, lane = tid & 63, i = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint8_t* const mem = smem + team * T::TEAM_LDS;
  // Blocks are dealt to the 8 XCDs in turn: give each XCD one run of tiles,
  // down the rows first, so that its L2 serves both operands' reuse.
  const int T_ = tiles_m * tiles_n, per = T_ >> 3, extra = T_ & 7;
  const int x = blockIdx.x & 7;
  const int tile = x * per + min(x, extra) + (blockIdx.x >> 3);
  const int r0 = (tile % tiles_m) * T::BM, n0 = (tile / tiles_m) * T::BN;
  // this team's steps [first, first + steps) of K's `all`; every team goes
  // through `loops` of them, idle past its own
  const int nb = P.K >> 5, all = (nb + 7) >> 3;
  const int loops = 2 * ((all + 2 * T::KS - 1) / (2 * T::KS));
  const int first = team * loops;
  const int steps = min(max(all - first, 0), loops), turns = (steps + 1) >> 1;
  const uint32_t rowb = (uint32_t)P.K >> 1;
  const uint8_t* const abase = P.xq + (size_t)r0 * rowb;
  const uint8_t* const bbase = P.wq + (size_t)n0 * rowb;
  const int arows = P.R - r0 - 1, brows = P.N - n0 - 1;  // last valid row of the tile

  // Copy j of the wave fills tile rows 8 (wave + NW j) .. + 7, and NW is even,
  // so the lane's chunk is the same for every j.
  const int rem = nb - 8 * (all - 1);  // blocks of K's last step, 1..8
  const int chunk = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
  const uint32_t over = 16u * (uint32_t)max(chunk - (rem - 1), 0);
  uint32_t off[T::J];
#pragma unroll
  for (int j = 0; j < T::J; ++j) {
    const int q = 8 * (wave + T::NW * j) + (lane >> 3);
    const int row = j < T::JA ? min(q, arows) : min(q - T::BM, brows);
    off[j] = (uint32_t)row * rowb + 16u * (uint32_t)chunk;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)mem;
  const auto copy = [&](int st, int j) {
    const int k = min(first + st, all - 1);  // past the team's steps: unused
    copy_to_lds(lds0 + (st & 1) * T::CODES + (wave + T::NW * j) * 1024,
                uniform((j < T::JA ? abase : bbase) + (size_t)k * 128),
                off[j] - (k + 1 == all ? over : 0));
  };
  // scales of the team's turns (16 blocks), tile row q at 16 q; 0 past K's end
  uint8_t* const sc = mem + 2 * T::CODES;
  uint4 sreg[T::SR];
  const auto load_scales = [&](int turn) {
    const int u = (first >> 1) + turn;
#pragma unroll
    for (int j = 0; j < T::SR; ++j) {
      const int q = tid + j * T::TEAM;
      const uint8_t* p = (q < T::BM ? P.xs + (size_t)(r0 + min(q, arows)) * nb
                                    : P.ws + (size_t)(n0 + min(q - T::BM, brows)) * nb) + 16 * u;
      if (16 * u + 16 <= nb) {
        __builtin_memcpy(&sreg[j], p, 16);
      } else {
        uint64_t lo = 0, hi = 0;
#pragma unroll 1
        for (int b = nb - 16 * u - 1; b >= 0; --b) {
          hi = hi << 8 | lo >> 56;
          lo = lo << 8 | p[b];
        }
        sreg[j] = make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
      }
    }
  };
  const auto store_scales = [&](int u) {
#pragma unroll
    for (int j = 0; j < T::SR; ++j) {
      const int q = tid + j * T::TEAM;
      if (T::ROWS % T::TEAM == 0 || q < T::ROWS)
        *(uint4*)(sc + (u & 1) * T::SCALES + q * 16) = sreg[j];
    }
  };
  const int wm = (wave / T::WC) * 32 * TM, wn = (wave % T::WC) * 32 * TN;
  const int qa = wm + i, qb = T::BM + wn + i;  // the lane's rows of the first ops
  v16f_t acc[TM][TN];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[m][n][j] = 0.f;

  struct Ops {
    uint4 v[NR];  // TM activation rows, then TN weight rows
  };
  struct Scl {
    uint32_t v[NR];
  };
  // operands in the order the ops use them: a0, b0 .. , a1 ..
  const auto nth = [](int r) { return r == 0 ? 0 : r <= TN ? TM + r - 1 : r - TN; };
  const auto row_of = [&](int r) { return r < TM ? qa + 32 * r : qb + 32 * (r - TM); };
  const auto read_op = [&](int st, int s, int r, Ops& o) {
    o.v[r] = *(const uint4*)(mem + (st & 1) * T::CODES + row_of(r) * 128 +
                             16 * ((2 * s + h) ^ ((i >> 1) & 7)));
  };
  uint2 raw[NR];  // a row's scales of the next step
  const auto read_raw = [&](int st, int r) {
    raw[r] = *(const uint2*)(sc + ((st >> 1) & 1) * T::SCALES + row_of(r) * 16 + 8 * (st & 1));
  };
  const uint32_t pick = h ? 0x07050301u : 0x06040200u;
  const auto sort_raw = [&](int r, Scl& c) {
    c.v[r] = __builtin_amdgcn_perm(raw[r].y, raw[r].x, pick);
  };
  // one group of ops with `side(n)` issued after the n-th
  const auto group = [&](auto sel, const Ops& o, const Scl& c, auto&& side) {
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int n = 0; n < TN; ++n) {
        acc[m][n] = mma4_32<decltype(sel)::value>(o.v[m], c.v[m], o.v[TM + n], c.v[TM + n],
                                                  acc[m][n]);
        side(m * TN + n);
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  // of `count` things spread over a group's M slots, those of slot n
  const auto spread = [](int n, int count, auto&& f) {
#pragma unroll
    for (int k = n * count / M; k < (n + 1) * count / M; ++k) f(k);
  };
  // of `count` things early in a group (the next group needs them), those of slot n
  const auto early = [](int n, int count, auto&& f) {
    constexpr int per_slot = (2 * NR + M - 1) / M;
#pragma unroll
    for (int k = n * per_slot; k < min(count, (n + 1) * per_slot); ++k) f(k);
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;

  Ops f0, f1;
  Scl cur;
  // Step st, of parity k, with LEFT more to follow (2: two or more).  Known to
  // the compiler: a branch among the ops would end what it may reorder and
  // count across.
  const auto step = [&](auto kk, auto left, int st) {
    constexpr int k = decltype(kk)::value, LEFT = decltype(left)::value;
    const bool live = (T::KS == 1 && LEFT > 0) || st < steps;
    if (live) {
      group(I0{}, f0, cur, [&](int n) {
        early(n, NR, [&](int r) { read_op(k, 1, nth(r), f1); });
        if constexpr (LEFT >= 1) spread(n, T::J - T::J1, [&](int j) { copy(st + 1, T::J1 + j); });
      });
      group(I1{}, f1, cur, [&](int n) {
        early(n, NR, [&](int r) { read_op(k, 2, nth(r), f0); });
        if constexpr (LEFT >= 1) spread(n, NR, [&](int r) { read_raw(st + 1, r); });
      });
      group(I2{}, f0, cur, [&](int n) {
        early(n, NR, [&](int r) { read_op(k, 3, nth(r), f1); });
      });
    }
    if constexpr (LEFT >= 1) {
      wait_copies();
      __syncthreads();  // step st + 1 is there, and every wave holds the rest of st
      // The scales of the turn after st + 1's, loaded a turn ago: ahead of the
      // copies, because the compiler's wait for those loads waits for all.
      if (k == 1 && (st >> 1) + 2 < turns) {
        store_scales((st >> 1) + 2);
        if ((st >> 1) + 3 < turns) load_scales((st >> 1) + 3);
      }
    }
    if (live) {
      group(I3{}, f1, cur, [&](int n) {
        if constexpr (LEFT >= 1) early(n, NR, [&](int r) { read_op(k + 1, 0, nth(r), f0); });
        if constexpr (LEFT >= 2) spread(n, T::J1, [&](int j) { copy(st + 2, j); });
      });
      if constexpr (LEFT >= 1) {
#pragma unroll
        for (int r = 0; r < NR; ++r) sort_raw(r, cur);
      }
    }
  };

#pragma unroll
  for (int j = 0; j < T::J; ++j) copy(0, j);
  if (turns > 0) {
    load_scales(0);
    store_scales(0);
  }
  if (turns > 1) {
    load_scales(1);
    store_scales(1);
  }
  if (turns > 2) load_scales(2);
  wait_copies();
  __syncthreads();
#pragma unroll
  for (int j = 0; j < T::J1; ++j) copy(1, j);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    read_op(0, 0, r, f0);
    read_raw(0, r);
  }
#pragma unroll
  for (int r = 0; r < NR; ++r) sort_raw(r, cur);
  int st = 0;
#pragma unroll 1
  for (; st + 2 < loops; st += 2) {  // loops is even
    step(I0{}, I2{}, st);
    step(I1{}, I2{}, st + 1);
  }
  step(I0{}, I1{}, st);
  step(I1{}, I0{}, st + 1);
  if constexpr (T::KS > 1) {
    __syncthreads();
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

  // The sums leave through LDS, 32 rows of the wave's columns at a time, so
  // that a lane stores 16 bytes of one row.  Register 4 a + b of a 32 x 32 block
  // is row 8 a + 4 h + b, column i; rows lie 8 words more than a multiple of 64
  // apart, which puts the two halves' rows on different banks.
  if constexpr (T::KS == 1) __syncthreads();  // every wave has read its last operands
  constexpr int COLS = T::COLS, PITCH = T::PITCH;
  float* const out = (float*)smem + wave * 32 * PITCH;
  constexpr int E = YBF ? 8 : 4;  // values in 16 bytes
  const bool wide = P.N % E == 0;
#pragma unroll
  for (int m = 0; m < TM; ++m) {
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int j = 0; j < 16; ++j)
        out[(8 * (j >> 2) + 4 * h + (j & 3)) * PITCH + 32 * n + i] = acc[m][n][j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the region is this wave's own
    const int row0 = r0 + wm + 32 * m, col0 = n0 + wn;
    if (wide) {
      constexpr int LR = COLS / E;  // lanes to a row, a power of two
#pragma unroll
      for (int z = 0; z < 32 * LR / 64; ++z) {
        const int row = (z * 64 + lane) / LR, col = (lane % LR) * E;
        if (row0 + row < P.R && col0 + col < P.N) {
          const size_t at = (size_t)(row0 + row) * P.N + col0 + col;
          const float4* p = (const float4*)(out + row * PITCH + col);
          if constexpr (YBF) {
            const float4 u = p[0], v = p[1];
            *(uint4*)((uint16_t*)P.y + at) = make_uint4(pack_bf16(u.x, u.y), pack_bf16(u.z, u.w),
                                                        pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
          } else {
            *(float4*)((float*)P.y + at) = p[0];
          }
        }
      }
    } else {
      for (int o = lane; o < 32 * COLS; o += 64) {
        const int row = o / COLS, col = o % COLS;
        if (row0 + row < P.R && col0 + col < P.N) {
          const size_t at = (size_t)(row0 + row) * P.N + col0 + col;
          const float v = out[row * PITCH + col];
          if constexpr (YBF) ((uint16_t*)P.y)[at] = (uint16_t)f32_to_bf16_bits(v);
          else ((float*)P.y)[at] = v;
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

template <class T>
static int launch_tile(const Mx4Params& P, bool ybf, hipStream_t s) {
  const int tm = (P.R + T::BM - 1) / T::BM, tn = (P.N + T::BN - 1) / T::BN;
  const dim3 grid((unsigned)(tm * tn));
  // a kernel that takes more than 64 KB of LDS declares it, once per device
  static std::atomic<uint64_t> declared[2];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) dev = 64;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!bit || !(declared[ybf].load(std::memory_order_relaxed) & bit)) {
    (void)hipFuncSetAttribute(ybf ? (const void*)mxfp4_tile_kernel<T, true>
                                  : (const void*)mxfp4_tile_kernel<T, false>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, (int)T::LDS);
    declared[ybf].fetch_or(bit, std::memory_order_relaxed);
  }
  if (ybf)
    return QMOE_LAUNCH("mxfp4_tile", (mxfp4_tile_kernel<T, true>), grid, T::THREADS, T::LDS, s, P,
                       tm, tn);
  return QMOE_LAUNCH("mxfp4_tile", (mxfp4_tile_kernel<T, false>), grid, T::THREADS, T::LDS, s, P,
                     tm, tn);
}

struct Choice {
  int bm, bn, threads, slots;
  float us;
  int (*launch)(const Mx4Params&, bool, hipStream_t);
};
template <class T>
static constexpr Choice choice(int slots, float us) {
  return {T::BM, T::BN, T::THREADS, slots, us, launch_tile<T>};
}

// Which kernel.  A round of tiles takes about as long as one tile, so with K
// given the choice goes by rounds times the time of one: as measured at K = 4096
// (us), with `slots` tiles to a compute unit.
//   rows   1 x 4096: 4.3, 16 x 4096: 5.1; 32 x 64: 6.6
//   32 x 64, four teams  128 x 4096: 6.9;  64 x 64: 8.5;  64 x 128: 11
//   64 x 64, four teams  64 x 14336: 10.7; 32 x 64: 15.0; 64 x 128: 14.8
//   64 x 128, two teams  512 x 4096: 11.4; 64 x 64: 14.3; 128 x 128: 13.0
//   128 x 128, two teams 256 x 14336: 15.2; 64 x 128: 20.9; 256 x 256: 28.6
//   128 x 128, two to a unit  2048 x 4096: 25.4; two teams: 30.0; 256 x 256: 30.2
//   256 x 256  2048 x 14336: 70; 128 x 128: 86
// The rule has no term for K.  Against the best of the six for R from 40 to 2048
// and N from 2048 to 14336 its choice takes at most 5 % longer at K = 4096, 6 % at
// 1024, 9 % at 14336 (700 x 4096: 40.2 and 36.9), and at 256, where the teams'
// tiles are short of steps, 22 % (700 x 14336: 13.4 and 11.0).
// A launch has fewer than 2^32 threads: a tile that would need more is passed over.
static int launch_product(const Mx4Params& P, bool ybf, hipStream_t s) {
  const int cus = std::max(1, cu_count());
  if (P.R <= 16 && P.N <= 32 * cus) return launch_rows(P, ybf, s);
  static constexpr Choice choices[] = {
      choice<Tile<1, 2, 1, 1, 4>>(1, 7.f),  choice<Tile<2, 2, 1, 1, 4>>(1, 9.5f),
      choice<Tile<2, 2, 1, 2, 2>>(1, 11.f), choice<Tile<2, 2, 2, 2, 2>>(1, 15.f),
      choice<Tile<2, 2, 2, 2, 1>>(2, 25.f), choice<Tile<2, 2, 4, 4, 1>>(1, 33.f)};
  const Choice* best = nullptr;
  float least = 0.f;
  for (const Choice& c : choices) {
    const long long tiles = (long long)((P.R + c.bm - 1) / c.bm) * ((P.N + c.bn - 1) / c.bn);
    if (tiles > 0xFFFFFFFFLL / c.threads) continue;
    const long long at_once = (long long)c.slots * cus;
    const float us = c.us * (float)((tiles + at_once - 1) / at_once);
    if (!best || us < least) {
      best = &c;
      least = us;
    }
  }
  if (!best)
    return fail(QMOE_ERR_UNSUPPORTED, "qgemm_mxfp4_mxfp4: R=%d N=%d: too many tiles", P.R, P.N);
  return best->launch(P, ybf, s);
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
  if (N > 1 << 30 || R > 1 << 30)  // tile positions past the last row stay below 2^31
    return fail(QMOE_ERR_UNSUPPORTED, "qgemm_mxfp4_mxfp4: N=%d R=%d beyond 2^30", N, R);
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
  return launch_product(P, ybf, s);
}
