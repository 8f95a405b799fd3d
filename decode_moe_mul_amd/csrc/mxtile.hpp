// Internal header: products of MXFP4 weights with MXFP4 or MXFP8 activations on the
// block-scaled matrix cores, for more rows than the few-row kernel takes; one
// product, or the gate and up products of a gated pair with the same activations.
//
//   y[r, n] = epilogue( sum_k w[n, k] x[r, k] )
//
// A block computes BM = 32 WR TM activation rows x BN = 32 WC TN weight rows
// with WR x WC waves of TM x TN 32x32x64 ops.  A step is 256 values of K, 128
// code bytes of a weight row and 128 (MXFP4) or 256 (MXFP8) of an activation row:
// four groups of ops.
//
// With the largest tile a SIMD holds one wave (its sums fill half the registers),
// so whatever that wave waits for, the matrix core waits for too; the smaller ones
// have two to four.  Everything else is therefore issued between matrix ops, in an
// order that the compiler keeps:
//  * codes go from memory to LDS without passing registers (16 bytes a lane,
//    1 KB of LDS, whole cache lines: half lines doubled the requests to L2,
//    which then set the pace), into one of two buffers, a step ahead;
//  * the operands of a group are read from LDS during the group before it; the
//    step's barrier stands before its last group, when every wave holds the
//    rest of the step's operands, and frees the step's buffer;
//  * scales pass through registers (their rows have any alignment): 16 bytes a
//    row serve two steps, in one of two LDS buffers; a byte permute gives each
//    lane its four blocks of a step in one word, whose bytes the ops select.
// The operands' layouts (measured against a CPU model): lane 32 h + i of group s
// takes row i; of MXFP4 block 2 s + h (values 32 h .. + 31 of the group's 64), of
// MXFP8 values 16 h .. + 15 and 32 + 16 h .. + 15; its scale is that of block
// 2 s + h in both.  The 16-byte chunk c of tile row q lies at chunk
// c ^ ((q >> 1) & 7) where a row has 128 bytes, at c ^ (q & 15) where it has 256,
// chosen by which chunk of memory a lane fetches, so that the rows one operand
// read touches spread over the banks.  Rows past the ends repeat the last one and
// are never stored; blocks past K's end repeat the row's last one with scale
// bytes of 0, and 2^-127 from either side leaves nothing of their products.
//
// KS teams of WR x WC waves split K where there are too few tiles to fill the
// part: each takes a run of whole turns (two steps) with buffers of its own,
// and the first team adds the others' sums to its own in team order.
//
// A gated pair (GLU): the tile's BN weight rows are 32 of the gate, the same 32 of
// up, and so on, so that a wave's blocks 2 p and 2 p + 1 hold a gate and its up in
// the same registers of the same lane; N counts the pair's columns.
#pragma once
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "copy.hpp"
#include "epilogue.hpp"

#pragma clang fp contract(off)

namespace qmoe {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float v4f_t __attribute__((ext_vector_type(4)));
typedef float v16f_t __attribute__((ext_vector_type(16)));

struct MxProduct {
  const uint8_t* wq;   // codes [N][K/2]; of the gate where there are two products
  const uint8_t* ws;   // E8M0 [N][K/32]
  const uint8_t* wq2;  // up's
  const uint8_t* ws2;
  const uint8_t* xq;   // codes [R][K/2] or [R][K]
  const uint8_t* xs;   // E8M0 [R][K/32]
  int N, K, R;
  Epilogue e;
};

template <int WR_, int WC_, int TM_, int TN_, int KS_, bool XF8_>
struct Tile {
  static constexpr int WR = WR_, WC = WC_, TM = TM_, TN = TN_, KS = KS_;
  static constexpr bool XF8 = XF8_;
  static constexpr int BM = 32 * WR * TM, BN = 32 * WC * TN, ROWS = BM + BN, NW = WR * WC;
  static constexpr int TEAM = 64 * NW, THREADS = TEAM * KS;
  static constexpr int AB = XF8 ? 256 : 128;                    // an activation row's bytes a step
  static constexpr int CODES = BM * AB + BN * 128, SCALES = ROWS * 16;  // bytes of one buffer
  static constexpr int TEAM_LDS = 2 * (CODES + SCALES);
  static constexpr int JA = BM * AB / 1024 / NW, J = CODES / 1024 / NW;  // copies per wave and step
  static constexpr int J1 = J / 2;                              // of them in the first part
  static constexpr int SR = (ROWS + TEAM - 1) / TEAM;           // scale rows per thread
  static_assert(NW % 2 == 0 && BM * AB % (1024 * NW) == 0 && BN % (8 * NW) == 0, "");
  // leaving: 32 rows of a wave's columns, then the other teams' sums
  static constexpr int COLS = 32 * TN, PITCH = leave_pitch(COLS), OUT = NW * 32 * PITCH * 4;
  static constexpr int SUMS = TM * TN * 16 * TEAM * 4;
  static constexpr size_t LDS = std::max(KS * TEAM_LDS, OUT + (KS - 1) * SUMS);
  static_assert(LDS <= 160 << 10, "");
};

// an activation operand: 16 bytes of MXFP4, 32 of MXFP8
template <bool XF8>
struct ActOp {
  uint4 lo;
};
template <>
struct ActOp<true> {
  uint4 lo, hi;
};
QMOE_D void set_op(ActOp<false>& o, uint4 lo, uint4) { o.lo = lo; }
QMOE_D void set_op(ActOp<true>& o, uint4 lo, uint4 hi) { o.lo = lo, o.hi = hi; }

// The matrix op aligns the products of eight consecutive values of MXFP8 to the
// largest of them and drops what lies more than 13 binary places below (measured): a
// sum of 64 N(0, 1) products is off by 4.5e-6, one beside a channel a thousand times
// louder by 2^-9 and more, and one whose largest products cancel loses all of it.  Cut
// at the middle exponent, the codes of either half span eight binary places, and every
// product stays: two exact ops.  `small` are the codes with an exponent field below 8,
// `big` the others, zeros in their places.
QMOE_D void split_e4m3(uint4 v, uint4& big, uint4& small) {
  const auto cut = [](uint32_t w, uint32_t& b, uint32_t& s) {
    // 0xFF in the bytes of large codes (bit 6 set): the permute repeats the top bits of
    // the odd bytes of its two sources, w moved up by a bit and by a byte and a bit
    b = w & __builtin_amdgcn_perm(w << 9, w << 1, 0x090B080Au);
    s = w ^ b;
  };
  cut(v.x, big.x, small.x);
  cut(v.y, big.y, small.y);
  cut(v.z, big.z, small.z);
  cut(v.w, big.w, small.w);
}
template <int SEL, bool XF8>
QMOE_D v16f_t mx_mma32(const ActOp<XF8>& x, uint32_t sa, uint4 b, uint32_t sb, v16f_t c) {
  const v8i_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  const uint4 a = x.lo;
  if constexpr (XF8) {
    const v8i_t av = {(int)a.x,    (int)a.y,    (int)a.z,    (int)a.w,
                      (int)x.hi.x, (int)x.hi.y, (int)x.hi.z, (int)x.hi.w};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 0, 4, SEL, (int)sa, SEL,
                                                           (int)sb);
  } else {
    const v8i_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, SEL, (int)sa, SEL,
                                                           (int)sb);
  }
}

template <class T, bool GLU>
__global__ __launch_bounds__(T::THREADS) void mx_tile_kernel(MxProduct P, int tiles_m,
                                                             int tiles_n) {
  constexpr int TM = T::TM, TN = T::TN, M = TM * TN, NR = TM + TN;
  constexpr bool XF8 = T::XF8;
  static_assert(!GLU || TN % 2 == 0, "");
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
  const int r0 = (tile % tiles_m) * T::BM, n0 = (tile / tiles_m) * (GLU ? T::BN / 2 : T::BN);
  // this team's steps [first, first + steps) of K's `all`; every team goes
  // through `loops` of them, idle past its own
  const int nb = P.K >> 5, all = (nb + 7) >> 3;
  const int loops = 2 * ((all + 2 * T::KS - 1) / (2 * T::KS));
  const int first = team * loops;
  const int steps = min(max(all - first, 0), loops), turns = (steps + 1) >> 1;
  const uint32_t rowb = (uint32_t)P.K >> 1, arowb = XF8 ? (uint32_t)P.K : rowb;
  const uint8_t* const abase = P.xq + (size_t)r0 * arowb;
  const uint8_t* const bbase = P.wq + (size_t)n0 * rowb;
  const uint8_t* const bbase2 = GLU ? P.wq2 + (size_t)n0 * rowb : nullptr;
  const int arows = P.R - r0 - 1, brows = P.N - n0 - 1;  // last valid row of the tile
  // weight row of the tile's row q: of a pair, 32 of the gate and 32 of up in turn
  const auto weight = [](int q) { return GLU ? (q >> 6 << 5) + (q & 31) : q; };

  // Copy j of the wave fills 1 KB of the tile: 8 rows of 128 bytes or 4 of 256.
  const int rem = nb - 8 * (all - 1);  // blocks of K's last step, 1..8
  uint32_t off[T::J];
  // by how much a lane's chunk lies past the last block of K's last step (of MXFP8,
  // where a block is two chunks, in whole blocks); the same for every second copy
  uint32_t over_a[2], over_b = 0;
#pragma unroll
  for (int j = 0; j < T::J; ++j) {
    if (XF8 && j < T::JA) {
      const int q = 4 * (wave + T::NW * j) + (lane >> 4);
      const int chunk = (lane & 15) ^ (q & 15);
      off[j] = (uint32_t)min(q, arows) * arowb + 16u * (uint32_t)chunk;
      if (j < 2) over_a[j] = 32u * (uint32_t)max((chunk >> 1) - (rem - 1), 0);
    } else {
      const int q = 8 * (wave + T::NW * (j < T::JA ? j : j - T::JA)) + (lane >> 3);
      const int chunk = (lane & 7) ^ ((q >> 1) & 7);  // NW is even: the same for every j
      const int row = j < T::JA ? min(q, arows) : min(weight(q), brows);
      off[j] = (uint32_t)row * rowb + 16u * (uint32_t)chunk;
      over_b = 16u * (uint32_t)max(chunk - (rem - 1), 0);
    }
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)mem;
  const auto copy = [&](int st, int j) {
    const int k = min(first + st, all - 1);  // past the team's steps: unused
    const bool a = j < T::JA;
    const uint8_t* base = a ? abase : bbase;
    if (GLU && !a && ((wave + T::NW * (j - T::JA)) >> 2 & 1)) base = bbase2;
    const uint32_t over = XF8 && a ? over_a[T::JA > 1 ? j & 1 : 0] : over_b;
    copy_to_lds(lds0 + (st & 1) * T::CODES + (wave + T::NW * j) * 1024,
                uniform(base + (size_t)k * (a ? T::AB : 128)), off[j] - (k + 1 == all ? over : 0));
  };
  // scales of the team's turns (16 blocks), tile row q at 16 q; 0 past K's end
  uint8_t* const sc = mem + 2 * T::CODES;
  uint4 sreg[T::SR];
  const auto load_scales = [&](int turn) {
    const int u = (first >> 1) + turn;
#pragma unroll
    for (int j = 0; j < T::SR; ++j) {
      const int q = tid + j * T::TEAM;
      const uint8_t* p;
      if (q < T::BM) {
        p = P.xs + (size_t)(r0 + min(q, arows)) * nb + 16 * u;
      } else {
        const uint8_t* plane = GLU && ((q - T::BM) >> 5 & 1) ? P.ws2 : P.ws;
        p = plane + (size_t)(n0 + min(weight(q - T::BM), brows)) * nb + 16 * u;
      }
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
    ActOp<XF8> a[TM];
    uint4 b[TN];
  };
  struct Scl {
    uint32_t v[NR];
  };
  // operands in the order the ops use them: a0, b0 .. , a1 ..
  const auto nth = [](auto rr) {
    constexpr int r = decltype(rr)::value;
    return Int<(r == 0 ? 0 : r <= TN ? TM + r - 1 : r - TN)>{};
  };
  const auto row_of = [&](int r) { return r < TM ? qa + 32 * r : qb + 32 * (r - TM); };
  const auto read_op = [&](int st, int s, auto rr, Ops& o) {
    constexpr int r = decltype(rr)::value;
    const uint8_t* const buf = mem + (st & 1) * T::CODES;
    if constexpr (XF8 && r < TM) {
      const uint8_t* const p = buf + row_of(r) * 256;
      set_op(o.a[r], *(const uint4*)(p + 16 * ((4 * s + h) ^ (i & 15))),
             *(const uint4*)(p + 16 * ((4 * s + 2 + h) ^ (i & 15))));
    } else {
      const uint8_t* const p = buf + (XF8 ? T::BM * 128 : 0) + row_of(r) * 128;
      const uint4 v = *(const uint4*)(p + 16 * ((2 * s + h) ^ ((i >> 1) & 7)));
      if constexpr (r < TM) set_op(o.a[r], v, v);
      else o.b[r - TM] = v;
    }
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
    ActOp<XF8> small, big;  // MXFP8: of the row that the last op took
    static_for<M>([&](auto slot) {
      constexpr int m = decltype(slot)::value / TN, n = decltype(slot)::value % TN;
      constexpr int SEL = decltype(sel)::value;
      if constexpr (XF8) {
        if constexpr (n == 0) {
          split_e4m3(o.a[m].lo, big.lo, small.lo);
          split_e4m3(o.a[m].hi, big.hi, small.hi);
        }
        acc[m][n] = mx_mma32<SEL, XF8>(small, c.v[m], o.b[n], c.v[TM + n], acc[m][n]);
        acc[m][n] = mx_mma32<SEL, XF8>(big, c.v[m], o.b[n], c.v[TM + n], acc[m][n]);
      } else {
        acc[m][n] = mx_mma32<SEL, XF8>(o.a[m], c.v[m], o.b[n], c.v[TM + n], acc[m][n]);
      }
      side(slot);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // of `count` things spread over a group's M slots, those of slot n
  const auto spread = [](auto n, auto count, auto&& f) {
    constexpr int c = decltype(count)::value, lo = n * c / M, hi = (n + 1) * c / M;
    static_for<hi - lo>([&](auto k) { f(Int<lo + k>{}); });
  };
  // of the NR operands, early in a group (the next group needs them), those of slot n
  const auto early = [](auto n, auto&& f) {
    constexpr int per_slot = (2 * NR + M - 1) / M;
    constexpr int lo = n * per_slot, hi = lo + per_slot < NR ? lo + per_slot : NR;
    static_for<(hi > lo ? hi - lo : 0)>([&](auto k) { f(Int<lo + k>{}); });
  };
  using I0 = Int<0>;
  using I1 = Int<1>;
  using I2 = Int<2>;
  using I3 = Int<3>;

  Ops f0, f1;
  Scl cur;
  // Step st, of parity k, with LEFT more to follow (2: two or more).  Known to
  // the compiler: a branch among the ops would end what it may reorder and
  // count across.
  const auto step = [&](auto kk, auto left, int st) {
    constexpr int k = decltype(kk)::value, LEFT = decltype(left)::value;
    const bool live = (T::KS == 1 && LEFT > 0) || st < steps;
    if (live) {
      group(I0{}, f0, cur, [&](auto n) {
        early(n, [&](auto r) { read_op(k, 1, nth(r), f1); });
        if constexpr (LEFT >= 1)
          spread(n, Int<T::J - T::J1>{}, [&](auto j) { copy(st + 1, T::J1 + j); });
      });
      group(I1{}, f1, cur, [&](auto n) {
        early(n, [&](auto r) { read_op(k, 2, nth(r), f0); });
        if constexpr (LEFT >= 1) spread(n, Int<NR>{}, [&](auto r) { read_raw(st + 1, r); });
      });
      group(I2{}, f0, cur, [&](auto n) {
        early(n, [&](auto r) { read_op(k, 3, nth(r), f1); });
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
      group(I3{}, f1, cur, [&](auto n) {
        if constexpr (LEFT >= 1) early(n, [&](auto r) { read_op(k + 1, 0, nth(r), f0); });
        if constexpr (LEFT >= 2) spread(n, Int<T::J1>{}, [&](auto j) { copy(st + 2, j); });
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
  static_for<NR>([&](auto r) {
    read_op(0, 0, r, f0);
    read_raw(0, r);
  });
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

  // Register 4 a + b of a 32 x 32 block is row 8 a + 4 h + b, column i.
  if constexpr (T::KS == 1) __syncthreads();  // every wave has read its last operands
  float* const out = (float*)smem + wave * 32 * T::PITCH;
  const Leave<T::COLS, GLU, XF8 ? kOutMx8 : kOutMx4> leave(
      P.e, out, n0 + (GLU ? wn / 2 : wn), P.R, P.N, lane);
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
static int launch_tile(const char* name, const MxProduct& P, hipStream_t s) {
  constexpr int cols = GLU ? T::BN / 2 : T::BN;
  const int tm = (P.R + T::BM - 1) / T::BM, tn = (P.N + cols - 1) / cols;
  const dim3 grid((unsigned)(tm * tn));
  // a kernel that takes more than 64 KB of LDS declares it, once per device
  static std::atomic<uint64_t> declared;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) dev = 64;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!bit || !(declared.load(std::memory_order_relaxed) & bit)) {
    (void)hipFuncSetAttribute((const void*)mx_tile_kernel<T, GLU>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, (int)T::LDS);
    declared.fetch_or(bit, std::memory_order_relaxed);
  }
  return QMOE_LAUNCH(name, (mx_tile_kernel<T, GLU>), grid, T::THREADS, T::LDS, s, P, tm, tn);
}

struct Choice {
  int bm, cols, threads, slots;
  float us, alone;
  int (*launch)(const char*, const MxProduct&, hipStream_t);
};
template <class T, bool GLU>
static constexpr Choice choice(int slots, float us, float alone = 0.f) {
  return {T::BM, GLU ? T::BN / 2 : T::BN, T::THREADS, slots, us, alone > 0.f ? alone : us,
          launch_tile<T, GLU>};
}

// A round of tiles takes about as long as one tile, so with K given the choice
// goes by rounds times the time of one, with `slots` tiles to a compute unit (`alone`:
// where a last round leaves each unit one of them).  A launch has fewer than 2^32
// threads: a tile that would need more is passed over.
template <int C>
static int launch_choice(const Choice (&choices)[C], const char* who, const char* name,
                         const MxProduct& P, hipStream_t s) {
  const int cus = std::max(1, cu_count());
  const Choice* best = nullptr;
  float least = 0.f;
  for (const Choice& c : choices) {
    const long long tiles =
        (long long)((P.R + c.bm - 1) / c.bm) * ((P.N + c.cols - 1) / c.cols);
    if (tiles > 0xFFFFFFFFLL / c.threads) continue;
    const long long at_once = (long long)c.slots * cus, last = tiles % at_once;
    const float us = c.us * (float)(tiles / at_once) +
                     (last == 0 ? 0.f : last <= cus ? c.alone : c.us);
    if (!best || us < least) {
      best = &c;
      least = us;
    }
  }
  if (!best)
    return fail(QMOE_ERR_UNSUPPORTED, "%s: R=%d N=%d: too many tiles", who, P.R, P.N);
  return best->launch(name, P, s);
}

}  // namespace qmoe
