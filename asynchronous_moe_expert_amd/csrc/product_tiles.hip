// The experts' products on large tiles: 256 x 256 of C, bf16 (v_mfma_f32_16x16x32_bf16) or 8 bits
// (v_mfma_f32_16x16x128_f8f6f4 with fp32 scales; for fp32 outputs of 8-bit operands bf16 again: dot128), operands
// copied straight into LDS.
//
// Two groups of four waves take half of a tile's rows each and change places: while one multiplies, the other reads
// its next fragments; group 0 makes all copies, group 1 finds tiles and rows, so that only one waits for memory.
// 256 x 256 is the most that two stages in LDS and the accumulators in registers allow; smaller tiles read more from
// L2 for each product.  Reached, 32 experts of 512 rows, 4096 x 4096: forward 473 to 493 us (1.14 PFLOP/s), rows' gradient 484
// to 500, 8 bits 321 to 370 by the codes' values (1.6); 8192 rows of one expert, 4096 x 8192: 390 to 399 (1.4, what a
// library product reaches) and 8 bits 258 to 262 (2.1).  Counted there: the matrix cores are busy for 56% of the cycles
// (8 bits 38%, the weights' gradient 32%), the waves wait for 37% of theirs (19%, 42%), LDS reads take 21% (17%, 12%)
// with no conflicts, 68% (77%, 61%) of what is asked of L2 is there.  In 8 bits the compiler spills 11 vector registers,
// with fp32 outputs 72.  With few rows an expert the weights' bytes bound it, with uneven ones the last tiles.
#include <type_traits>

#include "product_copy.hpp"

namespace moe {

constexpr int kTile = 256, kStageQ = kTile * 128;
constexpr int kPool = 3 * (kStageQ + 128 * 128);  // bytes of LDS for the stages: three of MT = 4, two of MT = 8

// How an operand lies in LDS and how a step of it is copied there.  A stage holds 256 p and 256 q by 64 k (128
// codes); a wave's copy instruction fills 1 KiB, eight runs of 128 bytes, each from one row of memory.
//   along k:  row r is 128 bytes, its 16-byte piece c at place c ^ key(r): key = bits 1..3 of r for P and bits 1,
//             3, 4 for Q.  Lane l reads piece l / 16 (+ 4) of P's row l % 16, of Q's row 8 (l % 16 / 4) + l % 4 (+ 4
//             for the next 16 of the matrix instruction's rows, so that a lane ends up with eight neighbouring
//             columns of C): sixteen rows' pieces lie in the sixteen places of the 256 bytes that LDS gives a cycle.
//   across k: blocks of 64 columns; in a block row k is 128 bytes, its 32-byte part c at place c ^ f(k), f(k) =
//             bits 1 and 3 of k.  ds_read_b64_tr_b16 gives lane l of a group of 16 column l of four rows, 8 g to 8 g
//             + 3 for group g; the eight rows that two groups read at a time lie in different places again.
// (read rates, bytes a cycle and CU: along 246 with these keys and 64 without any, across 264 and 43)
template <int MODE, int DT, int MT>
struct Tile {
  static constexpr int es = esize<DT>();
  static constexpr bool kPAlong = MODE != kWeightsGrad, kQAlong = MODE == kForward;
  static constexpr bool kScaled = esize<DT>() == 1;
  static constexpr int kHalf = MT / 2;
  static constexpr int kStages = MT <= 4 ? 3 : 2;  // steps in LDS
  static constexpr int kStageP = 32 * MT * 128;    // bytes of P in one, half for each group; Q has kStageQ
  static constexpr bool kTurn = kQAlong && MT <= 4;  // column tiles begin at different k
  // copies that a wave of group 0 makes in a step: of each group's rows of P, of Q, and of the rows' scales
  static constexpr int kP = MT / 2, kQ = 8, kScales = kScaled ? 1 : 0;
  static constexpr int kFirst = kQ + kP + kScales, kSecond = kP;
};
// What a workgroup has in LDS: the stages (all of Q's, then P's), four steps of the rows' scales, the weights' scales
// of the tile's two blocks of columns, and where the rows of this tile and the next come from.
struct Lds {
  char* pool;
  float *scale, *w_scale;
  int* slots;    // [2][256]
  Place* place;  // [2]
};

__device__ __forceinline__ Place load_place(const Place* from) {
  Place at;
  int* to = reinterpret_cast<int*>(&at);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(Place) / 4); ++i)
    to[i] = __builtin_amdgcn_readfirstlane(reinterpret_cast<const int*>(from)[i]);
  return at;
}

// The base and pitch of an operand's rows.
template <int MODE, int DT>
__device__ __forceinline__ const char* p_base(const ProductJob& j, const Place& at) {
  return MODE == kWeightsGrad ? (const char*)j.dout + at.k0 * j.dout_pitch * esize<DT>() : (const char*)j.x;
}
template <int MODE, int DT>
__device__ __forceinline__ int64_t q_pitch(const ProductJob& j) {
  return (MODE == kWeightsGrad ? j.x_pitch : j.w_pitch) * esize<DT>();
}
template <int MODE, int DT>
__device__ __forceinline__ const char* q_base(const ProductJob& j, const Place& at) {
  if constexpr (MODE == kWeightsGrad) return (const char*)j.x + at.k0 * j.x_pitch * esize<DT>();
  else return (const char*)j.w + (at.e * j.w_stride + (MODE == kForward ? at.q0 * j.w_pitch : 0)) * esize<DT>();
}

template <int MODE, int DT>
__device__ __forceinline__ int contraction_steps(const ProductJob& j, const Place& at) {
  return MODE == kWeightsGrad ? (at.kend - at.k0 + kStep - 1) / kStep : (j.D * esize<DT>() + 127) / 128;
}

// The copies of a tile's operands, all made by the four waves wq of group 0.
template <int MODE, int DT, int MT>
struct Copies {
  using T = Tile<MODE, DT, MT>;
  static constexpr int es = T::es;
  uint32_t poff[2][T::kPAlong ? T::kP : 1];  // along k: in units of 16 bytes from x
  uint32_t nosrc = 0;                        // copies of P whose row has no source, bit 31: the scale
  bool sourced = true;
  const float* sptr = nullptr;
  Across<T::kPAlong ? 1 : T::kP / 2> pa[2];
  uint32_t qoff = 0;
  Across<4> qa;
  int pieces;  // of a row along k
  int steps, turn;

  // the step of the contraction that is taken as the s-th
  __device__ __forceinline__ int step_of(int s) const {
    if constexpr (!T::kTurn) return s;
    return s + turn < steps ? s + turn : s + turn - steps;
  }
  static __device__ __forceinline__ int ppiece(int wq, int lane) { return (lane & 7) ^ (4 * (wq & 1) + (lane >> 4)); }
  static __device__ __forceinline__ int qpiece(int wq, int lane) { return (lane & 7) ^ (((lane >> 4) & 1) | 2 * wq); }

  __device__ __forceinline__ void set(const ProductJob& j, const Place& at, const int* slots, int wq, int lane) {
    pieces = j.D * es / 16;
    steps = contraction_steps<MODE, DT>(j, at);
    turn = turn_of(at, steps);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (T::kPAlong) {
#pragma unroll
        for (int c = 0; c < T::kP; ++c) {
          const int slot = slots[h * 16 * MT + 8 * (4 * c + wq) + (lane >> 3)];
          if (slot < 0) nosrc |= 1u << (h * T::kP + c);
          poff[h][c] = (uint32_t)((slot < 0 ? 0 : slot) * (j.x_pitch * es / 16) + ppiece(wq, lane));
        }
      } else {
        pa[h].set(wq, lane, at.p0 + h * 16 * MT, j.N, j.dout_pitch, es);
      }
    }
    if constexpr (T::kScaled) {
      const int slot = slots[(wq >> 1) * 16 * MT + min((wq & 1) * 64 + lane, 16 * MT - 1)];
      if (slot < 0) nosrc |= 1u << 31;
      else sptr = j.x_scale + (int64_t)slot * ((j.D + 127) / 128);
    }
    sourced = __ballot(nosrc != 0) == 0;
    if constexpr (T::kQAlong) qoff = (uint32_t)((lane >> 3) * (int)j.w_pitch * es + qpiece(wq, lane) * 16);
    else qa.set(wq, lane, at.q0, MODE == kWeightsGrad ? j.D : j.N, MODE == kWeightsGrad ? j.x_pitch : j.w_pitch, es);
  }
  // where the s-th step lies in LDS
  static __device__ __forceinline__ int p_at(int s) { return T::kStages * kStageQ + s % T::kStages * T::kStageP; }
  static __device__ __forceinline__ int q_at(int s) { return s % T::kStages * kStageQ; }
  // Weights whose rows are a power of two apart put the same step of all of them on a few memory channels: the
  // column tiles of an expert begin at different steps, which costs nothing where its rows fit the L2
  static __device__ __forceinline__ int turn_of(const Place& at, int steps) {
    return T::kTurn ? ((at.q0 / kTile) * 11 + at.e * 3) % steps : 0;
  }
  __device__ __forceinline__ void p_half(const ProductJob& j, const Place& at, const Lds& lds, int h, int s, int wq,
                                         int lane) const {
    const int step = step_of(s);
    const uint32_t dst = lds_at(lds.pool) + p_at(s) + h * (T::kStageP / 2) + wq * 1024;
    if constexpr (T::kPAlong) {
      const char* from = uniform_ptr(p_base<MODE, DT>(j, at) + (int64_t)step * 128);
      if (sourced && (step + 1) * 8 <= pieces) {
        each<T::kP>([&](auto c) { copy16<c() * 4096>(from + (uint64_t)poff[h][c()] * 16, dst); });
      } else {
        each<T::kP>([&](auto c) {
          const bool there = step * 8 + ppiece(wq, lane) < pieces && !(nosrc >> (h * T::kP + c()) & 1);
          copy16<c() * 4096>(there ? from + (uint64_t)poff[h][c()] * 16 : (const char*)&g_zeros, dst);
        });
      }
    } else {
      pa[h].copy(p_base<MODE, DT>(j, at), j.dout_pitch * es, dst, step, at.kend - at.k0, wq, lane);
    }
  }
  // Q, group 0's rows of P, and all rows' scales
  __device__ __forceinline__ void first(const ProductJob& j, const Place& at, const Lds& lds, int s, int wq, int lane) const {
    const int Qn = MODE == kWeightsGrad ? j.D : j.N, step = step_of(s);
    const uint32_t dst = lds_at(lds.pool) + q_at(s) + wq * 1024;
    const char* q = q_base<MODE, DT>(j, at);
    if constexpr (T::kQAlong) {  // N is a multiple of 8, so rows are past it by whole copies: read at the first ones
      const char* from = uniform_ptr(q + (int64_t)step * 128 + 8 * wq * j.w_pitch * es);
      if (at.q0 + kTile <= Qn && (step + 1) * 8 <= pieces) {
        const int64_t rows = 32 * j.w_pitch * es;
        each<T::kQ>([&](auto c) {
          copy16<c() * 4096>(from, qoff, dst);
          from += rows;
        });
      } else {
        const bool there = step * 8 + qpiece(wq, lane) < pieces;
        each<T::kQ>([&](auto c) {
          const int r = 32 * c();
          const char* row = uniform_ptr(at.q0 + 8 * wq + r < Qn ? from + r * j.w_pitch * es : q + (int64_t)step * 128);
          copy16<c() * 4096>(there ? row + qoff : (const char*)&g_zeros, dst);
        });
      }
    } else {
      qa.copy(q, q_pitch<MODE, DT>(j), dst, step, at.kend - at.k0, wq, lane);
    }
    p_half(j, at, lds, 0, s, wq, lane);
    if constexpr (T::kScaled) {
      const char* src = !(nosrc >> 31) ? (const char*)(sptr + step) : (const char*)&g_zeros;
      copy4(src, lds_at(lds.scale) + (s & 3) * 1024 + wq * 256);
    }
  }
  __device__ __forceinline__ void second(const ProductJob& j, const Place& at, const Lds& lds, int s, int wq, int lane) const {
    p_half(j, at, lds, 1, s, wq, lane);
  }
};

// Copies the first steps of a tile, as many as LDS holds.
template <int MODE, int DT, int MT>
__device__ __forceinline__ void begin(const ProductJob& j, const Place& at, const Lds& lds, const int* slots, int wq, int lane) {
  Copies<MODE, DT, MT> c;
  c.set(j, at, slots, wq, lane);
#pragma unroll
  for (int s = 0; s < Tile<MODE, DT, MT>::kStages; ++s) {
    if (s < c.steps) {
      c.first(j, at, lds, s, wq, lane);
      c.second(j, at, lds, s, wq, lane);
    }
  }
}
template <int MODE, int DT>
__device__ __forceinline__ void begin_any(const ProductJob& j, const Place& at, const Lds& lds, const int* slots, int wq,
                                          int lane) {
  switch (at.mt) {
    case 2:
      if constexpr (MODE != kWeightsGrad) begin<MODE, DT, 2>(j, at, lds, slots, wq, lane);
      break;
    case 4: begin<MODE, DT, 4>(j, at, lds, slots, wq, lane); break;
    case 6:
      if constexpr (MODE != kWeightsGrad) begin<MODE, DT, 6>(j, at, lds, slots, wq, lane);
      break;
    default: begin<MODE, DT, 8>(j, at, lds, slots, wq, lane);
  }
}

// Where the next tile's rows come from: group 1's part, which waits for nothing else in memory.
template <int MODE>
__device__ __forceinline__ void find_rows(const ProductJob& j, const Place& at, int* slots, int i) {
  if constexpr (MODE != kWeightsGrad) {
    const int row = min(at.p0 + i, at.pend - 1);
    int slot = row;
    if (j.row_slot) {
      slot = j.row_slot[row];
      if (slot < 0 || slot >= j.x_rows) {
        atomicOr(j.err, MOE_ERR_SLOT_RANGE);
        slot = -1;
      }
    }
    slots[i] = slot;
  }
}

template <int MODE, int DT, int MT, int G, typename W>
__device__ __forceinline__ Place tile(const ProductJob& j, const Place& at, W& walk, const Lds& lds, int par, int wq, int lane) {
  using T = Tile<MODE, DT, MT>;
  constexpr int es = T::es, kHalf = T::kHalf;
  const int g = lane >> 4, l16 = lane & 15;
  const int steps = contraction_steps<MODE, DT>(j, at);
  const int Qn = MODE == kWeightsGrad ? j.D : j.N;

  // ---- where this lane's fragments lie, in bytes
  int pr, qr, tr;
  if constexpr (T::kPAlong) pr = l16 * 128 + ((g ^ ((l16 >> 1) & 7)) << 4);
  if constexpr (T::kQAlong)
    qr = wq * 8192 + (8 * (l16 >> 2) + (l16 & 3)) * 128 + ((g ^ (((l16 >> 1) & 1) | ((l16 >> 1) & 6))) << 4);
  if constexpr (!T::kPAlong || !T::kQAlong)
    tr = (8 * g + (l16 >> 2)) * 128 + ((((l16 >> 3) & 1) | (g & 1) << 1) << 5) + (l16 & 3) * 8;
  // the second slice's piece is 4 further, the next 16 columns' part c further: both by exclusive or, which the
  // compiler is kept from holding in registers for every stage
  auto flip = [](int a, int bits) {
    int r;
    asm volatile("v_xor_b32 %0, %1, %2" : "=v"(r) : "n"(bits), "v"(a));
    return r;
  };
  auto along = [&](const char* stage, int at_) { return *reinterpret_cast<const u32x4*>(stage + at_); };
  auto across = [&](const char* stage, int at_) -> u32x4 {
    const char* b = stage + at_;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(b));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(b + 512));
    u32x4 r;
    __builtin_memcpy(&r, &lo, 8);
    __builtin_memcpy((char*)&r + 8, &hi, 8);
    return r;
  };

  f32x4 acc[MT][4];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 pf[kHalf][2], qf[4][2];
  float sc[kHalf], sw = 0.f;
  auto read_p = [&](const char* ps, const float* ss, int a0, int a, int at0, int at1) {  // tile a0 + a of the group's rows
    if constexpr (T::kPAlong) {
      pf[a][0] = along(ps, at0 + (a0 + a) * 2048);
      pf[a][1] = along(ps, at1 + (a0 + a) * 2048);
    }
    if constexpr (T::kScaled) sc[a] = ss[G * 128 + (a0 + a) * 16 + l16];
  };
  auto read = [&](const char* ps, const char* qs, const float* ss, int step) {
    if constexpr (T::kScaled) sw = lds.w_scale[(wq >> 1) * kMaxBlocks + step];
    if constexpr (T::kQAlong) {
      const int q1 = flip(qr, 64);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        qf[b][0] = along(qs, qr + (b & 1) * 512 + (b >> 1) * 4096);
        qf[b][1] = along(qs, q1 + (b & 1) * 512 + (b >> 1) * 4096);
      }
    } else {
      const int tq = wq * 8192 + tr;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int t = b ? flip(tq, 32 * b) : tq;
        qf[b][0] = across(qs, t);
        qf[b][1] = across(qs, t + 4096);
      }
    }
    if constexpr (T::kPAlong) {
      const int p1 = flip(pr, 64);
#pragma unroll
      for (int a = 0; a < kHalf; ++a) read_p(ps, ss, 0, a, pr, p1);
    } else {
#pragma unroll
      for (int a = 0; a < kHalf; ++a) {
        const int t = (a & 3) ? flip(tr, 32 * (a & 3)) : tr;
        pf[a][0] = across(ps, t);
        pf[a][1] = across(ps, t + 4096);
      }
    }
  };
  auto pipe = [&](int a0, int a) {  // 8 bits: the products of tile a0 + a, whose fragments are pf[a]
    // each instruction's result is scaled and added two instructions later, in the shadow of the next ones
    i32x8 p;
    __builtin_memcpy(&p, &pf[a][0], 32);
    const float s = sc[a] * sw;
    f32x4 v[4];
#pragma unroll
    for (int b = 0; b < 6; ++b) {
      if (b < 4) {
        i32x8 q;
        __builtin_memcpy(&q, &qf[b][0], 32);
        v[b] = dot128<DT>(q, p);
      }
      if (b >= 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[a0 + a][b - 2][i] = fmaf(v[b - 2][i], s, acc[a0 + a][b - 2][i]);
        asm volatile("" : "+v"(acc[a0 + a][b - 2]));  // here, not after the step's last instruction
      }
    }
  };
  auto row = [&](int a0, int a) {  // the products of tile a0 + a
    if constexpr (T::kScaled) {
      pipe(a0, a);
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          bf16x8 p, q;
          __builtin_memcpy(&p, &pf[a][s], 16);
          __builtin_memcpy(&q, &qf[b][s], 16);
          acc[a0 + a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q, p, acc[a0 + a][b], 0, 0, 0);
        }
    }
  };
  auto multiply = [&](const char* ps, const float* ss, auto&& meanwhile) {
    __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
    int p1 = 0;
    if constexpr (T::kPAlong) p1 = flip(pr, 64);
#pragma unroll
    for (int a = 0; a < kHalf; ++a) {
      row(0, a);
      if (a == 0) {  // issued while the matrix core works
        __builtin_amdgcn_sched_barrier(0);
        meanwhile();
      }
      if constexpr (T::kPAlong) {
        read_p(ps, ss, kHalf, a, pr, p1);
      } else {
        const int c = (kHalf + a) & 3, t = (c ? flip(tr, 32 * c) : tr) + ((kHalf + a) >> 2) * 8192;
        pf[a][0] = across(ps, t);
        pf[a][1] = across(ps, t + 4096);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int a = 0; a < kHalf; ++a) {
      row(kHalf, a);
      if constexpr (T::kScaled) __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
  };

  // ---- The waves of a SIMD, one of each group, take turns: while one multiplies a step's fragments, which it
  // holds in registers, the other reads its next ones (Q's and half of P's; the other half takes the place of
  // what has been multiplied).  Group 0 reads step i in phase 2 i and multiplies in phase 2 i + 1, group 1 one
  // phase later; a barrier ends each phase.  So of a stage, Q and group 0's rows of P are free after phase 2 i + 1,
  // group 1's after 2 i + 2: group 0 copies step i + 2 there in the phase after, two phases before it is read.
  // The steps that LDS holds have been copied when the tile begins; from then on step s + S - 1 goes where step s - 1
  // was (S = 2, or 3 where the rows are few and the weights come from HBM).
  using C = Copies<MODE, DT, MT>;
  constexpr int S = T::kStages, kBoth = T::kFirst + T::kSecond;
  static_assert((S - 1) * kBoth < 64, "a wave's copies are counted in six bits");
  if constexpr (G == 0) {
    C c;
    c.set(j, at, lds.slots + par * 256, wq, lane);
    wait_lds();
    meet();
#pragma clang loop unroll(disable)
    for (int i = 0; i < steps; i += S) {
#pragma unroll
      for (int h = 0; h < S; ++h) {
        const int s = i + h;
        if (s >= steps) break;
        const char *ps = lds.pool + C::p_at(h), *qs = lds.pool + C::q_at(h);
        const float* ss = lds.scale + (s & 3) * 256;
        const bool more = s > 0 && s + S - 1 < steps;
        read(ps, qs, ss, c.step_of(s));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (more) c.first(j, at, lds, s + S - 1, wq, lane);
        wait_lds();
        if (s >= S) {  // group 1's rows of step s
          if (more) wait_copies<(S - 2) * kBoth + T::kFirst>();
          else wait_copies<0>();
        }
        meet();
        multiply(ps, ss, [&]() {
          if (more) c.second(j, at, lds, s + S - 1, wq, lane);
        });
        if (s + 1 >= S) {  // the rest of step s + 1
          if (more) wait_copies<(S - 2) * kBoth + T::kSecond>();
          else wait_copies<0>();
        }
        meet();
      }
    }
    meet();
  } else {
    if constexpr (T::kScaled) {
      const int nb = (j.N + 127) / 128;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float* from = j.w_scale + ((int64_t)at.e * nb + min((at.q0 >> 7) + b, nb - 1)) * steps;
        for (int k = wq * 64 + lane; k < steps; k += 256) lds.w_scale[b * kMaxBlocks + k] = from[k];
      }
    }
    {
      const Place next = walk.next(j);
      if (next.e >= 0) find_rows<MODE>(j, next, lds.slots + (par ^ 1) * 256, wq * 64 + lane);
      if (wq == 0 && lane == 0) lds.place[par ^ 1] = next;
    }
    const int turn = C::turn_of(at, steps);
    wait_lds();
    meet();
    meet();
#pragma clang loop unroll(disable)
    for (int i = 0; i < steps; i += S) {
#pragma unroll
      for (int h = 0; h < S; ++h) {
        if (i + h >= steps) break;
        const char *ps = lds.pool + C::p_at(h) + T::kStageP / 2, *qs = lds.pool + C::q_at(h);
        const float* ss = lds.scale + ((i + h) & 3) * 256;
        read(ps, qs, ss, i + h + turn < steps ? i + h + turn : i + h + turn - steps);
        wait_lds();
        meet();
        multiply(ps, ss, []() {});
        meet();
      }
    }
  }
  const Place next = load_place(lds.place + (par ^ 1));
  // the next tile's first copies go out before this one's stores, which the waits would count otherwise
  if constexpr (G == 0) {
    if (next.e >= 0) begin_any<MODE, DT>(j, next, lds, lds.slots + (par ^ 1) * 256, wq, lane);
  }

  // ---- outputs, in whole lines of 128 bytes (but for forward fp32 ones and sums added to bf16).  A large fp32
  // gradient goes through the caches without staying: it would push out the rows that the next tiles read.  32 experts
  // of 512 rows, 4096 x 4096, us through the caches / so: calls back to back 820 / 697, with x and dout from HBM (1 GiB
  // written in between) 847 / 877 (bf16: 705 / 702, 699 / 702).  In a layer's step the rows have just been written: its
  // whole backward pass, 8192 tokens, 32 experts, K 2, 4096 x 2048: 2330 / 2275; 2048 tokens, 8, K 4, 2880 x 2880:
  // 1041 / 1012.
  const int64_t out0 = MODE == kWeightsGrad ? at.e * j.out_stride : 0;
  const bool odd = l16 & 1;
#pragma unroll
  for (int a = 0; a < MT; ++a) {
    const int row = at.p0 + G * 16 * MT + a * 16, p = row + l16, pe = row + (l16 & 14);
    const int q0 = at.q0 + 64 * wq;
    if (j.out_f32 && !T::kQAlong) {
#pragma unroll
      for (int b = 0; b < 4; b += 2) {
        f32x4 u = acc[a][b], v = acc[a][b + 1];
        pair_rows(u, v, odd);
        const int q = q0 + 16 * b + (odd ? 16 : 0) + 4 * g;
        if (MODE == kWeightsGrad && j.through) {
          if (pe < at.pend && q < Qn) put4<true>(j, out0 + pe * j.out_pitch + q, u);
          if (pe + 1 < at.pend && q < Qn) put4<true>(j, out0 + (pe + 1) * j.out_pitch + q, v);
        } else {
          if (pe < at.pend && q < Qn) put4(j, out0 + pe * j.out_pitch + q, u);
          if (pe + 1 < at.pend && q < Qn) put4(j, out0 + (pe + 1) * j.out_pitch + q, v);
        }
      }
    } else if (j.out_f32 || j.accumulate) {
      if (p >= at.pend) continue;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int q = q0 + (T::kQAlong ? 32 * (b >> 1) + 8 * g + 4 * (b & 1) : 16 * b + 4 * g);
        if (q < Qn) put4(j, out0 + p * j.out_pitch + q, acc[a][b]);
      }
    } else {
      u32x4 v[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        v[b] = u32x4{pack_bf16x2(acc[a][2 * b][0], acc[a][2 * b][1]), pack_bf16x2(acc[a][2 * b][2], acc[a][2 * b][3]),
                     pack_bf16x2(acc[a][2 * b + 1][0], acc[a][2 * b + 1][1]),
                     pack_bf16x2(acc[a][2 * b + 1][2], acc[a][2 * b + 1][3])};
        if constexpr (!T::kQAlong) neighbours(v[b]);
      }
      pair_rows(v[0], v[1], odd);
      const int q = q0 + (odd ? 32 : 0) + 8 * g;
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (pe + b < at.pend && q < Qn) {
          u32x4* o = reinterpret_cast<u32x4*>((uint16_t*)j.out + out0 + (pe + b) * j.out_pitch + q);
          *o = v[b];
        }
    }
  }
  // the copies have landed when no more is on its way than this wave's stores, which a whole tile has a known number of
  if constexpr (G == 0) {
    if (next.e >= 0) {
      const bool whole = at.pend - at.p0 == 32 * MT && at.q0 + kTile <= Qn && !j.accumulate;
      asm volatile("" ::: "memory");
      if (whole && j.out_f32) wait_copies<4 * MT>();
      else if (whole) wait_copies<2 * MT>();
      else wait_copies<0>();
    }
  }
  return next;
}

constexpr int kXcds = 8;

// Which tiles a workgroup computes, one after the other.  One workgroup runs on a CU; those of an XCD (blockIdx % 8)
// share an L2.
template <int MODE>
struct Walk;

// Forward and rows' gradient: an expert's rows make tiles of 256 and one of the rest, of 64, 128, 192 or 256.  The tiles
// of each height are dealt out to the XCDs evenly, a contiguous part to each (an expert's row tiles of one column
// block after the other, in bands of at most eight, so that what an XCD computes at a time shares weights and rows),
// the highest first.  An XCD's workgroups take its tiles in turns, back and forth, so that one that drew a higher
// tile draws a lower one next; half of them go through theirs from the last to the first, so that low tiles, which
// are bound by reading their weights, run beside high ones, which are bound by the matrix cores.
template <>
struct Walk<kForward> {
  static constexpr int kHeights = 4;  // MT = 8, 6, 4, 2
  struct Table {
    int upto[kHeights][257];  // tiles of the experts before, by height, for one column of tiles
  };
  Table& t;
  int round = 0;

  __device__ __forceinline__ Walk(const ProductJob& j, Table& table) : t(table) {
    const int lane = threadIdx.x & 63, k = threadIdx.x >> 6;  // four experts to a lane, a height to a wave
    if (k < kHeights) {
      int n[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int r0 = 0, r1 = 0;
        if (4 * lane + i < j.E) expert_rows(j, 4 * lane + i, r0, r1);
        const int full = (r1 - r0) / kTile, rest = (r1 - r0) % kTile, height = rest ? kHeights - 1 - (rest - 1) / 64 : -1;
        n[i] = (k == 0 ? full : 0) + (height == k);
        sum += n[i];
      }
      int upto = sum;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
      }
      if (lane == 63) t.upto[k][256] = upto;
      upto -= sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t.upto[k][4 * lane + i] = upto;
        upto += n[i];
      }
    }
    __syncthreads();
  }
  // this XCD's tiles of a height
  __device__ __forceinline__ void share(int ct, int xcd, int k, int& u0, int& n) const {
    const int64_t all = (int64_t)t.upto[k][256] * ct;
    u0 = (int)(all * xcd / kXcds);
    n = (int)(all * (xcd + 1) / kXcds) - u0;
  }
  __device__ __forceinline__ Place next(const ProductJob& j) {
    Place at = {-1, 0, 0, 0, 0, 0, 0};
    const int ct = (j.N + kTile - 1) / kTile, xcd = blockIdx.x % kXcds, idx = blockIdx.x / kXcds;
    const int per = ((int)gridDim.x - xcd + kXcds - 1) / kXcds;
    int all = 0, u = 0, u0, n, k = kHeights;
    for (int i = 0; i < kHeights; ++i) {
      share(ct, xcd, i, u0, n);
      all += n;
    }
    const int rounds = (all + per - 1) / per;
    while (k == kHeights && round < rounds) {
      const int r = 2 * idx < per ? round : rounds - 1 - round;
      u = r * per + (r & 1 ? per - 1 - idx : idx);
      ++round;
      for (k = 0; k < kHeights; ++k) {
        share(ct, xcd, k, u0, n);
        if (u < n) {
          u += u0;
          break;
        }
        u -= n;
      }
    }
    k = __builtin_amdgcn_readfirstlane(k);
    u = __builtin_amdgcn_readfirstlane(u);
    if (k == kHeights) return at;
    const int* upto = t.upto[k];
    int lo = 0, hi = 256;  // the last expert whose tiles begin at or before u and that has any
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (upto[mid] * ct <= u) lo = mid;
      else hi = mid;
    }
    int r0, r1;
    expert_rows(j, lo, r0, r1);
    const int base = upto[lo], tiles = upto[lo + 1] - base;
    const int v = u - base * ct, bands = (tiles + 7) / 8, bh = (tiles + bands - 1) / bands;
    const int band = v / (bh * ct), h = min(bh, tiles - band * bh), w = v - band * bh * ct;
    const int first = k == 0 ? 0 : (r1 - r0) / kTile;  // the rest's tile is the last one
    at.e = __builtin_amdgcn_readfirstlane(lo);
    at.p0 = __builtin_amdgcn_readfirstlane(r0 + (first + band * bh + w % h) * kTile);
    at.q0 = __builtin_amdgcn_readfirstlane(w / h * kTile);
    at.pend = __builtin_amdgcn_readfirstlane(min(r1, at.p0 + kTile));
    at.k0 = 0;
    at.kend = j.D;
    at.mt = 8 - 2 * k;
    return at;
  }
};

// Weights' gradient: the tiles of the experts with most rows first, which take longest; each XCD takes an eighth of every
// expert's, so that what it computes at a time reads the same rows; its workgroups take them in turns, back and forth.
template <>
struct Walk<kWeightsGrad> {
  struct Table {
    int rows[256], order[256];
  };
  Table& t;
  int rank = 0, before = 0, round = 0;  // before: this XCD's tiles of the experts before `rank`
  __device__ __forceinline__ Walk(const ProductJob& j, Table& table) : t(table) {
    const int i = threadIdx.x;
    if (i < 256) {
      int r0 = 0, r1 = 0;
      if (i < j.E) expert_rows(j, i, r0, r1);
      t.rows[i] = r1 - r0;
    }
    __syncthreads();
    if (i < j.E) {
      int at = 0;
      for (int k = 0; k < j.E; ++k) at += t.rows[k] > t.rows[i] || (t.rows[k] == t.rows[i] && k < i);
      t.order[at] = i;
    }
    __syncthreads();
  }
  __device__ __forceinline__ Place next(const ProductJob& j) {
    Place at = {-1, 0, 0, 0, 0, 0, 0};
    const int ct = (j.D + kTile - 1) / kTile, V = (j.N + kTile - 1) / kTile * ct, xcd = blockIdx.x % kXcds;
    const int idx = blockIdx.x / kXcds, per = ((int)gridDim.x - xcd + kXcds - 1) / kXcds;
    int m = round * per + (round & 1 ? per - 1 - idx : idx);
    ++round;
    while (rank < j.E) {
      const int e = __builtin_amdgcn_readfirstlane(t.order[rank]), x = (xcd + rank) % kXcds;
      const int v0 = (int)((int64_t)V * x / kXcds), cnt = (int)((int64_t)V * (x + 1) / kXcds) - v0;
      if (m >= before + cnt) {
        before += cnt;
        ++rank;
        continue;
      }
      const int v = v0 + m - before;
      expert_rows(j, e, at.k0, at.kend);
      at.k0 = __builtin_amdgcn_readfirstlane(at.k0);
      at.kend = __builtin_amdgcn_readfirstlane(at.kend);
      at.p0 = v / ct * kTile;
      at.q0 = v % ct * kTile;
      at.pend = min(j.N, at.p0 + kTile);
      if (at.kend > at.k0) {
        at.e = e;
        at.mt = at.pend - at.p0 <= 128 ? 4 : 8;
        return at;
      }
      if (!j.accumulate)  // no rows: zeros, or what was there
        for (int i = threadIdx.x & 255; i < kTile * kTile / 4; i += 256) {  // (group 1 walks)
          const int p = at.p0 + i / 64, q = at.q0 + i % 64 * 4;
          if (p < j.N && q < j.D) put4(j, e * j.out_stride + p * j.out_pitch + q, f32x4{0.f, 0.f, 0.f, 0.f});
        }
      m = round * per + (round & 1 ? per - 1 - idx : idx);
      ++round;
    }
    return at;
  }
};

template <int MODE, int DT>
__global__ __launch_bounds__(512) void tiles_kernel(ProductJob j) {
  constexpr bool kScaled = esize<DT>() == 1;
  using W = Walk<MODE == kWeightsGrad ? kWeightsGrad : kForward>;
  __shared__ __attribute__((aligned(1024))) char pool[kPool];
  __shared__ float scale[kScaled ? 1024 : 1], w_scale[kScaled ? 2 * kMaxBlocks : 1];
  __shared__ int slots[MODE == kWeightsGrad ? 1 : 2 * 256];
  __shared__ typename W::Table table;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __shared__ Place place[2];
  const Lds lds = {pool, scale, w_scale, slots, place};

  W walk(j, table);
  if (wv >= 4) {
    const Place first = walk.next(j);
    if (first.e >= 0) find_rows<MODE>(j, first, slots, threadIdx.x - 256);
    if (threadIdx.x == 256) place[0] = first;
  }
  __syncthreads();
  Place at = load_place(place);
  if (at.e < 0) return;
  if (wv < 4) {
    begin_any<MODE, DT>(j, at, lds, slots, wv, lane);
    wait_copies<0>();
  }
  for (int par = 0; at.e >= 0; par ^= 1) {
    auto run = [&](auto mt) {
      if (wv < 4) at = tile<MODE, DT, mt(), 0>(j, at, walk, lds, par, wv, lane);
      else at = tile<MODE, DT, mt(), 1>(j, at, walk, lds, par, wv - 4, lane);
    };
    const int mt = at.mt;
    if (mt == 4) run(std::integral_constant<int, 4>{});
    else if (MODE == kWeightsGrad || mt == 8) run(std::integral_constant<int, 8>{});
    else if (mt == 2) run(std::integral_constant<int, MODE == kWeightsGrad ? 8 : 2>{});
    else run(std::integral_constant<int, MODE == kWeightsGrad ? 8 : 6>{});
  }
}

int run_tiles(const ProductJob& j, int dtype, int mode, int cus, hipStream_t stream) {
  const unsigned grid = (unsigned)cus;
  if (dtype == MOE_FP8_E4M3)
    return j.out_f32 ? launch(tiles_kernel<kForward, kFp8Wide>, grid, 512u, stream, j)
                     : launch(tiles_kernel<kForward, MOE_FP8_E4M3>, grid, 512u, stream, j);
  if (mode == kForward) return launch(tiles_kernel<kForward, MOE_BF16>, grid, 512u, stream, j);
  if (mode == kRowsGrad) return launch(tiles_kernel<kRowsGrad, MOE_BF16>, grid, 512u, stream, j);
  return launch(tiles_kernel<kWeightsGrad, MOE_BF16>, grid, 512u, stream, j);
}

}  // namespace moe
