// The experts' products on large tiles: 256 x 256 of C, bf16 (v_mfma_f32_16x16x32_bf16) or 8 bits
// (v_mfma_f32_16x16x128_f8f6f4 with fp32 scales), operands copied straight into LDS.
#include <type_traits>

#include "product_copy.hpp"

namespace moe {

constexpr int kTile = 256;

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
  static constexpr bool kScaled = DT == MOE_FP8_E4M3;
  static constexpr int kHalf = MT / 2;
  // copies that a wave of group 0 makes in a step: of each group's rows of P, of Q, and of the rows' scales
  static constexpr int kP = MT / 2, kQ = 8, kScales = kScaled ? 1 : 0;
  static constexpr int kFirst = kQ + kP + kScales, kSecond = kP;
};
// NB blocks of 64 columns of an operand whose rows lie across k: byte offsets of this lane's copies from row k0 of
// the matrix, two copies to a block, of row() and of the row 32 further.  Columns past the end are read at others.
template <int NB>
struct Across {
  uint32_t off[NB];
  __device__ __forceinline__ void set(int wq, int lane, int col0, int cols, int64_t pitch, int es) {
    const int k = row(wq, lane), f = ((k >> 1) & 1) | ((k >> 3) & 1) << 1, piece = (lane & 7) ^ (2 * f);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int first = col0 + 64 * b < cols ? col0 + 64 * b : col0 < cols ? col0 : 0;
      off[b] = (uint32_t)(k * (int)pitch * es + (first + min(piece * 8, cols - 8 - first)) * es);
    }
  }
  static __device__ __forceinline__ int row(int wq, int lane) { return 8 * wq + (lane >> 3); }
  // step `step` of the contraction's rows 0 .. end - 1, which begin at base
  __device__ __forceinline__ void copy(const char* base, int64_t pitch_bytes, uint32_t dst, int step, int end, int wq,
                                       int lane) const {
    const char* from = uniform_ptr(base + (int64_t)step * kStep * pitch_bytes);
    const char* odd = uniform_ptr(from + 32 * pitch_bytes);
    if ((step + 1) * kStep <= end) {
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c) copy16(c & 1 ? odd : from, off[c >> 1], dst + c * 4096);
    } else {
      const int k = step * kStep + row(wq, lane);
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c) {
        const char* src = (c & 1 ? odd : from) + off[c >> 1];
        copy16(k + 32 * (c & 1) < end ? src : (const char*)&g_zeros, dst + c * 4096);
      }
    }
  }
};

// What a workgroup has in LDS: two stages of P (16 KiB for each group's rows) and of Q, four of the rows' scales.
struct Lds {
  u32x4 *p[2], *q[2];
  float *scale, *w_scale;
};


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

// The row of the tile's P that lies at place r of group h's 16 MT, and where it comes from (-1: nowhere).
template <int MT>
__device__ __forceinline__ int64_t p_source(const ProductJob& j, const Place& at, int h, int r) {
  const int row = min(at.p0 + h * 16 * MT + min(r, 16 * MT - 1), at.pend - 1);
  if (!j.row_slot) return row;
  const int64_t slot = j.row_slot[row];
  return slot < 0 || slot >= j.x_rows ? -1 : slot;
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
  int steps;

  static __device__ __forceinline__ int ppiece(int wq, int lane) { return (lane & 7) ^ (4 * (wq & 1) + (lane >> 4)); }
  static __device__ __forceinline__ int qpiece(int wq, int lane) { return (lane & 7) ^ (((lane >> 4) & 1) | 2 * wq); }

  __device__ __forceinline__ void set(const ProductJob& j, const Place& at, int steps_, int wq, int lane) {
    pieces = j.D * es / 16;
    steps = steps_;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (T::kPAlong) {
#pragma unroll
        for (int c = 0; c < T::kP; ++c) {
          int64_t slot = p_source<MT>(j, at, h, 8 * (4 * c + wq) + (lane >> 3));
          if (slot < 0) {
            atomicOr(j.err, MOE_ERR_SLOT_RANGE);
            slot = 0;
            nosrc |= 1u << (h * T::kP + c);
          }
          poff[h][c] = (uint32_t)(slot * (j.x_pitch * es / 16) + ppiece(wq, lane));
        }
      } else {
        pa[h].set(wq, lane, at.p0 + h * 16 * MT, j.N, j.dout_pitch, es);
      }
    }
    if constexpr (T::kScaled) {
      const int64_t slot = p_source<MT>(j, at, wq >> 1, (wq & 1) * 64 + lane);
      if (slot < 0) nosrc |= 1u << 31;
      else sptr = j.x_scale + slot * ((j.D + 127) / 128);
    }
    sourced = __ballot(nosrc != 0) == 0;
    if constexpr (T::kQAlong) qoff = (uint32_t)((lane >> 3) * (int)j.w_pitch * es + qpiece(wq, lane) * 16);
    else qa.set(wq, lane, at.q0, MODE == kWeightsGrad ? j.D : j.N, MODE == kWeightsGrad ? j.x_pitch : j.w_pitch, es);
  }
  __device__ __forceinline__ void p_half(const ProductJob& j, const Place& at, int h, const u32x4* stage, int step, int wq,
                                         int lane) const {
    const uint32_t dst = lds_at(stage) + h * 16384 + wq * 1024;
    if constexpr (T::kPAlong) {
      const char* from = uniform_ptr(p_base<MODE, DT>(j, at) + (int64_t)step * 128);
      if (sourced && (step + 1) * 8 <= pieces) {
#pragma unroll
        for (int c = 0; c < T::kP; ++c) copy16(from + (uint64_t)poff[h][c] * 16, dst + c * 4096);
      } else {
#pragma unroll
        for (int c = 0; c < T::kP; ++c)
          copy16(step * 8 + ppiece(wq, lane) < pieces && !(nosrc >> (h * T::kP + c) & 1) ? from + (uint64_t)poff[h][c] * 16
                                                                                        : (const char*)&g_zeros,
                 dst + c * 4096);
      }
    } else {
      pa[h].copy(p_base<MODE, DT>(j, at), j.dout_pitch * es, dst, step, at.kend - at.k0, wq, lane);
    }
  }
  // Q, group 0's rows of P, and all rows' scales
  __device__ __forceinline__ void first(const ProductJob& j, const Place& at, const Lds& lds, int step, int wq,
                                        int lane) const {
    const int Qn = MODE == kWeightsGrad ? j.D : j.N;
    const uint32_t dst = lds_at(lds.q[step & 1]) + wq * 1024;
    const char* q = q_base<MODE, DT>(j, at);
    if constexpr (T::kQAlong) {  // N is a multiple of 8, so rows are past it by whole copies: read at the first ones
      const bool whole = (step + 1) * 8 <= pieces;
#pragma unroll
      for (int c = 0; c < T::kQ; ++c) {
        const int r = 8 * (4 * c + wq);
        const char* from = uniform_ptr(q + (int64_t)step * 128 + (at.q0 + r < Qn ? r : 0) * j.w_pitch * es);
        if (whole) copy16(from, qoff, dst + c * 4096);
        else copy16(step * 8 + qpiece(wq, lane) < pieces ? from + qoff : (const char*)&g_zeros, dst + c * 4096);
      }
    } else {
      qa.copy(q, q_pitch<MODE, DT>(j), dst, step, at.kend - at.k0, wq, lane);
    }
    p_half(j, at, 0, lds.p[step & 1], step, wq, lane);
    if constexpr (T::kScaled) {
      const char* src = !(nosrc >> 31) ? (const char*)(sptr + step) : (const char*)&g_zeros;
      copy4(src, lds_at(lds.scale) + (step & 3) * 1024 + wq * 256);
    }
  }
  __device__ __forceinline__ void second(const ProductJob& j, const Place& at, const Lds& lds, int step, int wq,
                                         int lane) const {
    p_half(j, at, 1, lds.p[step & 1], step, wq, lane);
  }
};

template <int MODE, int DT, int MT, int G>
__device__ __forceinline__ void tile(const ProductJob& j, const Place& at, const Lds& lds, int wq, int lane) {
  using T = Tile<MODE, DT, MT>;
  constexpr int es = T::es, kHalf = T::kHalf;
  const int g = lane >> 4, l16 = lane & 15;
  const int steps = MODE == kWeightsGrad ? (at.kend - at.k0 + kStep - 1) / kStep : (j.D * es + 127) / 128;
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
  auto along = [&](const u32x4* stage, int at_) { return *reinterpret_cast<const u32x4*>((const char*)stage + at_); };
  auto across = [&](const u32x4* stage, int at_) -> u32x4 {
    const char* b = (const char*)stage + at_;
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
  auto read_p = [&](const u32x4* ps, const float* ss, int a0, int a, int at0, int at1) {  // tile a0 + a of the group's rows
    if constexpr (T::kPAlong) {
      pf[a][0] = along(ps, at0 + (a0 + a) * 2048);
      pf[a][1] = along(ps, at1 + (a0 + a) * 2048);
    }
    if constexpr (T::kScaled) sc[a] = ss[G * 128 + (a0 + a) * 16 + l16];
  };
  auto read = [&](const u32x4* ps, const u32x4* qs, const float* ss, int step) {
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
        v[b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q, p, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
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
  auto multiply = [&](const u32x4* ps, const float* ss) {
    __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
    int p1 = 0;
    if constexpr (T::kPAlong) p1 = flip(pr, 64);
#pragma unroll
    for (int a = 0; a < kHalf; ++a) {
      row(0, a);
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

  if constexpr (T::kScaled) {  // the scales of the tile's two blocks of columns
    const int nb = (j.N + 127) / 128;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float* from = j.w_scale + ((int64_t)at.e * nb + min((at.q0 >> 7) + b, nb - 1)) * steps;
      for (int k = G * 256 + wq * 64 + lane; k < steps; k += 512) lds.w_scale[b * kMaxBlocks + k] = from[k];
    }
    wait_lds();
  }

  // ---- The waves of a SIMD, one of each group, take turns: while one multiplies a step's fragments, which it
  // holds in registers, the other reads its next ones (Q's and half of P's; the other half takes the place of
  // what has been multiplied).  Group 0 reads step i in phase 2 i and multiplies in phase 2 i + 1, group 1 one
  // phase later; a barrier ends each phase.  So of a stage, Q and group 0's rows of P are free after phase 2 i + 1,
  // group 1's after 2 i + 2: group 0 copies step i + 2 there in the phase after, two phases before it is read.
  if constexpr (G == 0) {
    Copies<MODE, DT, MT> c;
    c.set(j, at, steps, wq, lane);
    c.first(j, at, lds, 0, wq, lane);
    c.second(j, at, lds, 0, wq, lane);
    wait_copies<T::kSecond>();
    meet();
#pragma clang loop unroll(disable)
    for (int i = 0; i < steps; i += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (i + h >= steps) break;
        const u32x4* ps = lds.p[h];
        const float* ss = lds.scale + ((i + h) & 3) * 256;
        if (i + h + 1 < steps) c.first(j, at, lds, i + h + 1, wq, lane);
        read(ps, lds.q[h], ss, i + h);
        wait_lds();
        if (i + h + 1 < steps) wait_copies<T::kFirst>();
        else wait_copies<0>();
        meet();
        if (i + h + 1 < steps) c.second(j, at, lds, i + h + 1, wq, lane);
        multiply(ps, ss);
        wait_copies<T::kSecond>();
        meet();
      }
    }
    meet();
  } else {
    meet();
    meet();
#pragma clang loop unroll(disable)
    for (int i = 0; i < steps; i += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (i + h >= steps) break;
        const u32x4* ps = lds.p[h] + 1024;
        const float* ss = lds.scale + ((i + h) & 3) * 256;
        read(ps, lds.q[h], ss, i + h);
        wait_lds();
        meet();
        multiply(ps, ss);
        meet();
      }
    }
  }

  // ---- outputs
  const int64_t out0 = MODE == kWeightsGrad ? at.e * j.out_stride : 0;
#pragma unroll
  for (int a = 0; a < MT; ++a) {
    const int p = at.p0 + G * 16 * MT + a * 16 + l16;
    const int64_t at0 = out0 + p * j.out_pitch;
    if (j.out_f32 || j.accumulate) {
      if (p >= at.pend) continue;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int q = at.q0 + 64 * wq + (T::kQAlong ? 32 * (b >> 1) + 8 * g + 4 * (b & 1) : 16 * b + 4 * g);
        if (q < Qn) put4(j, at0 + q, acc[a][b]);
      }
    } else {
#pragma unroll
      for (int b = 0; b < 4; b += 2) {
        u32x4 v = {pack_bf16x2(acc[a][b][0], acc[a][b][1]), pack_bf16x2(acc[a][b][2], acc[a][b][3]),
                   pack_bf16x2(acc[a][b + 1][0], acc[a][b + 1][1]), pack_bf16x2(acc[a][b + 1][2], acc[a][b + 1][3])};
        if constexpr (!T::kQAlong) neighbours(v);
        const int q = at.q0 + 64 * wq + 16 * b + 8 * g;
        if (p < at.pend && q < Qn) *reinterpret_cast<u32x4*>((uint16_t*)j.out + at0 + q) = v;
      }
    }
  }
}

constexpr int kXcds = 8;

template <int MODE, int DT>
__global__ __launch_bounds__(512) void tiles_kernel(ProductJob j) {
  __shared__ u32x4 p0[2048], p1[2048], q0[2048], q1[2048];
  constexpr bool kScaled = DT == MOE_FP8_E4M3;
  __shared__ float scale[kScaled ? 1024 : 1], w_scale[kScaled ? 2 * kMaxBlocks : 1];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int Qn = MODE == kWeightsGrad ? j.D : j.N, ct = (Qn + kTile - 1) / kTile;
  const Lds lds = {{p0, p1}, {q0, q1}, scale, w_scale};

  auto run = [&](const Place& at, auto mt) {
    if (wv < 4) tile<MODE, DT, mt(), 0>(j, at, lds, wv, lane);
    else tile<MODE, DT, mt(), 1>(j, at, lds, wv - 4, lane);
  };
  const int xcd = blockIdx.x % kXcds, idx = blockIdx.x / kXcds, per = (gridDim.x - xcd + kXcds - 1) / kXcds;

  if constexpr (MODE == kWeightsGrad) {
    const int rt = (j.N + kTile - 1) / kTile, V = rt * ct;
    // each XCD takes an eighth of every expert's tiles, so that all of them have the same share of every
    // expert's rows
    int pos = idx;
    for (int e = 0; e < j.E; ++e) {
      const int x = (xcd + e) % kXcds, v0 = (int)((int64_t)V * x / kXcds), cnt = (int)((int64_t)V * (x + 1) / kXcds) - v0;
      if (pos >= cnt) {
        pos -= cnt;
        continue;
      }
      Place at;
      at.e = e;
      expert_rows(j, e, at.k0, at.kend);
      at.k0 = __builtin_amdgcn_readfirstlane(at.k0);
      at.kend = __builtin_amdgcn_readfirstlane(at.kend);
      for (; pos < cnt; pos += per) {
        const int v = v0 + pos;
        at.p0 = v / ct * kTile;
        at.q0 = v % ct * kTile;
        at.pend = min(j.N, at.p0 + kTile);
        if (at.kend == at.k0) {  // no rows: zeros, or what was there
          if (!j.accumulate)
            for (int i = threadIdx.x; i < kTile * kTile / 4; i += 512) {
              const int p = at.p0 + i / 64, q = at.q0 + i % 64 * 4;
              if (p < j.N && q < Qn) put4(j, e * j.out_stride + p * j.out_pitch + q, f32x4{0.f, 0.f, 0.f, 0.f});
            }
          continue;
        }
        if (at.pend - at.p0 <= 128) run(at, std::integral_constant<int, 4>{});
        else run(at, std::integral_constant<int, 8>{});
      }
      pos -= cnt;
    }
  } else {
    // four experts to a lane: how many row tiles each has, the sum over those before
    __shared__ int s_tiles[256], s_upto[64];
    int upto = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      int r0 = 0, r1 = 0;
      if (4 * lane + k < j.E) expert_rows(j, 4 * lane + k, r0, r1);
      const int tiles = (r1 - r0 + kTile - 1) / kTile;
      if (wv == 0) s_tiles[4 * lane + k] = tiles;
      upto += tiles;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    if (wv == 0) s_upto[lane] = upto;
    const int total = __builtin_amdgcn_readlane(upto, 63) * ct;
    __syncthreads();
    const int u0 = (int)((int64_t)total * xcd / kXcds), u1 = (int)((int64_t)total * (xcd + 1) / kXcds);
    for (int u = u0 + idx; u < u1; u += per) {
      // the expert whose tiles u lies among
      const int owner = __popcll(__ballot(s_upto[lane] * ct <= u));
      int e = 4 * owner, base = owner ? s_upto[owner - 1] : 0, tiles = s_tiles[e];
      while (u >= (base + tiles) * ct) {
        base += tiles;
        tiles = s_tiles[++e];
      }
      e = __builtin_amdgcn_readfirstlane(e);
      base = __builtin_amdgcn_readfirstlane(base);
      tiles = __builtin_amdgcn_readfirstlane(tiles);
      int r0, r1;
      expert_rows(j, e, r0, r1);
      // tiles of one expert: bands of at most eight row tiles, in a band the row tiles of one column block
      // after the other, so that workgroups of an XCD share rows and weights in its L2
      const int v = u - base * ct, bands = (tiles + 7) / 8, bh = (tiles + bands - 1) / bands;
      const int band = v / (bh * ct), h = min(bh, tiles - band * bh), w = v - band * bh * ct;
      Place at;
      at.e = e;
      at.p0 = __builtin_amdgcn_readfirstlane(r0 + (band * bh + w % h) * kTile);
      at.q0 = __builtin_amdgcn_readfirstlane(w / h * kTile);
      at.pend = __builtin_amdgcn_readfirstlane(min(r1, at.p0 + kTile));
      at.k0 = 0;
      at.kend = j.D;
      const int rows = at.pend - at.p0;
      if (rows <= 64) run(at, std::integral_constant<int, 2>{});
      else if (rows <= 128) run(at, std::integral_constant<int, 4>{});
      else if (rows <= 192) run(at, std::integral_constant<int, 6>{});
      else run(at, std::integral_constant<int, 8>{});
    }
  }
  wait_copies<0>();  // nothing lands in this LDS once it is another workgroup's
}

int run_tiles(const ProductJob& j, int dtype, int mode, int units, hipStream_t stream) {
  const unsigned cus = (unsigned)units;
  if (dtype == MOE_FP8_E4M3) return launch(tiles_kernel<kForward, MOE_FP8_E4M3>, cus, 512u, stream, j);
  if (mode == kForward) return launch(tiles_kernel<kForward, MOE_BF16>, cus, 512u, stream, j);
  if (mode == kRowsGrad) return launch(tiles_kernel<kRowsGrad, MOE_BF16>, cus, 512u, stream, j);
  return launch(tiles_kernel<kWeightsGrad, MOE_BF16>, cus, 512u, stream, j);
}

}  // namespace moe
