// What the kernels of the experts' products share (products.hip, product_tiles.hip, product_narrow.hip).
#pragma once

#include "home.hpp"

namespace moe {

// Every kernel computes tiles of a matrix  C[p][q] = sum_k P[p][k] Q[q][k].  The matrix instruction's
// second operand is P and its first is Q, so that a lane ends up with four neighbouring q of one p, that
// is, with neighbouring elements of an output row:
//   forward        p = batch row,      q = output column, k = d    P rows along k,   Q = w[e]'s rows along k
//   rows' gradient p = batch row,      q = input column,  k = j    P rows along k,   Q = w[e]'s rows across k
//   weights'       p = output column,  q = input column,  k = row  both across k; k runs over an expert's rows
enum { kForward = 0, kRowsGrad = 1, kWeightsGrad = 2 };

struct ProductJob {
  int n, E, N, D;  // forward and rows' gradient: C is [n][N], D the contraction; weights' gradient: C is [N][D]
  const int32_t* offsets;
  const void *x, *w, *dout;
  int64_t x_rows, x_pitch, w_pitch, w_stride, dout_pitch, out_pitch, out_stride;
  const int32_t* row_slot;
  const float *x_scale, *w_scale;
  void* out;
  int out_f32, accumulate, through;  // through: outputs past the caches
  uint32_t* err;
};

constexpr int kFp8Wide = 16;  // 8-bit codes, widened to bf16 where they are multiplied (dot128)

template <int DT>
constexpr int esize() { return DT == MOE_F32 ? 4 : DT == MOE_BF16 ? 2 : 1; }

// offsets cut to an ascending range within [0, n]
__device__ __forceinline__ void expert_rows(const ProductJob& j, int e, int& r0, int& r1) {
  r0 = min(max(j.offsets[e], 0), j.n);
  r1 = max(r0, min(j.offsets[e + 1], j.n));
}

// How many tiles of S rows each expert has, four experts to a lane of a whole wave, and the sums up to them: one round
// trip to memory for all offsets.
template <int S>
struct RowTiles {
  int tiles[4], mine = 0, upto;

  __device__ __forceinline__ RowTiles(const ProductJob& j, int lane) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      int r0 = 0, r1 = 0;
      if (4 * lane + k < j.E) expert_rows(j, 4 * lane + k, r0, r1);
      tiles[k] = (r1 - r0 + S - 1) / S;
      mine += tiles[k];
    }
    upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
  }
  __device__ __forceinline__ int total() const { return __builtin_amdgcn_readlane(upto, 63); }
  // The expert of tile u < total() * ct, where a tile of rows makes ct tiles: the row tiles before it, and its own.
  __device__ __forceinline__ void find(int u, int ct, int& e, int& base, int& n) const {
    const int owner = __popcll(__ballot(upto * ct <= u));
    base = __builtin_amdgcn_readlane(upto, owner) - __builtin_amdgcn_readlane(mine, owner);
    e = 4 * owner;
    n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      n = __builtin_amdgcn_readlane(tiles[k], owner);
      if (u < (base + n) * ct) break;
      base += n;
      ++e;
    }
  }
};

// Four neighbouring elements of an output row.
template <bool NT = false>
__device__ __forceinline__ void put4(const ProductJob& j, int64_t at, f32x4 v) {
  if (j.out_f32) {
    f32x4* o = reinterpret_cast<f32x4*>((float*)j.out + at);
    if (j.accumulate) v += *o;
    st<NT>(o, v);
  } else {
    u32x2* o = reinterpret_cast<u32x2*>((uint16_t*)j.out + at);
    if (j.accumulate) {
      const u32x2 old = *o;
      v[0] += __uint_as_float(old[0] << 16);
      v[1] += __uint_as_float(old[0] & 0xffff0000u);
      v[2] += __uint_as_float(old[1] << 16);
      v[3] += __uint_as_float(old[1] & 0xffff0000u);
    }
    st<NT>(o, u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
  }
}

// product_tiles.hip: 256 x 256 tiles on the bf16 and 8-bit matrix instructions
int run_tiles(const ProductJob& j, int dtype, int mode, int cus, hipStream_t stream);
// product_narrow.hip: tiles of few rows, for products that are bound by reading the weights
int run_narrow(const ProductJob& j, int dtype, int mode, int cus, hipStream_t stream);

}  // namespace moe
