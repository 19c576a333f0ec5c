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
  int out_f32, accumulate;
  uint32_t* err;
};

template <int DT>
constexpr int esize() { return DT == MOE_F32 ? 4 : DT == MOE_BF16 ? 2 : 1; }

// offsets cut to an ascending range within [0, n]
__device__ __forceinline__ void expert_rows(const ProductJob& j, int e, int& r0, int& r1) {
  r0 = min(max(j.offsets[e], 0), j.n);
  r1 = max(r0, min(j.offsets[e + 1], j.n));
}

// Four neighbouring elements of an output row.
__device__ __forceinline__ void put4(const ProductJob& j, int64_t at, f32x4 v) {
  if (j.out_f32) {
    f32x4* o = reinterpret_cast<f32x4*>((float*)j.out + at);
    if (j.accumulate) v += *o;
    *o = v;
  } else {
    u32x2* o = reinterpret_cast<u32x2*>((uint16_t*)j.out + at);
    if (j.accumulate) {
      const u32x2 old = *o;
      v[0] += __uint_as_float(old[0] << 16);
      v[1] += __uint_as_float(old[0] & 0xffff0000u);
      v[2] += __uint_as_float(old[1] << 16);
      v[3] += __uint_as_float(old[1] & 0xffff0000u);
    }
    *o = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

// product_tiles.hip: 256 x 256 tiles on the bf16 and 8-bit matrix instructions
int run_tiles(const ProductJob& j, int dtype, int mode, int cus, hipStream_t stream);
// product_narrow.hip: tiles of few rows, for products that are bound by reading the weights
int run_narrow(const ProductJob& j, int dtype, int mode, int cus, hipStream_t stream);

}  // namespace moe
