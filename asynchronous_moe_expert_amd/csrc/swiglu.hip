// moe_swiglu, moe_swiglu_backward, moe_quantize_weights: what stands between the experts' products, and
// weights in 8 bits for them.
#include <math.h>

#include "home.hpp"

namespace moe {

// s = 1 / (1 + exp(-g)).  exp(-g) = 2^t with t = -g log2(e): t's own rounding error times ln 2 is put back to
// first order (v_exp_f32 alone is off by |g| 2^-24), so that s is within 5 x 2^-24 of itself as long as it is a normal
// number, g >= -87.3: 2 x 2^-24 of v_exp_f32, a rounding of each sum, the quotient's (g s measured: within 4.3 x 2^-24).
// Below, s is off by at most 2^-126: its subnormal values come out as 0.  Past |t| = 127 the exponential is 0 or
// infinite or about to be, and the correction, which would be NaN for infinite g, is left out.
__device__ __forceinline__ float sigmoid(float g) {
  const float t = -1.44269504f * g;
  float lo = fmaf(-1.44269504f, g, -t);      // what rounding t lost
  lo = fmaf(-1.92596299e-8f, g, lo);         // log2(e) - fl(log2(e))
  const float x = __builtin_amdgcn_exp2f(t);
  const float fix = fabsf(t) < 127.f ? x * (lo * 0.693147181f) : 0.f;
  const float d = 1.f + (x + fix);
  const float q = __builtin_amdgcn_rcpf(d);
  return d < 1e30f ? fmaf(fmaf(-d, q, 1.f), q, q) : q;  // one correction: the quotient's own rounding
}

struct SwigluJob {
  int n, I, tpr, many, groups, group_lanes;
  const void *gu, *dh;
  int64_t gu_pitch, h_pitch, dh_pitch, dgu_pitch;
  const int32_t* count;
  void *h, *dgu;
  float* h_scale;
};

constexpr int kSwigluT = 512;  // threads at most

// A row's chunks of eight columns lie on tpr threads (a multiple of 16, so that a scale's columns are a run
// of lanes), `many` short rows at a time in a workgroup.  A chunk has one owner: the gradient may lie where its inputs
// do, so no other thread may read them.  Bound by memory: 16384 rows of 2 x 2048 bf16 to bf16 take 33 us
// (6.1 TB/s), to 8 bits with a scale per 128 37 to 42 (4.0 to 4.6), with the gradients and h 61 to 63 (6.5); 256 rows
// of 2 x 2880 are a launch, 3.8.
template <int XT, int OT, int S>
__global__ __launch_bounds__(kSwigluT) void swiglu_kernel(SwigluJob j) {
  const int rows = j.count ? min(j.n, max(*j.count, 0)) : j.n;
  const int sub = j.many > 1 ? (int)threadIdx.x / j.tpr : 0, lt = (int)threadIdx.x - sub * j.tpr;
  if (sub >= j.many || lt >= j.tpr) return;  // (workgroups are whole waves, tpr is whole runs of 16)
  constexpr int xs = XT == MOE_F32 ? 4 : 2, os = OT == MOE_F32 ? 4 : OT == MOE_BF16 ? 2 : 1;
  for (int64_t t = (int64_t)blockIdx.x * j.many + sub; t < rows; t += (int64_t)gridDim.x * j.many) {
    const char* gu = (const char*)j.gu + t * j.gu_pitch * xs;
    char* h = (char*)j.h + t * j.h_pitch * os;
    for (int c = lt; c < ((j.I / 8 + 15) & ~15); c += j.tpr) {  // whole runs of 16 lanes take part
      const int at = c * 8;
      float g[8], u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = u[e] = 0.f;
      if (at < j.I) {
        Chunk<XT> a, b;
        a.template load<(S >= kReadOnce)>(gu, at);
        b.template load<(S >= kReadOnce)>(gu, j.I + at);
        a.get(g);
        b.get(u);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = g[e] * sigmoid(g[e]) * u[e];
      }
      if constexpr (OT == MOE_FP8_E4M3) {
        float a = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(g[e]));
        const Coding coded = coding_of(run_max(a, j.group_lanes), 1.f, true);
        coded(g);
        if (at < j.I && (threadIdx.x & (j.group_lanes - 1)) == 0)
          j.h_scale[t * j.groups + at / (j.group_lanes * 8)] = coded.scale;
      }
      if (at < j.I) st8<OT, S == kThrough>(h, at, g);
    }
  }
}

// One scale for a whole row: a workgroup per row, which goes over it twice (the second time from the
// caches) so that rows of any length take the same registers.  16384 rows of 2 x 2048 bf16: 55 us, where a scale per
// 128 columns takes 39: the exponentials are computed twice.
template <int XT>
__global__ __launch_bounds__(256) void swiglu_row_scale_kernel(SwigluJob j) {
  __shared__ float s_max[2][4];
  const int rows = j.count ? min(j.n, max(*j.count, 0)) : j.n;
  constexpr int xs = XT == MOE_F32 ? 4 : 2;
  int par = 0;
  for (int t = blockIdx.x; t < rows; t += gridDim.x, par ^= 1) {
    const char* gu = (const char*)j.gu + (int64_t)t * j.gu_pitch * xs;
    uint8_t* h = (uint8_t*)j.h + (int64_t)t * j.h_pitch;
    auto values = [&](int at, float* g) {
      Chunk<XT> a, b;
      float u[8];
      a.load(gu, at);
      b.load(gu, j.I + at);
      a.get(g);
      b.get(u);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = g[e] * sigmoid(g[e]) * u[e];
    };
    float amax = 0.f;
    for (int at = (int)threadIdx.x * 8; at < j.I; at += (int)blockDim.x * 8) {
      float g[8];
      values(at, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(g[e]));
    }
    amax = wave_max(amax);
    if ((threadIdx.x & 63) == 0) s_max[par][threadIdx.x >> 6] = amax;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x >> 6; ++w) amax = fmaxf(amax, s_max[par][w]);
    const Coding coded = coding_of(amax, 1.f, true);
    if (threadIdx.x == 0) j.h_scale[t] = coded.scale;
    for (int at = (int)threadIdx.x * 8; at < j.I; at += (int)blockDim.x * 8) {
      float g[8];
      values(at, g);
      coded(g);
      st8<MOE_FP8_E4M3>(h, at, g);
    }
  }
}

template <int DT, int S>
__global__ __launch_bounds__(kSwigluT) void swiglu_backward_kernel(SwigluJob j) {
  const int rows = j.count ? min(j.n, max(*j.count, 0)) : j.n;
  const int sub = j.many > 1 ? (int)threadIdx.x / j.tpr : 0, lt = (int)threadIdx.x - sub * j.tpr;
  if (sub >= j.many || lt >= j.tpr) return;  // (workgroups are whole waves, tpr is whole runs of 16)
  constexpr int xs = DT == MOE_F32 ? 4 : 2;
  for (int64_t t = (int64_t)blockIdx.x * j.many + sub; t < rows; t += (int64_t)gridDim.x * j.many) {
    const char* gu = (const char*)j.gu + t * j.gu_pitch * xs;
    const char* dh = (const char*)j.dh + t * j.dh_pitch * xs;
    char* dgu = (char*)j.dgu + t * j.dgu_pitch * xs;
    char* h = (char*)j.h + t * j.h_pitch * xs;
    for (int at = lt * 8; at < j.I; at += j.tpr * 8) {
      Chunk<DT> a, b, c;
      a.template load<(S >= kReadOnce)>(gu, at);
      b.template load<(S >= kReadOnce)>(gu, j.I + at);
      c.template load<(S >= kReadOnce)>(dh, at);
      float g[8], u[8], d[8];
      a.get(g);
      b.get(u);
      c.get(d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = sigmoid(g[e]), silu = g[e] * s, keep = u[e];
        u[e] = d[e] * silu;
        d[e] *= keep * s * fmaf(g[e], 1.f - s, 1.f);
        g[e] = silu * keep;
      }
      st8<DT, S == kThrough>(dgu, at, d);
      st8<DT, S == kThrough>(dgu, j.I + at, u);
      if (j.h) st8<DT, S == kThrough>(h, at, g);
    }
  }
}

struct QuantizeJob {
  int N, D;
  const void* w;
  int64_t w_pitch, w_stride, codes_pitch, codes_stride;
  uint8_t* codes;
  float* scale;
};

// A workgroup per 128 x 128 block, 64 values a thread; the transposed codes cross through LDS.  Bound by
// memory: 32 x 4096 x 4096 bf16 285 us (5.7 TB/s), transposed 284.
template <int DT, bool T>
__global__ __launch_bounds__(256) void quantize_kernel(QuantizeJob j) {
  __shared__ float s_max[4];
  constexpr int kRow = 136;  // bytes between a transposed tile's rows: 128 and 8, so that they do not share banks
  __shared__ __attribute__((aligned(16))) uint8_t s_t[T ? 128 * kRow : 16];
  const int nb = (j.N + 127) / 128, db = (j.D + 127) / 128;
  const int e = blockIdx.x / (nb * db), b = blockIdx.x - e * nb * db, bn = b / db, bd = b - bn * db;
  constexpr int xs = DT == MOE_F32 ? 4 : 2;
  const char* w = (const char*)j.w + e * j.w_stride * xs;
  const int at = bd * 128 + (int)(threadIdx.x & 15) * 8, row0 = bn * 128 + (int)(threadIdx.x >> 4);
  float v[8][8], amax = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = 0.f;
    if (row0 + 16 * k < j.N && at < j.D) {
      Chunk<DT> q;
      q.load(w + (int64_t)(row0 + 16 * k) * j.w_pitch * xs, at);
      q.get(v[k]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[k][i]));
  }
  amax = wave_max(amax);
  if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) amax = fmaxf(amax, s_max[k]);
  const Coding coded = coding_of(amax, 1.f, true);
  if (threadIdx.x == 0) j.scale[(int64_t)e * nb * db + (T ? bd * nb + bn : b)] = coded.scale;
  uint8_t* codes = j.codes + e * j.codes_stride;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    coded(v[k]);
    const int row = row0 + 16 * k;
    if constexpr (!T) {
      if (row < j.N && at < j.D) st8<MOE_FP8_E4M3>(codes + (int64_t)row * j.codes_pitch, at, v[k]);
    } else {
      uint8_t q[8] __attribute__((aligned(8)));
      st8<MOE_FP8_E4M3>(q, 0, v[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) s_t[((threadIdx.x & 15) * 8 + i) * kRow + (threadIdx.x >> 4) + 16 * k] = q[i];
    }
  }
  if constexpr (T) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int d = (int)(threadIdx.x >> 4) + 16 * k, n = (int)(threadIdx.x & 15) * 8;
      if (bd * 128 + d < j.D && bn * 128 + n < j.N)
        *reinterpret_cast<u32x2*>(codes + (int64_t)(bd * 128 + d) * j.codes_pitch + bn * 128 + n) =
            *reinterpret_cast<const u32x2*>(s_t + d * kRow + n);
    }
  }
}

// threads to a row and rows to a workgroup: the lanes that cover a row's chunks, in whole runs of 16
static void swiglu_shape(SwigluJob& j, unsigned& grid, unsigned& block) {
  const int run = (j.I / 8 + 15) / 16 * 16;
  const int passes = (run + kSwigluT - 1) / kSwigluT;
  j.tpr = ((run + passes - 1) / passes + 15) / 16 * 16;
  j.many = j.tpr <= 128 ? 256 / j.tpr : 1;
  block = (unsigned)((j.tpr * j.many + 63) / 64 * 64);
  grid = grid_of(((int64_t)j.n + j.many - 1) / j.many);
}

template <int XT, int OT>
static int swiglu_by_kind(const SwigluJob& j0, int kind, hipStream_t stream) {
  SwigluJob j = j0;
  unsigned grid, block;
  swiglu_shape(j, grid, block);
  if (kind == kThrough) return launch(swiglu_kernel<XT, OT, kThrough>, grid, block, stream, j);
  if (kind == kReadOnce) return launch(swiglu_kernel<XT, OT, kReadOnce>, grid, block, stream, j);
  return launch(swiglu_kernel<XT, OT, kNear>, grid, block, stream, j);
}

template <int XT>
static int swiglu_by_out(const SwigluJob& j, int ot, int kind, hipStream_t stream) {
  if (ot == MOE_F32) return swiglu_by_kind<XT, MOE_F32>(j, kind, stream);
  if (ot == MOE_BF16) return swiglu_by_kind<XT, MOE_BF16>(j, kind, stream);
  if (j.group_lanes) return swiglu_by_kind<XT, MOE_FP8_E4M3>(j, kind, stream);
  const int chunks = (j.I / 8 + 63) / 64 * 64;
  return launch(swiglu_row_scale_kernel<XT>, grid_of(j.n), (unsigned)(chunks < 256 ? chunks : 256), stream, j);
}

template <int DT>
static int swiglu_backward_by_kind(const SwigluJob& j0, int kind, hipStream_t stream) {
  SwigluJob j = j0;
  unsigned grid, block;
  swiglu_shape(j, grid, block);
  if (kind == kThrough) return launch(swiglu_backward_kernel<DT, kThrough>, grid, block, stream, j);
  if (kind == kReadOnce) return launch(swiglu_backward_kernel<DT, kReadOnce>, grid, block, stream, j);
  return launch(swiglu_backward_kernel<DT, kNear>, grid, block, stream, j);
}

static bool plain_type(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }

}  // namespace moe

using namespace moe;

extern "C" int moe_swiglu(const moe_swiglu_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  if (a->n < 0 || a->n > (1 << 24) || a->I < 1 || a->I > kHMaxRows / 2) return MOE_EINVAL_SIZE;
  const bool fp8 = a->h_dtype == MOE_FP8_E4M3;
  if (!plain_type(a->dtype) || !(plain_type(a->h_dtype) || fp8)) return MOE_EINVAL_DTYPE;
  if (a->I % 8) return MOE_EINVAL_SHAPE;
  if (a->gu_pitch < 2 * a->I || a->h_pitch < a->I) return MOE_EINVAL_SIZE;
  if (fp8 && a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128) return MOE_EINVAL_SIZE;
  if (a->n == 0) return MOE_OK;
  if (!a->gu || !a->h || (fp8 && !a->h_scale)) return MOE_EINVAL_NULL;
  const int xs = dtype_size(a->dtype), os = dtype_size(a->h_dtype);
  if (!aligned_rows(a->gu, a->gu_pitch, xs, 16) || !aligned_rows(a->h, a->h_pitch, os, chunk_align(a->h_dtype)))
    return MOE_EINVAL_ALIGN;
  SwigluJob j = {};
  j.n = a->n; j.I = a->I; j.gu = a->gu; j.gu_pitch = a->gu_pitch; j.count = a->count;
  j.h = a->h; j.h_pitch = a->h_pitch; j.h_scale = a->h_scale;
  j.group_lanes = fp8 ? a->group / 8 : 0;
  j.groups = fp8 && a->group ? (a->I + a->group - 1) / a->group : 1;
  const int kind = stream_kind((int64_t)a->n * a->I * (2 * xs + os));
  return a->dtype == MOE_F32 ? swiglu_by_out<MOE_F32>(j, a->h_dtype, kind, stream)
                             : swiglu_by_out<MOE_BF16>(j, a->h_dtype, kind, stream);
}

extern "C" int moe_swiglu_backward(const moe_swiglu_backward_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  if (a->n < 0 || a->n > (1 << 24) || a->I < 1 || a->I > kHMaxRows / 2) return MOE_EINVAL_SIZE;
  if (!plain_type(a->dtype)) return MOE_EINVAL_DTYPE;
  if (a->I % 8) return MOE_EINVAL_SHAPE;
  if (a->gu_pitch < 2 * a->I || a->dgu_pitch < 2 * a->I || a->dh_pitch < a->I || (a->h && a->h_pitch < a->I))
    return MOE_EINVAL_SIZE;
  if (a->n == 0) return MOE_OK;
  if (!a->gu || !a->dh || !a->dgu) return MOE_EINVAL_NULL;
  const int xs = dtype_size(a->dtype);
  if (!aligned_rows(a->gu, a->gu_pitch, xs, 16) || !aligned_rows(a->dh, a->dh_pitch, xs, 16) ||
      !aligned_rows(a->dgu, a->dgu_pitch, xs, 16) || (a->h && !aligned_rows(a->h, a->h_pitch, xs, 16)))
    return MOE_EINVAL_ALIGN;
  SwigluJob j = {};
  j.n = a->n; j.I = a->I; j.gu = a->gu; j.gu_pitch = a->gu_pitch; j.count = a->count;
  j.dh = a->dh; j.dh_pitch = a->dh_pitch; j.dgu = a->dgu; j.dgu_pitch = a->dgu_pitch; j.h = a->h; j.h_pitch = a->h_pitch;
  const int kind = stream_kind((int64_t)a->n * a->I * xs * (a->h ? 6 : 5));
  return a->dtype == MOE_F32 ? swiglu_backward_by_kind<MOE_F32>(j, kind, stream)
                             : swiglu_backward_by_kind<MOE_BF16>(j, kind, stream);
}

extern "C" int moe_quantize_weights(const moe_quantize_weights_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  if (a->E_loc < 1 || a->E_loc > 256 || a->N < 1 || a->N > kHMaxRows || a->D < 1 || a->D > kHMaxRows ||
      (a->transposed != 0 && a->transposed != 1))
    return MOE_EINVAL_SIZE;
  if (!plain_type(a->dtype)) return MOE_EINVAL_DTYPE;
  if (a->N % 8 || a->D % 8) return MOE_EINVAL_SHAPE;
  const int out_rows = a->transposed ? a->D : a->N, out_cols = a->transposed ? a->N : a->D;
  if (a->w_pitch < a->D || a->codes_pitch < out_cols || a->w_pitch > ((int64_t)1 << 32) ||
      a->codes_pitch > ((int64_t)1 << 32))
    return MOE_EINVAL_SIZE;
  if (a->E_loc > 1 && (a->w_stride < (int64_t)(a->N - 1) * a->w_pitch + a->D ||
                       a->codes_stride < (int64_t)(out_rows - 1) * a->codes_pitch + out_cols))
    return MOE_EINVAL_SIZE;
  if (!a->w || !a->codes || !a->scale) return MOE_EINVAL_NULL;
  const int xs = dtype_size(a->dtype);
  if (!aligned_rows(a->w, a->w_pitch, xs, 16) || (a->E_loc > 1 && (a->w_stride * xs) % 16) ||
      !aligned_rows(a->codes, a->codes_pitch, 1, 8) || (a->E_loc > 1 && a->codes_stride % 8))
    return MOE_EINVAL_ALIGN;
  QuantizeJob j;
  j.N = a->N; j.D = a->D; j.w = a->w; j.w_pitch = a->w_pitch; j.w_stride = a->w_stride;
  j.codes = (uint8_t*)a->codes; j.codes_pitch = a->codes_pitch; j.codes_stride = a->codes_stride; j.scale = a->scale;
  const int64_t blocks = (int64_t)a->E_loc * ((a->N + 127) / 128) * ((a->D + 127) / 128);  // at most 2^26
  // grids stay below 2^32 threads: as many as 2^26 blocks are 2^34, so experts are taken some at a time
  const int64_t per = blocks / a->E_loc;
  const int step = (int)(((int64_t)1 << 23) / per > 0 ? ((int64_t)1 << 23) / per : 1);
  for (int e = 0; e < a->E_loc; e += step) {
    const int k = a->E_loc - e < step ? a->E_loc - e : step;
    QuantizeJob q = j;
    q.w = (const char*)j.w + (a->E_loc > 1 ? e * j.w_stride * xs : 0);
    q.codes += a->E_loc > 1 ? e * j.codes_stride : 0;
    q.scale += e * per;
    const unsigned grid = (unsigned)(per * k);
    const int rc = a->dtype == MOE_F32
                       ? (a->transposed ? launch(quantize_kernel<MOE_F32, true>, grid, 256u, stream, q)
                                        : launch(quantize_kernel<MOE_F32, false>, grid, 256u, stream, q))
                       : (a->transposed ? launch(quantize_kernel<MOE_BF16, true>, grid, 256u, stream, q)
                                        : launch(quantize_kernel<MOE_BF16, false>, grid, 256u, stream, q));
    if (rc != MOE_OK) return rc;
  }
  return MOE_OK;
}
