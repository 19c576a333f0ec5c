// moe_residual_norm, moe_residual_norm_backward: h = x + residual, y = h * rsqrt(mean h^2 + eps) *
// gamma in fp32, bf16 or 8 bits with scales; and its gradient.  A row stays in registers between
// its reduction and its output, so each input is read once and each output written once.
#include <math.h>

#include "home.hpp"

namespace moe {

constexpr int kNormT = 512, kNormWaves = kNormT / kWave;  // at most
constexpr int kNormH = 16384;     // longest row: 512 threads x 4 chunks of 8
constexpr int kPartials = 512;    // rows of the workspace that the sum over tokens goes through

struct NormJob {
  int T, H, groups, group_lanes, gamma_f32;  // group_lanes: lanes per scale, 0 for one per row
  float eps;
  const void *x, *residual, *gamma;
  int64_t x_pitch, res_pitch, out_pitch, res_out_pitch;
  void *out, *residual_out;
  float *out_scale, *rstd;
  const int32_t *row_list, *row_count;
  uint32_t* err;
};

template <int DT>
__device__ __forceinline__ int64_t row_bytes(int64_t t, int64_t pitch) {
  return t * pitch * (DT == MOE_F32 ? 4 : DT == MOE_BF16 ? 2 : 1);
}

__device__ __forceinline__ void gamma8(const void* gamma, int f32, int64_t at, float* g) {
  if (f32) {
    Chunk<MOE_F32> q;
    q.load(gamma, at);
    q.get(g);
  } else {
    Chunk<MOE_BF16> q;
    q.load(gamma, at);
    q.get(g);
  }
}

// The workgroup's sum / maximum in every thread; s[] is free again after the next barrier.
__device__ __forceinline__ float group_sum(float v, float* s) {
  v = wave_sum(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  float all = s[0];
  for (int w = 1; w < waves; ++w) all += s[w];
  return all;
}
__device__ __forceinline__ float group_max(float v, float* s) {
  v = wave_max(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  float all = s[0];
  for (int w = 1; w < waves; ++w) all = fmaxf(all, s[w]);
  return all;
}

// group_sum of the row group `sub` of a workgroup that holds several rows, tpr threads to each
template <bool MANY>
__device__ __forceinline__ float rows_sum(float v, float* s, int sub, int tpr) {
  if constexpr (!MANY) {
    return group_sum(v, s);
  } else {
    v = wave_sum(v);
    const int waves = tpr >> 6;
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    float all = s[sub * waves];
    for (int w = 1; w < waves; ++w) all += s[sub * waves + w];
    return all;
  }
}

// Bound by memory: 16384 x 4096 bf16 with the residual, 8 bits out, 470 MB in 80 us a call (5.9 TB/s); 8192 x
// 2880, bf16 out, 189 MB in 32 us.  The fp8 outputs' arithmetic shows as well (84 us before the
// ordinary groups had their own branch).  A call of 64 rows is launch and latency, 4.0 us.  Rows of
// four chunks per thread in bf16 are held to six waves per SIMD, three workgroups per CU (4096 x 16384
// to 8 bits 82 us, 85 with two); in fp32 that would spill (98 instead of 89 us).
// A workgroup per row (rows blockIdx, blockIdx + gridDim, ...); thread i holds the chunks i, i + blockDim, ...
template <int XT, int RT, int OT, int C, int S>
__global__ __launch_bounds__(kNormT, RT == MOE_BF16 ? 6 : 4) void norm_kernel(NormJob j) {
  __shared__ float s_a[2][kNormWaves], s_b[2][kNormWaves];
  const int rows = j.row_list ? min(j.T, *j.row_count) : j.T;
  int par = 0;
  for (int k = blockIdx.x; k < rows; k += gridDim.x) {
    int t = k;
    if (j.row_list) {
      t = j.row_list[k];
      if (t < 0 || t >= j.T) {
        if (threadIdx.x == 0) atomicOr(j.err, MOE_ERR_ROW_RANGE);
        continue;
      }
    }
    const char* x = (const char*)j.x + row_bytes<XT>(t, j.x_pitch);
    // G chunks' loads before the first use: one chunk after the other took 85 instead of 81 us at
    // 16384 x 4096 bf16 (C = 1), four at once 86 instead of 82 at 4096 x 16384 (C = 4)
    constexpr int G = C <= 2 ? C : 1;
    float h[C][8], ss = 0.f;
#pragma unroll
    for (int c0 = 0; c0 < C; c0 += G) {
      Chunk<XT> q[G];
      Chunk<RT> o[G];
#pragma unroll
      for (int c = 0; c < G; ++c) {
        const int at = ((c0 + c) * (int)blockDim.x + (int)threadIdx.x) * 8;
        if (at < j.H) {
          q[c].template load<(S >= kReadOnce)>(x, at);
          if (j.residual) o[c].template load<(S >= kReadOnce)>((const char*)j.residual + row_bytes<RT>(t, j.res_pitch), at);
        }
      }
#pragma unroll
      for (int c = 0; c < G; ++c) {
        float* hc = h[c0 + c];
#pragma unroll
        for (int e = 0; e < 8; ++e) hc[e] = 0.f;
        if (((c0 + c) * (int)blockDim.x + (int)threadIdx.x) * 8 >= j.H) continue;
        q[c].get(hc);
        if (j.residual) {
          float f[8];
          o[c].get(f);
#pragma unroll
          for (int e = 0; e < 8; ++e) hc[e] += f[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(hc[e], hc[e], ss);
      }
    }
    const float r = 1.f / sqrtf(group_sum(ss, s_a[par]) / (float)j.H + j.eps);
    if (j.rstd && threadIdx.x == 0) j.rstd[t] = r;
    char* out = (char*)j.out + row_bytes<OT>(t, j.out_pitch);
    const bool plain = OT == MOE_FP8_E4M3 && r >= 0x1p-40f && r <= 0x1p40f;
    const float pre = plain ? 1.f : r;
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * (int)blockDim.x + (int)threadIdx.x) * 8;
      if (at < j.H) {
        if (j.residual_out) st8<RT, S == kThrough>((char*)j.residual_out + row_bytes<RT>(t, j.res_out_pitch), at, h[c]);
        float g[8];
        gamma8(j.gamma, j.gamma_f32, at, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] *= pre * g[e];
        if constexpr (OT != MOE_FP8_E4M3) st8<OT, S == kThrough>(out, at, h[c]);
      }
      if constexpr (OT == MOE_FP8_E4M3) {
        float a = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(h[c][e]));
        amax = fmaxf(amax, a);
        if (j.group_lanes) {
          const Coding coded = coding_of(run_max(a, j.group_lanes), r, plain);
          if (at < j.H) {
            coded(h[c]);
            st8<OT, S == kThrough>(out, at, h[c]);
            const int lane = threadIdx.x & (j.group_lanes - 1);
            if (lane == 0) j.out_scale[(int64_t)t * j.groups + at / (j.group_lanes * 8)] = coded.scale;
          }
        }
      }
    }
    if constexpr (OT == MOE_FP8_E4M3) {
      if (!j.group_lanes) {
        const Coding coded = coding_of(group_max(amax, s_b[par]), r, plain);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int at = (c * (int)blockDim.x + (int)threadIdx.x) * 8;
          if (at < j.H) {
            coded(h[c]);
            st8<OT, S == kThrough>(out, at, h[c]);
          }
        }
        if (threadIdx.x == 0) j.out_scale[t] = coded.scale;
      }
    }
    par ^= 1;
  }
}

struct NormBackJob {
  int T, H, gamma_f32, row_threads;
  const void *dout, *h, *gamma, *dres;
  int64_t dout_pitch, h_pitch, dres_pitch, dx_pitch, dresidual_pitch;
  const float* rstd;
  void *dx, *dresidual;
  float* part;  // [gridDim.x][H] sums over this workgroup's tokens, or NULL
};

// With r = rstd, g = dout gamma:
//   dh = r g - h r^2 <r g, h> / H + dres,  dgamma = sum_t (dout r) h
// so that dout r is formed once and serves both.  A workgroup takes the rows blockIdx, blockIdx +
// gridDim, ... , the next row's loads in flight, and keeps its share of dgamma in registers.
// 8191 x 2880 bf16, 189 MB: 34 us (5.5 TB/s) and 4.6 us for the sum of the 512 shares; the arithmetic
// is half of that time (36 us with h r and gamma formed anew for each row).  256 workgroups 46 us in
// all, 512 40 before that change, 1024 39 with twice the workspace; a second row in flight changes nothing.
// MANY (C = 1): several rows at a time in a workgroup, row_threads threads to a row, so that short rows
// still fill the waves.  16384 rows of 64 columns 24 us one at a time, 9.7 with eight; of 512 25 and
// 15.5, of 1024 37 and 27 (four), of 1536 42.5 and 39.4 (two), but of 2048 48.5 and 49.7 (two).
template <int DT, int HT, int C, int S, bool MANY>
__global__ __launch_bounds__(kNormT) void norm_backward_kernel(NormBackJob j) {
  __shared__ float s_a[2][kNormWaves];
  __shared__ __attribute__((aligned(16))) float s_share[MANY ? kNormT * 8 : 4];
  static_assert(!MANY || C == 1, "");
  const int tpr = MANY ? j.row_threads : (int)blockDim.x;  // threads to a row
  const int sub = MANY ? (int)threadIdx.x / tpr : 0, lt = (int)threadIdx.x - sub * tpr;
  const int many = MANY ? (int)blockDim.x / tpr : 1, step = (int)gridDim.x * many;
  float dg[C][8];
  Chunk<DT> nd[C];  // the next row on its way
  constexpr bool kDresAhead = C <= 2 || HT == MOE_BF16;  // four fp32 chunks more would spill
  Chunk<HT> nh[C], ns[kDresAhead ? C : 1];
  float nr = 0.f;
  auto fetch = [&](int t) {
    const char* dout = (const char*)j.dout + row_bytes<DT>(t, j.dout_pitch);
    const char* hr = (const char*)j.h + row_bytes<HT>(t, j.h_pitch);
    const char* dres = (const char*)j.dres + row_bytes<HT>(t, j.dres_pitch);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * tpr + lt) * 8;
      if (at < j.H) {
        nd[c].template load<(S >= kReadOnce)>(dout, at);
        nh[c].template load<(S >= kReadOnce)>(hr, at);
        if constexpr (kDresAhead) {
          if (j.dres) ns[c].template load<(S >= kReadOnce)>(dres, at);
        }
      }
    }
    nr = j.rstd[t];
  };
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[c][e] = 0.f;
  constexpr bool kGammaHeld = C == 1;  // two chunks' took 87 instead of 83 us at 8192 x 7168 bf16
  float gm[kGammaHeld ? C : 1][8];
  if constexpr (kGammaHeld) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * tpr + lt) * 8;
      if (at < j.H) gamma8(j.gamma, j.gamma_f32, at, gm[c]);
    }
  }
  int par = 0;
  if ((int)blockIdx.x * many + sub < j.T) fetch(blockIdx.x * many + sub);
  // every thread takes as many turns as the workgroup's first row does
  for (int t0 = blockIdx.x * many; t0 < j.T; t0 += step, par ^= 1) {
    const int t = t0 + sub;
    const bool there = !MANY || t < j.T;
    const float r = nr;
    float h[C][8], rg[C][8], dot = 0.f;
    Chunk<HT> ds[kDresAhead ? C : 1];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * tpr + lt) * 8;
      if (there && at < j.H) {
        nd[c].get(rg[c]);
        nh[c].get(h[c]);
        if constexpr (kDresAhead) ds[c] = ns[c];
        if constexpr (!kGammaHeld) gamma8(j.gamma, j.gamma_f32, at, gm[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = rg[c][e] * r;
          dg[c][e] = fmaf(a, h[c][e], dg[c][e]);
          rg[c][e] = a * gm[kGammaHeld ? c : 0][e];
          dot = fmaf(rg[c][e], h[c][e], dot);
        }
      }
    }
    if (t + step < j.T) fetch(t + step);
    const float back = rows_sum<MANY>(dot, s_a[par], sub, tpr) / (float)j.H * (r * r);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * tpr + lt) * 8;
      if (there && at < j.H) {
        float d[8];
        if (j.dres) {
          if constexpr (kDresAhead) {
            ds[c].get(d);
          } else {
            ds[0].template load<(S >= kReadOnce)>((const char*)j.dres + row_bytes<HT>(t, j.dres_pitch), at);
            ds[0].get(d);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = fmaf(-h[c][e], back, rg[c][e] + d[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = fmaf(-h[c][e], back, rg[c][e]);
        }
        if (j.dx) st8<DT, S == kThrough>((char*)j.dx + row_bytes<DT>(t, j.dx_pitch), at, d);
        if (j.dresidual) st8<HT, S == kThrough>((char*)j.dresidual + row_bytes<HT>(t, j.dresidual_pitch), at, d);
      }
    }
  }
  if constexpr (MANY) {  // the rows' shares of dgamma together, in the order of the rows
    if (!j.part) return;
    if (lt * 8 < j.H) st8<MOE_F32>(s_share + sub * j.H, lt * 8, dg[0]);
    __syncthreads();
    for (int col = threadIdx.x; col < j.H; col += blockDim.x) {
      float sum = 0.f;
      for (int q = 0; q < many; ++q) sum += s_share[q * j.H + col];
      j.part[(int64_t)blockIdx.x * j.H + col] = sum;
    }
    return;
  }
  if (j.part) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * tpr + lt) * 8;
      if (at < j.H) st8<MOE_F32>(j.part + (int64_t)blockIdx.x * j.H, at, dg[c]);
    }
  }
}

// dgamma[col] = sum of the partial rows: 64 columns per workgroup, four to a thread, the rows dealt
// to 64 groups of threads.
__global__ __launch_bounds__(1024) void norm_dgamma_kernel(const float* __restrict__ part, int rows, int H,
                                                           float* __restrict__ dgamma) {
  __shared__ float s[64][65];
  const int cx = (threadIdx.x & 15) * 4, ry = threadIdx.x >> 4, col = blockIdx.x * 64 + cx;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if (col < H) {
#pragma unroll 8
    for (int r = ry; r < rows; r += 64) sum += *reinterpret_cast<const f32x4*>(part + (int64_t)r * H + col);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) s[ry][cx + k] = sum[k];
  __syncthreads();
  const int c = threadIdx.x >> 4, l = threadIdx.x & 15;  // 16 lanes add a column's 64 groups
  const float all = sum16((s[l][c] + s[l + 16][c]) + (s[l + 32][c] + s[l + 48][c]));
  if (l == 0 && blockIdx.x * 64 + c < H) dgamma[blockIdx.x * 64 + c] = all;
}

// Threads for a row of H and the chunks that each holds (1, 2 or 4): the fewest passes of at most
// 512 lanes, the lanes spread evenly.
struct RowShape {
  unsigned threads;
  int chunks;
};
static RowShape row_shape(int H) {
  const int chunks = H / 8, c = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : 4, per = (chunks + c - 1) / c;
  return {(unsigned)((per + 63) / 64 * 64), c};
}

static bool norm_pitch_ok(int64_t pitch, int32_t H) { return pitch >= H && pitch <= ((int64_t)1 << 32); }
static bool norm_types_ok(int a, int b) {
  return (a == MOE_BF16 && (b == MOE_BF16 || b == MOE_F32)) || (a == MOE_F32 && b == MOE_F32);
}

template <int XT, int RT, int OT, int C>
static int norm_launch(const NormJob& j, unsigned threads, hipStream_t stream) {
  const int rs = dtype_size(RT) * ((j.residual != nullptr) + (j.residual_out != nullptr));
  const unsigned grid = grid_of(j.T);
  switch (stream_kind((int64_t)j.T * j.H * (dtype_size(XT) + dtype_size(OT) + rs))) {
    case kThrough: return launch(norm_kernel<XT, RT, OT, C, kThrough>, grid, threads, stream, j);
    case kReadOnce: return launch(norm_kernel<XT, RT, OT, C, kReadOnce>, grid, threads, stream, j);
    default: return launch(norm_kernel<XT, RT, OT, C, kNear>, grid, threads, stream, j);
  }
}
template <int XT, int RT, int OT>
static int norm_by_width(const NormJob& j, hipStream_t stream) {
  const RowShape r = row_shape(j.H);
  if (r.chunks == 1) return norm_launch<XT, RT, OT, 1>(j, r.threads, stream);
  if (r.chunks == 2) return norm_launch<XT, RT, OT, 2>(j, r.threads, stream);
  return norm_launch<XT, RT, OT, 4>(j, r.threads, stream);
}

template <int XT, int RT>
static int norm_by_out(const NormJob& j, int out, hipStream_t stream) {
  if (out == MOE_F32) return norm_by_width<XT, RT, MOE_F32>(j, stream);
  if (out == MOE_BF16) return norm_by_width<XT, RT, MOE_BF16>(j, stream);
  return norm_by_width<XT, RT, MOE_FP8_E4M3>(j, stream);
}

template <int DT, int HT, int C, bool MANY>
static int norm_backward_launch(const NormBackJob& j, unsigned grid, unsigned threads, hipStream_t stream) {
  const int hs = dtype_size(HT) * (1 + (j.dres != nullptr) + (j.dresidual != nullptr));
  switch (stream_kind((int64_t)j.T * j.H * (dtype_size(DT) * (1 + (j.dx != nullptr)) + hs))) {
    case kThrough: return launch(norm_backward_kernel<DT, HT, C, kThrough, MANY>, grid, threads, stream, j);
    case kReadOnce: return launch(norm_backward_kernel<DT, HT, C, kReadOnce, MANY>, grid, threads, stream, j);
    default: return launch(norm_backward_kernel<DT, HT, C, kNear, MANY>, grid, threads, stream, j);
  }
}

// rows that a workgroup of the gradient takes at a time: one up to kPartials rows, which then have a
// workgroup each, and from 1537 columns on
static int norm_backward_many(int T, int H) {
  const RowShape r = row_shape(H);
  return r.threads > 192 || r.chunks > 1 || T <= kPartials ? 1 : kNormT / (int)r.threads;
}

template <int DT, int HT>
static int norm_backward_by_width(NormBackJob& j, unsigned grid, hipStream_t stream) {
  const RowShape r = row_shape(j.H);
  const int many = norm_backward_many(j.T, j.H);
  j.row_threads = (int)r.threads;
  if (many > 1) return norm_backward_launch<DT, HT, 1, true>(j, grid, r.threads * many, stream);
  if (r.chunks == 1) return norm_backward_launch<DT, HT, 1, false>(j, grid, r.threads, stream);
  if (r.chunks == 2) return norm_backward_launch<DT, HT, 2, false>(j, grid, r.threads, stream);
  return norm_backward_launch<DT, HT, 4, false>(j, grid, r.threads, stream);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_residual_norm(const moe_residual_norm_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  if (a->T < 0 || a->T > (1 << 24) || a->H < 1 || a->H > kNormH || !(a->eps >= 0.f)) return MOE_EINVAL_SIZE;
  const bool fp8 = a->out_dtype == MOE_FP8_E4M3;
  if (!norm_types_ok(a->x_dtype, a->res_dtype) || (a->gamma_dtype != MOE_F32 && a->gamma_dtype != MOE_BF16) ||
      (a->out_dtype != MOE_F32 && a->out_dtype != MOE_BF16 && !fp8))
    return MOE_EINVAL_DTYPE;
  if (a->H % 8) return MOE_EINVAL_SHAPE;
  if (!norm_pitch_ok(a->x_pitch, a->H) || !norm_pitch_ok(a->out_pitch, a->H) ||
      (a->residual && !norm_pitch_ok(a->res_pitch, a->H)) ||
      (a->residual_out && !norm_pitch_ok(a->res_out_pitch, a->H)))
    return MOE_EINVAL_SIZE;
  if (fp8 && a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128) return MOE_EINVAL_SIZE;
  if (!a->row_list != !a->row_count || (a->row_list && !a->err)) return MOE_EINVAL_NULL;
  if (a->T == 0) return MOE_OK;
  if (!a->x || !a->gamma || !a->out || (fp8 && !a->out_scale)) return MOE_EINVAL_NULL;
  const int xs = dtype_size(a->x_dtype), rs = dtype_size(a->res_dtype), os = dtype_size(a->out_dtype);
  if (!aligned_rows(a->x, a->x_pitch, xs, 16) || !aligned16(a->gamma) ||
      !aligned_rows(a->out, a->out_pitch, os, chunk_align(a->out_dtype)) ||
      (a->residual && !aligned_rows(a->residual, a->res_pitch, rs, 16)) ||
      (a->residual_out && !aligned_rows(a->residual_out, a->res_out_pitch, rs, 16)))
    return MOE_EINVAL_ALIGN;
  NormJob j;
  j.T = a->T; j.H = a->H; j.eps = a->eps; j.gamma_f32 = a->gamma_dtype == MOE_F32;
  j.group_lanes = fp8 ? a->group / 8 : 0;
  j.groups = fp8 && a->group ? (a->H + a->group - 1) / a->group : 1;
  j.x = a->x; j.residual = a->residual; j.gamma = a->gamma; j.out = a->out; j.residual_out = a->residual_out;
  j.x_pitch = a->x_pitch; j.res_pitch = a->res_pitch; j.out_pitch = a->out_pitch; j.res_out_pitch = a->res_out_pitch;
  j.out_scale = a->out_scale; j.rstd = a->rstd; j.row_list = a->row_list; j.row_count = a->row_count; j.err = a->err;
  if (a->x_dtype == MOE_F32) return norm_by_out<MOE_F32, MOE_F32>(j, a->out_dtype, stream);
  if (a->res_dtype == MOE_F32) return norm_by_out<MOE_BF16, MOE_F32>(j, a->out_dtype, stream);
  return norm_by_out<MOE_BF16, MOE_BF16>(j, a->out_dtype, stream);
}

extern "C" size_t moe_residual_norm_backward_workspace_size(int32_t H) {
  return H > 0 ? (size_t)kPartials * (size_t)H * sizeof(float) : 0;
}

extern "C" int moe_residual_norm_backward(const moe_residual_norm_backward_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  if (a->T < 0 || a->T > (1 << 24) || a->H < 1 || a->H > kNormH) return MOE_EINVAL_SIZE;
  if (!norm_types_ok(a->dtype, a->h_dtype) || (a->gamma_dtype != MOE_F32 && a->gamma_dtype != MOE_BF16))
    return MOE_EINVAL_DTYPE;
  if (a->H % 8) return MOE_EINVAL_SHAPE;
  if (!norm_pitch_ok(a->dout_pitch, a->H) || !norm_pitch_ok(a->h_pitch, a->H) ||
      (a->dres && !norm_pitch_ok(a->dres_pitch, a->H)) || (a->dx && !norm_pitch_ok(a->dx_pitch, a->H)) ||
      (a->dresidual && !norm_pitch_ok(a->dresidual_pitch, a->H)))
    return MOE_EINVAL_SIZE;
  if (a->T > 0) {
    if (!a->dx && !a->dresidual && !a->dgamma) return MOE_EINVAL_NULL;
    if (!a->dout || !a->h || !a->gamma || !a->rstd) return MOE_EINVAL_NULL;
    const int ds = dtype_size(a->dtype), hs = dtype_size(a->h_dtype);
    if (!aligned_rows(a->dout, a->dout_pitch, ds, 16) || !aligned_rows(a->h, a->h_pitch, hs, 16) ||
        !aligned16(a->gamma) || (a->dres && !aligned_rows(a->dres, a->dres_pitch, hs, 16)) ||
        (a->dx && !aligned_rows(a->dx, a->dx_pitch, ds, 16)) ||
        (a->dresidual && !aligned_rows(a->dresidual, a->dresidual_pitch, hs, 16)))
      return MOE_EINVAL_ALIGN;
    if (a->dgamma) {
      if (!a->workspace || a->workspace_bytes < moe_residual_norm_backward_workspace_size(a->H)) return MOE_EWORKSPACE;
      if (!aligned16(a->workspace)) return MOE_EINVAL_ALIGN;
    }
  }
  const int many = norm_backward_many(a->T, a->H), units = (a->T + many - 1) / many;
  const unsigned grid = (unsigned)(units < kPartials ? units : kPartials);
  if (a->T > 0) {
    NormBackJob j;
    j.T = a->T; j.H = a->H; j.gamma_f32 = a->gamma_dtype == MOE_F32;
    j.dout = a->dout; j.h = a->h; j.gamma = a->gamma; j.dres = a->dres;
    j.dout_pitch = a->dout_pitch; j.h_pitch = a->h_pitch; j.dres_pitch = a->dres_pitch; j.dx_pitch = a->dx_pitch;
    j.dresidual_pitch = a->dresidual_pitch;
    j.rstd = a->rstd; j.dx = a->dx; j.dresidual = a->dresidual;
    j.part = a->dgamma ? (float*)a->workspace : nullptr;
    int rc;
    if (a->dtype == MOE_F32) rc = norm_backward_by_width<MOE_F32, MOE_F32>(j, grid, stream);
    else if (a->h_dtype == MOE_F32) rc = norm_backward_by_width<MOE_BF16, MOE_F32>(j, grid, stream);
    else rc = norm_backward_by_width<MOE_BF16, MOE_BF16>(j, grid, stream);
    if (rc != MOE_OK) return rc;
  }
  if (!a->dgamma) return MOE_OK;
  return launch(norm_dgamma_kernel, (unsigned)((a->H + 63) / 64), 1024, stream, (const float*)a->workspace, (int)grid,
                a->H, a->dgamma);
}
