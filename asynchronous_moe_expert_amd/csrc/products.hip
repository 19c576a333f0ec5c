// moe_expert_matmul, moe_expert_matmul_backward: the products of each expert's rows with its row-major
// weights, in either direction, and the weights' gradient.
#include <atomic>

#include "products.hpp"

namespace moe {

// ------------------------------------------------------------------------------------------------ fp32
// S x S tiles by v_mfma_f32_16x16x4_f32, a quarter to each of four waves; the next 32 k are on their way to registers
// while those in LDS are multiplied.  LDS rows are 32 k, 36 apart, so that four neighbouring ones begin in different
// banks.  Lane l of a wave holds k = 4 (l / 16) + i in its i-th step of 16 k: which k a step takes does not matter as
// long as both operands agree.  S = 128 where that makes two tiles for every CU, 64 otherwise.  Forward, us as 64 / 128:
// 8 experts of 64 rows, 1024 x 1024: 33 / 84; 16 of 256: 88 / 89; 32 of 512: 332 / 314 (109 TFLOP/s); 1 of 4096 rows,
// 4096 x 4096: 1226 / 1119 (123 of the 154 TFLOP/s that a library product reaches).  The matrix unit bounds the large
// ones, the latency of one tile's k steps the small ones.  An element is one running sum over D: off by 5.7e-7 of the
// outputs' norm at D = 1024 and 1.1e-6 at 4096, as a library product's is with many rows; with few (40), where that one
// splits D, it has half.
constexpr int kSK = 32, kSLd = 36;

template <int MODE, int S>
__global__ __launch_bounds__(256) void product_f32_kernel(ProductJob j) {
  __shared__ __attribute__((aligned(16))) float sp[S * kSLd], sq[S * kSLd];
  constexpr int T = S / 32, C = S / 64;  // 16 x 16 tiles of a wave's edge; chunks of an operand to a thread
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, wp = (wv >> 1) * (S / 2), wq = (wv & 1) * (S / 2);
  const int Q = MODE == kWeightsGrad ? j.D : j.N, ct = (Q + S - 1) / S;
  const int rt = (j.N + S - 1) / S;  // weights' gradient
  const RowTiles<S> all(j, lane);
  const uint32_t total = (uint32_t)(MODE == kWeightsGrad ? j.E * rt : all.total()) * ct;
  for (uint32_t u = blockIdx.x; u < total; u += gridDim.x) {
    int e, p0, pend, k0 = 0, kend = j.D, q0;
    if constexpr (MODE == kWeightsGrad) {
      const int b = u / ct;
      e = b / rt;
      p0 = (b - e * rt) * S;
      pend = j.N;
      q0 = (u - b * ct) * S;
      expert_rows(j, e, k0, kend);
    } else {
      int base, n;
      all.find(u, ct, e, base, n);
      expert_rows(j, e, p0, pend);
      const int b = u / ct;
      p0 += (b - base) * S;
      q0 = (u - b * ct) * S;
    }
    // operands along k: a thread's rows are tid / 4 + 64 c, 8 k each; across k: its k is tid / 8, 8 columns + 64 c
    const int ar = tid >> 2, ak = (tid & 3) * 8, bk = tid >> 3, bc = (tid & 7) * 8;
    const float *prow[C] = {}, *w = nullptr;
    if constexpr (MODE != kWeightsGrad) {
      w = (const float*)j.w + e * j.w_stride;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int row = p0 + ar + 64 * c;
        if (row >= pend) continue;
        int64_t slot = row;
        if (j.row_slot) {
          slot = j.row_slot[row];
          if (slot < 0 || slot >= j.x_rows) {
            atomicOr(j.err, MOE_ERR_SLOT_RANGE);
            continue;
          }
        }
        prow[c] = (const float*)j.x + slot * j.x_pitch;
      }
    }
    float f[C][8], g[C][8];
    auto fetch = [&](int k) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[c][i] = g[c][i] = 0.f;
        Chunk<MOE_F32> x;
        if constexpr (MODE == kWeightsGrad) {
          if (k + bk < kend && p0 + bc + 64 * c < pend) {
            x.load((const float*)j.dout + (k + bk) * j.dout_pitch, p0 + bc + 64 * c);
            x.get(f[c]);
          }
          if (k + bk < kend && q0 + bc + 64 * c < Q) {
            x.load((const float*)j.x + (k + bk) * j.x_pitch, q0 + bc + 64 * c);
            x.get(g[c]);
          }
        } else {
          if (prow[c] && k + ak < kend) {
            x.load(prow[c], k + ak);
            x.get(f[c]);
          }
          if constexpr (MODE == kForward) {
            if (q0 + ar + 64 * c < Q && k + ak < kend) {
              x.load(w + (q0 + ar + 64 * c) * j.w_pitch, k + ak);
              x.get(g[c]);
            }
          } else if (k + bk < kend && q0 + bc + 64 * c < Q) {
            x.load(w + (k + bk) * j.w_pitch, q0 + bc + 64 * c);
            x.get(g[c]);
          }
        }
      }
    };
    f32x4 acc[T][T];
#pragma unroll
    for (int a = 0; a < T; ++a)
#pragma unroll
      for (int c = 0; c < T; ++c) acc[a][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    fetch(k0);
    for (int k = k0; k < kend; k += kSK) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if constexpr (MODE == kWeightsGrad) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sp[(bc + 64 * c + i) * kSLd + bk] = f[c][i];
        } else {
          float* o = sp + (ar + 64 * c) * kSLd + ak;
          *reinterpret_cast<f32x4*>(o) = f32x4{f[c][0], f[c][1], f[c][2], f[c][3]};
          *reinterpret_cast<f32x4*>(o + 4) = f32x4{f[c][4], f[c][5], f[c][6], f[c][7]};
        }
        if constexpr (MODE == kForward) {
          float* o = sq + (ar + 64 * c) * kSLd + ak;
          *reinterpret_cast<f32x4*>(o) = f32x4{g[c][0], g[c][1], g[c][2], g[c][3]};
          *reinterpret_cast<f32x4*>(o + 4) = f32x4{g[c][4], g[c][5], g[c][6], g[c][7]};
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) sq[(bc + 64 * c + i) * kSLd + bk] = g[c][i];
        }
      }
      __syncthreads();
      fetch(k + kSK);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        f32x4 p[T], q[T];
#pragma unroll
        for (int a = 0; a < T; ++a) {
          p[a] = *reinterpret_cast<const f32x4*>(sp + (wp + a * 16 + (lane & 15)) * kSLd + s * 16 + (lane >> 4) * 4);
          q[a] = *reinterpret_cast<const f32x4*>(sq + (wq + a * 16 + (lane & 15)) * kSLd + s * 16 + (lane >> 4) * 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int a = 0; a < T; ++a)
#pragma unroll
            for (int c = 0; c < T; ++c)
              acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(q[c][i], p[a][i], acc[a][c], 0, 0, 0);
      }
    }
    if (MODE == kWeightsGrad && k0 == kend && j.accumulate) continue;  // no rows: what was there stays
#pragma unroll
    for (int a = 0; a < T; ++a) {
      const int p = p0 + wp + a * 16 + (lane & 15);
      if (p >= pend) continue;
#pragma unroll
      for (int c = 0; c < T; ++c) {
        const int q = q0 + wq + c * 16 + (lane >> 4) * 4;
        if (q < Q) put4(j, (MODE == kWeightsGrad ? e * j.out_stride : 0) + p * j.out_pitch + q, acc[a][c]);
      }
    }
  }
}

// ------------------------------------------------------------------------------------ checks and dispatch
constexpr int64_t kReach = (int64_t)1 << 36;  // bytes of x, or of an expert's matrix
constexpr int64_t kPitch = (int64_t)1 << 24;  // bytes between its rows

// The current device's compute units, looked up once per device (0: none).
static int compute_units() {
  static std::atomic<int> known[64];
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 0;
  if (dev < 64 && (cus = known[dev].load(std::memory_order_relaxed)) > 0) return cus;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
  if (dev < 64) known[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

template <int MODE>
static int run_f32(const ProductJob& j, int cus, hipStream_t stream) {
  const auto tiles = [&](int s) {  // as many as there can be: under 2^29 with n <= 2^24 and sides <= 2^16
    const int64_t ct = ((MODE == kWeightsGrad ? j.D : j.N) + s - 1) / s;
    return ct * (MODE == kWeightsGrad ? (int64_t)j.E * ((j.N + s - 1) / s) : j.n / s + (j.n < j.E ? j.n : j.E));
  };
  if (tiles(128) >= 2 * cus) return launch(product_f32_kernel<MODE, 128>, grid_of(tiles(128)), 256u, stream, j);
  return launch(product_f32_kernel<MODE, 64>, grid_of(tiles(64)), 256u, stream, j);
}

// Up to 64 rows of an expert on average a product is a pass over its weights.  32 experts, 4096 x 4096 bf16, us as
// tiles / narrow, forward: 4 rows each 187 / 159, 32 187 / 164, 64 193 / 177, 96 211 / 246, 128 216 / 259.  The rows'
// gradient: 185 / 188, 187 / 195, 190 / 204, 198 / 261, 207 / 277; but where the tiles leave CUs idle the narrow ones
// win: 8 experts, 5760 x 2880, 4 rows each 69 / 44, 32 69 / 44, 64 73 / 58; one of 4096 x 4096, 49 / 31, 50 / 32, 50 / 41.
// It goes by the same rule: a third saved there for at most 7% lost.
template <int MODE>
static int run_product(const ProductJob& j, int dtype, hipStream_t stream) {
  const int cus = compute_units();
  if (!cus) return MOE_ELAUNCH;
  if (dtype == MOE_F32) return run_f32<MODE>(j, cus, stream);
  if (MODE != kWeightsGrad && j.n <= 64 * (int64_t)j.E) return run_narrow(j, dtype, MODE, cus, stream);
  return run_tiles(j, dtype, MODE, cus, stream);
}

// a matrix of `rows` rows of `cols` elements, one of several `stride` apart
static int matrix_status(const void* p, int64_t rows, int64_t cols, int64_t pitch, int64_t stride, int many, int es) {
  if (pitch < cols || pitch > kPitch / es || rows * pitch * es > kReach) return MOE_EINVAL_SIZE;
  if (many > 1 && (stride < (rows - 1) * pitch + cols || stride > kReach)) return MOE_EINVAL_SIZE;
  if (!aligned_rows(p, pitch, es, 16) || (many > 1 && (stride * es) % 16)) return MOE_EINVAL_ALIGN;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_expert_matmul(const moe_expert_matmul_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  if (a->n < 0 || a->n > (1 << 24) || a->E_loc < 1 || a->E_loc > 256 || a->N < 1 || a->N > kHMaxRows || a->D < 1 ||
      a->D > kHMaxRows || (a->w_transposed != 0 && a->w_transposed != 1))
    return MOE_EINVAL_SIZE;
  const bool fp8 = a->dtype == MOE_FP8_E4M3;
  if ((a->dtype != MOE_F32 && a->dtype != MOE_BF16 && !fp8) || (a->out_dtype != MOE_F32 && a->out_dtype != MOE_BF16) ||
      (a->dtype == MOE_F32 && a->out_dtype != MOE_F32) || (fp8 && a->w_transposed))
    return MOE_EINVAL_DTYPE;
  if (a->N % 8 || a->D % (fp8 ? 16 : 8)) return MOE_EINVAL_SHAPE;
  const int64_t x_rows = a->row_slot ? a->x_rows : a->n;
  if (x_rows < 0 || x_rows > (1 << 24) || a->x_pitch < a->D || a->out_pitch < a->N) return MOE_EINVAL_SIZE;
  if (a->n == 0) return MOE_OK;
  if (!a->offsets || !a->x || !a->w || !a->out || (fp8 && (!a->x_scale || !a->w_scale)) || (a->row_slot && !a->err))
    return MOE_EINVAL_NULL;
  const int es = dtype_size(a->dtype);
  int rc = matrix_status(a->x, x_rows, a->D, a->x_pitch, 0, 1, es);
  if (rc != MOE_OK) return rc;
  rc = matrix_status(a->w, a->w_transposed ? a->D : a->N, a->w_transposed ? a->N : a->D, a->w_pitch, a->w_stride,
                     a->E_loc, es);
  if (rc != MOE_OK) return rc;
  if (!aligned_rows(a->out, a->out_pitch, dtype_size(a->out_dtype), 16)) return MOE_EINVAL_ALIGN;
  ProductJob j = {};
  j.n = a->n; j.E = a->E_loc; j.N = a->N; j.D = a->D; j.offsets = a->offsets;
  j.x = a->x; j.x_rows = x_rows; j.x_pitch = a->x_pitch; j.row_slot = a->row_slot; j.x_scale = a->x_scale;
  j.w = a->w; j.w_pitch = a->w_pitch; j.w_stride = a->E_loc > 1 ? a->w_stride : 0; j.w_scale = a->w_scale;
  j.out = a->out; j.out_pitch = a->out_pitch; j.out_f32 = a->out_dtype == MOE_F32; j.err = a->err;
  return a->w_transposed ? run_product<kRowsGrad>(j, a->dtype, stream) : run_product<kForward>(j, a->dtype, stream);
}

extern "C" int moe_expert_matmul_backward(const moe_expert_matmul_backward_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  if (a->n < 0 || a->n > (1 << 24) || a->E_loc < 1 || a->E_loc > 256 || a->N < 1 || a->N > kHMaxRows || a->D < 1 ||
      a->D > kHMaxRows || (a->accumulate != 0 && a->accumulate != 1))
    return MOE_EINVAL_SIZE;
  if ((a->dtype != MOE_F32 && a->dtype != MOE_BF16) || (a->dw_dtype != MOE_F32 && a->dw_dtype != MOE_BF16) ||
      (a->dtype == MOE_F32 && a->dw_dtype != MOE_F32))
    return MOE_EINVAL_DTYPE;
  if (a->N % 8 || a->D % 8) return MOE_EINVAL_SHAPE;
  if (a->dout_pitch < a->N || a->x_pitch < a->D) return MOE_EINVAL_SIZE;
  if (!a->offsets || !a->dw || (a->n > 0 && (!a->dout || !a->x))) return MOE_EINVAL_NULL;
  const int es = dtype_size(a->dtype);
  int rc = matrix_status(a->dw, a->N, a->D, a->dw_pitch, a->dw_stride, a->E_loc, dtype_size(a->dw_dtype));
  if (rc != MOE_OK) return rc;
  if ((rc = matrix_status(a->dout, a->n, a->N, a->dout_pitch, 0, 1, es)) != MOE_OK) return rc;
  if ((rc = matrix_status(a->x, a->n, a->D, a->x_pitch, 0, 1, es)) != MOE_OK) return rc;
  ProductJob j = {};
  j.n = a->n; j.E = a->E_loc; j.N = a->N; j.D = a->D; j.offsets = a->offsets;
  j.x = a->x; j.x_rows = a->n; j.x_pitch = a->x_pitch; j.dout = a->dout; j.dout_pitch = a->dout_pitch;
  j.out = a->dw; j.out_pitch = a->dw_pitch; j.out_stride = a->E_loc > 1 ? a->dw_stride : 0;
  j.out_f32 = a->dw_dtype == MOE_F32; j.accumulate = a->accumulate;
  // fp32 ones of 96 MiB and more, which no cache would keep (both sides' times are in product_tiles.hip)
  j.through = j.out_f32 && (int64_t)a->E_loc * a->N * a->D * 4 >= (96ll << 20);
  return run_product<kWeightsGrad>(j, a->dtype, stream);
}
