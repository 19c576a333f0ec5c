// moe_expert_matmul, moe_expert_matmul_backward: the products of each expert's rows with its row-major
// weights, in either direction, and the weights' gradient.
#include <atomic>

#include "products.hpp"

namespace moe {

// ------------------------------------------------------------------------------------ any type, any size
// 64 x 64 tiles in fp32: elements are widened (8-bit ones scaled) into LDS rows of 32 k, 36 apart so that
// rows four apart begin in the same bank only every eighth, and multiplied by v_mfma_f32_16x16x4_f32.  Lane l
// of a wave holds k = 4 (l / 16) + i in its i-th step: which k a step takes does not matter as long as both
// operands agree.
constexpr int kS = 64, kSK = 32, kSLd = 36;

template <int DT, int MODE>
__global__ __launch_bounds__(256) void product_kernel(ProductJob j) {
  __shared__ __attribute__((aligned(16))) float sp[kS * kSLd], sq[kS * kSLd];
  constexpr int es = esize<DT>();
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, wp = (wv >> 1) * 32, wq = (wv & 1) * 32;
  const int Q = MODE == kWeightsGrad ? j.D : j.N;
  const int ct = (Q + kS - 1) / kS;
  int e, p0, pend, k0 = 0, kend;
  const int q0 = (int)(blockIdx.x % ct) * kS;
  if constexpr (MODE == kWeightsGrad) {
    const int rt = (j.N + kS - 1) / kS, b = blockIdx.x / ct;
    e = b / rt;
    p0 = (b - e * rt) * kS;
    pend = j.N;
    expert_rows(j, e, k0, kend);
  } else {
    int b = blockIdx.x / ct;
    kend = j.D;
    for (e = 0; e < j.E; ++e) {
      expert_rows(j, e, p0, pend);
      const int t = (pend - p0 + kS - 1) / kS;
      if (b < t) break;
      b -= t;
    }
    if (e == j.E) return;
    p0 += b * kS;
  }
  // the thread's row (along k) or k and columns (across k) of each operand
  const int ar = tid >> 2, ak = (tid & 3) * 8, bk = tid >> 3, bc = (tid & 7) * 8;
  const char* prow = nullptr;
  int64_t pslot = p0 + ar;
  if constexpr (MODE != kWeightsGrad) {
    if (p0 + ar < pend) {
      if (j.row_slot) {
        pslot = j.row_slot[p0 + ar];
        if (pslot < 0 || pslot >= j.x_rows) {
          atomicOr(j.err, MOE_ERR_SLOT_RANGE);
          pslot = -1;
        }
      }
      if (pslot >= 0) prow = (const char*)j.x + pslot * j.x_pitch * es;
    }
  }
  const int kb = (j.D + 127) / 128;
  f32x4 acc[2][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k = k0; k < kend; k += kSK) {
    float f[8], g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = g[i] = 0.f;
    Chunk<DT> c;
    if constexpr (MODE == kWeightsGrad) {
      if (k + bk < kend && p0 + bc < pend) {
        c.load((const char*)j.dout + (int64_t)(k + bk) * j.dout_pitch * es, p0 + bc);
        c.get(f);
      }
      if (k + bk < kend && q0 + bc < Q) {
        c.load((const char*)j.x + (int64_t)(k + bk) * j.x_pitch * es, q0 + bc);
        c.get(g);
      }
    } else {
      if (prow && k + ak < kend) {
        c.load(prow, k + ak);
        c.get(f);
        if constexpr (DT == MOE_FP8_E4M3) {
          const float s = j.x_scale[pslot * kb + (k + ak) / 128];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= s;
        }
      }
      const char* w = (const char*)j.w + e * j.w_stride * es;
      if constexpr (MODE == kForward) {
        if (q0 + ar < Q && k + ak < kend) {
          c.load(w + (int64_t)(q0 + ar) * j.w_pitch * es, k + ak);
          c.get(g);
          if constexpr (DT == MOE_FP8_E4M3) {
            const float s = j.w_scale[((int64_t)e * ((j.N + 127) / 128) + (q0 + ar) / 128) * kb + (k + ak) / 128];
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] *= s;
          }
        }
      } else if (k + bk < kend && q0 + bc < Q) {
        c.load(w + (int64_t)(k + bk) * j.w_pitch * es, q0 + bc);
        c.get(g);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (MODE == kWeightsGrad) sp[(bc + i) * kSLd + bk] = f[i];
      else sp[ar * kSLd + ak + i] = f[i];
      if constexpr (MODE == kForward) sq[ar * kSLd + ak + i] = g[i];
      else sq[(bc + i) * kSLd + bk] = g[i];
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f32x4 p[2], q[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        p[a] = *reinterpret_cast<const f32x4*>(sp + (wp + a * 16 + (lane & 15)) * kSLd + s * 16 + (lane >> 4) * 4);
        q[a] = *reinterpret_cast<const f32x4*>(sq + (wq + a * 16 + (lane & 15)) * kSLd + s * 16 + (lane >> 4) * 4);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(q[b][i], p[a][i], acc[a][b], 0, 0, 0);
    }
  }
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const int p = p0 + wp + a * 16 + (lane & 15);
    if (p >= pend) continue;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int q = q0 + wq + b * 16 + (lane >> 4) * 4;
      if (q >= Q) continue;
      const int64_t at = (MODE == kWeightsGrad ? e * j.out_stride : 0) + p * j.out_pitch + q;
      put4(j, at, acc[a][b]);
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

template <int DT, int MODE>
static int run_product(const ProductJob& j, hipStream_t stream) {
  if (DT != MOE_F32) {
    const bool few = MODE != kWeightsGrad && j.n <= 64 * (int64_t)j.E;
    const int cus = compute_units();
    if (!cus) return MOE_ELAUNCH;
    return few ? run_narrow(j, DT, MODE, cus, stream) : run_tiles(j, DT, MODE, cus, stream);
  }
  const int64_t ct = ((MODE == kWeightsGrad ? j.D : j.N) + kS - 1) / kS;
  const int64_t rt = MODE == kWeightsGrad ? (int64_t)j.E * ((j.N + kS - 1) / kS) : j.n / kS + (j.n < j.E ? j.n : j.E);
  if (rt * ct > (1 << 24) - 1) return MOE_EINVAL_SIZE;
  return launch(product_kernel<DT, MODE>, (unsigned)(rt * ct), 256u, stream, j);
}

// a matrix of `rows` rows of `cols` elements, one of several `stride` apart
static int matrix_status(const void* p, int64_t rows, int64_t cols, int64_t pitch, int64_t stride, int many, int es) {
  if (pitch < cols || pitch * es > kPitch || rows * pitch * es > kReach) return MOE_EINVAL_SIZE;
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
  if (fp8) return run_product<MOE_FP8_E4M3, kForward>(j, stream);
  if (a->dtype == MOE_F32)
    return a->w_transposed ? run_product<MOE_F32, kRowsGrad>(j, stream) : run_product<MOE_F32, kForward>(j, stream);
  return a->w_transposed ? run_product<MOE_BF16, kRowsGrad>(j, stream) : run_product<MOE_BF16, kForward>(j, stream);
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
  return a->dtype == MOE_F32 ? run_product<MOE_F32, kWeightsGrad>(j, stream) : run_product<MOE_BF16, kWeightsGrad>(j, stream);
}
