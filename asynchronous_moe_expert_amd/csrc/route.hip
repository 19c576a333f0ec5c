// moe_route, moe_route_backward: choice of experts and router weights from logits, and the
// logits' gradient.
//
// A token belongs to one row of 16 lanes (four tokens per wave), lane l holding the logits of
// experts l V .. l V + V - 1, V = 1, 2, 4, ... 32 the smallest that covers E.  Reductions stay
// inside the row, as DPP operands.
#include <float.h>
#include <math.h>

#include "home.hpp"

namespace moe {

constexpr int kRouteE = 512, kRouteK = 32;
constexpr int kRouteT = 256;               // threads per workgroup
constexpr int kRouteTok = kRouteT / 16;    // tokens per workgroup

struct RouteJob {
  int T, E, K, dtype, vec, score, renorm;
  int64_t pitch;
  float scale;
  const void* logits;
};

__device__ __forceinline__ float logit_at(const RouteJob& j, int64_t at) {
  return j.dtype == MOE_F32 ? ((const float*)j.logits)[at] : bf16_to_f32(((const uint16_t*)j.logits)[at]);
}

// The lane's V logits (NaN past E).  vec: rows start on 16 bytes and E is whole chunks, so that a
// chunk of 16 bytes is either all inside the row or all past it.
template <int V>
__device__ __forceinline__ void load_logits(const RouteJob& j, int t, int e0, float* l) {
  const int64_t row = (int64_t)t * j.pitch;
  if constexpr (V >= 4) {
    if (j.vec && j.dtype == MOE_F32) {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        f32x4 q = {NAN, NAN, NAN, NAN};
        if (e0 + v < j.E) q = *reinterpret_cast<const f32x4*>((const float*)j.logits + row + e0 + v);
#pragma unroll
        for (int k = 0; k < 4; ++k) l[v + k] = q[k];
      }
      return;
    }
  }
  if constexpr (V >= 8) {
    if (j.vec && j.dtype == MOE_BF16) {
#pragma unroll
      for (int v = 0; v < V; v += 8) {
        u32x4 q = {~0u, ~0u, ~0u, ~0u};  // bf16 NaN
        if (e0 + v < j.E) q = *reinterpret_cast<const u32x4*>((const uint16_t*)j.logits + row + e0 + v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          l[v + 2 * k] = __uint_as_float(q[k] << 16);
          l[v + 2 * k + 1] = __uint_as_float(q[k] & 0xffff0000u);
        }
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = e0 + v < j.E ? logit_at(j, row + e0 + v) : NAN;
}

// exp(l - m) with NaN and -inf as 0, and equal shares where the largest is +inf
__device__ __forceinline__ float part_of(float l, float m) {
  if (!(l > -INFINITY)) return 0.f;
  if (m == INFINITY) return l == INFINITY ? 1.f : 0.f;
  return expf(l - m);
}

// log(sigma(l)): the renormalised sigmoid is the softmax of these, which neither the sum of
// many tiny sigmoids nor their quotients underflow in
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.f) - log1pf(expf(-fabsf(l))); }
__device__ __forceinline__ float sigmoid(float l) { return 1.f / (1.f + expf(-l)); }

// fp32 order as unsigned integers; 0 for what is never chosen (NaN, -inf).  The addition makes
// -0 and +0 equal.
__device__ __forceinline__ uint32_t order_key(float score) {
  if (!(score > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(score + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// The chosen position's share of the weights before `scale`: position lane (and lane + 16) of the
// row in each lane, l[] its logit, there[] whether it names an expert.  For softmax over all
// experts m and z are given; otherwise they are taken over the chosen.
struct Shares {
  float p[2];
};
__device__ __forceinline__ Shares chosen_shares(const RouteJob& j, const float* l, const bool* there, float m_all,
                                                float z_all) {
  Shares s;
  if (j.score == MOE_SIGMOID && !j.renorm) {
#pragma unroll
    for (int r = 0; r < 2; ++r) s.p[r] = there[r] ? sigmoid(l[r]) : 0.f;
    return s;
  }
  float v[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) v[r] = !there[r] ? -INFINITY : j.score == MOE_SIGMOID ? log_sigmoid(l[r]) : l[r];
  const float m = j.renorm ? max16(fmaxf(v[0], v[1])) : m_all;
#pragma unroll
  for (int r = 0; r < 2; ++r) s.p[r] = part_of(v[r], m);
  const float z = j.renorm ? sum16(s.p[0] + s.p[1]) : z_all;
#pragma unroll
  for (int r = 0; r < 2; ++r) s.p[r] = z > 0.f ? s.p[r] / z : 0.f;
  return s;
}

template <int V>
__device__ __forceinline__ void softmax_of_all(const float* l, float& m, float& z) {
  m = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) m = fmaxf(m, l[v]);  // fmaxf passes over NaN
  m = max16(m);
  z = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) z += part_of(l[v], m);
  z = sum16(z);
}

// K rounds, each taking the row's largest key: the maximum of the lane's own, then of the 16
// lanes; the lowest expert that has it (lanes hold ascending experts) is struck out by its owner.
template <int V>
__global__ __launch_bounds__(kRouteT) void route_kernel(RouteJob j, const float* __restrict__ bias,
                                                        int32_t* __restrict__ expert, float* __restrict__ w) {
  const int t = blockIdx.x * kRouteTok + (threadIdx.x >> 4), lane = threadIdx.x & 15;
  if (t >= j.T) return;  // whole rows of 16 lanes leave; no barrier follows
  const int e0 = lane * V;
  float l[V];
  uint32_t key[V];
  load_logits<V>(j, t, e0, l);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float s = l[v];
    if (bias && e0 + v < j.E) s = s + bias[e0 + v];
    key[v] = order_key(s);
  }
  int ce[2] = {-1, -1};
  for (int k = 0; k < j.K; ++k) {
    uint32_t best = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) best = max(best, key[v]);
    best = max16u(best);
    uint32_t at = ~0u;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) at = key[v] == best ? (uint32_t)(e0 + v) : at;
    at = min16u(at);
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = at == (uint32_t)(e0 + v) ? 0u : key[v];
    const int e = best ? (int)at : -1;
    if (lane == (k & 15)) {
      if (k < 16) ce[0] = e;
      else ce[1] = e;
    }
  }
  float m = 0.f, z = 0.f, lc[2];
  bool there[2];
  if (j.score == MOE_SOFTMAX && !j.renorm) softmax_of_all<V>(l, m, z);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    there[r] = ce[r] >= 0;
    lc[r] = there[r] ? logit_at(j, (int64_t)t * j.pitch + ce[r]) : 0.f;
  }
  const Shares s = chosen_shares(j, lc, there, m, z);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int k = lane + 16 * r;
    if (k < j.K) {
      expert[(int64_t)t * j.K + k] = ce[r];
      w[(int64_t)t * j.K + k] = j.scale * s.p[r];
    }
  }
}

// With p the shares and v = scale dw:
//   softmax over the chosen:  dl_j = p_j (v_j - <v, p>)
//   softmax over all:         dl_e = p_e (sum of v_j over j that name e - <v, p>)
//   sigmoid:                  dl_j = v_j p_j sigma(-l_j)
//   sigmoid over the chosen:  dl_j = p_j (v_j - <v, p>) sigma(-l_j)
template <int V>
__global__ __launch_bounds__(kRouteT) void route_backward_kernel(RouteJob j, const int32_t* __restrict__ expert,
                                                                 const float* __restrict__ dw, void* dlogits,
                                                                 int64_t dpitch, uint32_t* err) {
  const int t = blockIdx.x * kRouteTok + (threadIdx.x >> 4), lane = threadIdx.x & 15;
  if (t >= j.T) return;
  const int e0 = lane * V;
  const bool all = j.score == MOE_SOFTMAX && !j.renorm;
  int ce[2];
  float lc[2], v[2], dl[2];
  bool there[2], bad = false;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int k = lane + 16 * r;
    ce[r] = k < j.K ? expert[(int64_t)t * j.K + k] : -1;
    there[r] = ce[r] >= 0 && ce[r] < j.E;
    bad |= !there[r] && ce[r] != -1;
    v[r] = there[r] ? j.scale * dw[(int64_t)t * j.K + k] : 0.f;
    lc[r] = there[r] ? logit_at(j, (int64_t)t * j.pitch + ce[r]) : 0.f;
  }
  if (bad) atomicOr(err, MOE_ERR_EXPERT_NONLOCAL);
  float l[V], m = 0.f, z = 0.f;
  if (all) {
    load_logits<V>(j, t, e0, l);
    softmax_of_all<V>(l, m, z);
  }
  const Shares s = chosen_shares(j, lc, there, m, z);
  const bool alone = j.score == MOE_SIGMOID && !j.renorm;
  const float vp = alone ? 0.f : sum16(v[0] * s.p[0] + v[1] * s.p[1]);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    dl[r] = s.p[r] * (all ? v[r] : v[r] - vp);
    if (j.score == MOE_SIGMOID) dl[r] *= sigmoid(-lc[r]);
  }
  float d[V];
#pragma unroll
  for (int q = 0; q < V; ++q) d[q] = all && z > 0.f ? -(part_of(l[q], m) / z) * vp : 0.f;
  for (int k = 0; k < j.K; ++k) {
    const int e = __shfl(k < 16 ? ce[0] : ce[1], k & 15, 16);
    const float g = __shfl(k < 16 ? dl[0] : dl[1], k & 15, 16);
#pragma unroll
    for (int q = 0; q < V; ++q) d[q] += e == e0 + q ? g : 0.f;
  }
  const int64_t row = (int64_t)t * dpitch;
#pragma unroll
  for (int q = 0; q < V; ++q) {
    if (e0 + q >= j.E) continue;
    if (j.dtype == MOE_F32) ((float*)dlogits)[row + e0 + q] = d[q];
    else ((uint16_t*)dlogits)[row + e0 + q] = f32_to_bf16(d[q]);
  }
}

static int check_route(int32_t T, int32_t E, int32_t K, int32_t dtype, int64_t pitch, int32_t score, int32_t renorm) {
  if (T < 0 || T > (1 << 24) || E < 1 || E > kRouteE || K < 1 || K > kRouteK || K > E || (int64_t)T * K > (1 << 24) ||
      pitch < E || pitch > ((int64_t)1 << 32))
    return MOE_EINVAL_SIZE;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EINVAL_DTYPE;
  if ((score != MOE_SOFTMAX && score != MOE_SIGMOID) || (renorm != 0 && renorm != 1)) return MOE_EINVAL_SIZE;
  return MOE_OK;
}

static RouteJob make_route_job(int32_t T, int32_t E, int32_t K, int32_t dtype, int64_t pitch, int32_t score,
                               int32_t renorm, float scale, const void* logits) {
  const int esz = dtype_size(dtype);
  RouteJob j;
  j.T = T; j.E = E; j.K = K; j.dtype = dtype; j.score = score; j.renorm = renorm;
  j.pitch = pitch; j.scale = scale; j.logits = logits;
  j.vec = aligned_rows(logits, pitch, esz, 16) && (E * esz) % 16 == 0;
  return j;
}

// the smallest V of 16 V >= E: a token's row of lanes holds every logit
template <template <int> class F, typename... A>
static int by_width(int E, A... a) {
  if (E <= 16) return F<1>::go(a...);
  if (E <= 32) return F<2>::go(a...);
  if (E <= 64) return F<4>::go(a...);
  if (E <= 128) return F<8>::go(a...);
  if (E <= 256) return F<16>::go(a...);
  return F<32>::go(a...);
}

template <int V>
struct Route {
  static int go(const RouteJob& j, const moe_route_args* a, hipStream_t stream) {
    return launch(route_kernel<V>, (unsigned)((a->T + kRouteTok - 1) / kRouteTok), kRouteT, stream, j, a->bias,
                  a->expert, a->w);
  }
};

template <int V>
struct RouteBackward {
  static int go(const RouteJob& j, const moe_route_backward_args* a, hipStream_t stream) {
    return launch(route_backward_kernel<V>, (unsigned)((a->T + kRouteTok - 1) / kRouteTok), kRouteT, stream, j,
                  a->expert, a->dw, a->dlogits, a->dlogits_pitch, a->err);
  }
};

}  // namespace moe

using namespace moe;

extern "C" int moe_route(const moe_route_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  const int rc = check_route(a->T, a->E, a->K, a->dtype, a->pitch, a->score, a->renorm);
  if (rc != MOE_OK) return rc;
  if (a->T == 0) return MOE_OK;
  if (!a->logits || !a->expert || !a->w) return MOE_EINVAL_NULL;
  if ((uintptr_t)a->logits % dtype_size(a->dtype)) return MOE_EINVAL_ALIGN;
  const RouteJob j = make_route_job(a->T, a->E, a->K, a->dtype, a->pitch, a->score, a->renorm, a->scale, a->logits);
  return by_width<Route>(a->E, j, a, stream);
}

extern "C" int moe_route_backward(const moe_route_backward_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  const int rc = check_route(a->T, a->E, a->K, a->dtype, a->pitch, a->score, a->renorm);
  if (rc != MOE_OK) return rc;
  if (a->dlogits_pitch < a->E || a->dlogits_pitch > ((int64_t)1 << 32)) return MOE_EINVAL_SIZE;
  if (!a->err) return MOE_EINVAL_NULL;
  if (a->T == 0) return MOE_OK;
  if (!a->logits || !a->expert || !a->dw || !a->dlogits) return MOE_EINVAL_NULL;
  if ((uintptr_t)a->logits % dtype_size(a->dtype) || (uintptr_t)a->dlogits % dtype_size(a->dtype))
    return MOE_EINVAL_ALIGN;
  const RouteJob j = make_route_job(a->T, a->E, a->K, a->dtype, a->pitch, a->score, a->renorm, a->scale, a->logits);
  return by_width<RouteBackward>(a->E, j, a, stream);
}
