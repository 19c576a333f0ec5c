// moe_route, moe_route_backward: choice of experts and router weights from logits, and the
// logits' gradient.
//
// A token belongs to one row of 16 lanes (four tokens per wave), which holds its logits in runs of
// W = min(V, 4) experts: lane l has e = (v / W) 16 W + l W + v % W for v < V, V = 1, 2, 4, ... 32 the
// smallest that covers E, so that a load covers 64 consecutive logits.  Reductions stay inside the
// row, as DPP operands.
#include <float.h>
#include <math.h>

#include "home.hpp"

namespace moe {

constexpr int kRouteE = 512, kRouteK = 32;
constexpr int kRouteT = 256;               // threads per workgroup
constexpr int kRouteTok = kRouteT / 16;    // tokens per workgroup

struct RouteJob {
  int T, E, K, dtype, vec, vec_bias, score, renorm;  // score without MOE_BIAS_ON_SCORE
  int64_t pitch;
  float scale;
  const void* logits;
};

__device__ __forceinline__ float logit_at(const RouteJob& j, int64_t at) {
  return j.dtype == MOE_F32 ? ((const float*)j.logits)[at] : bf16_to_f32(((const uint16_t*)j.logits)[at]);
}

template <int V>
__device__ __forceinline__ int expert_of(int lane, int v) {
  constexpr int W = V < 4 ? V : 4;
  return (v / W) * (16 * W) + lane * W + v % W;
}

// The lane's V logits (NaN past E).  vec: runs of four start on their own size, and E is whole runs.
template <int V>
__device__ __forceinline__ void load_logits(const RouteJob& j, int t, int lane, float* l) {
  const int64_t row = (int64_t)t * j.pitch;
  if constexpr (V >= 4) {
    if (j.vec) {
      if (j.dtype == MOE_F32) {
#pragma unroll
        for (int v = 0; v < V; v += 4) {
          const int e = expert_of<V>(lane, v);
          f32x4 q = {NAN, NAN, NAN, NAN};
          if (e < j.E) q = *reinterpret_cast<const f32x4*>((const float*)j.logits + row + e);
#pragma unroll
          for (int k = 0; k < 4; ++k) l[v + k] = q[k];
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; v += 4) {
          const int e = expert_of<V>(lane, v);
          u32x2 q = {~0u, ~0u};  // bf16 NaN
          if (e < j.E) q = *reinterpret_cast<const u32x2*>((const uint16_t*)j.logits + row + e);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            l[v + 2 * k] = __uint_as_float(q[k] << 16);
            l[v + 2 * k + 1] = __uint_as_float(q[k] & 0xffff0000u);
          }
        }
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<V>(lane, v);
    l[v] = e < j.E ? logit_at(j, row + e) : NAN;
  }
}

template <int V>
__device__ __forceinline__ void load_bias(const RouteJob& j, const float* bias, int lane, float* b) {
  if constexpr (V >= 4) {
    if (j.vec_bias) {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const int e = expert_of<V>(lane, v);
        f32x4 q = {0.f, 0.f, 0.f, 0.f};
        if (e < j.E) q = *reinterpret_cast<const f32x4*>(bias + e);
#pragma unroll
        for (int k = 0; k < 4; ++k) b[v + k] = q[k];
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<V>(lane, v);
    b[v] = e < j.E ? bias[e] : 0.f;
  }
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
__device__ __forceinline__ uint32_t order_key(float rank) {
  if (!(rank > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(rank + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// the rank of a key (not of 0)
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key ^ (~(uint32_t)((int32_t)key >> 31) | 0x80000000u));
}

// The chosen position's share of the weights before `scale`: position lane (and lane + 16) of the
// row in each lane, l[] its logit, there[] whether it names an expert.  For softmax over all
// experts m and z are given; otherwise they are taken over the chosen.
template <int R>
__device__ __forceinline__ void chosen_shares(const RouteJob& j, const float* l, const bool* there, float m_all,
                                              float z_all, float* p) {
  if (j.score == MOE_SIGMOID && !j.renorm) {
#pragma unroll
    for (int r = 0; r < R; ++r) p[r] = there[r] ? sigmoid(l[r]) : 0.f;
    return;
  }
  float v[R], m = -INFINITY, z = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    v[r] = !there[r] ? -INFINITY : j.score == MOE_SIGMOID ? log_sigmoid(l[r]) : l[r];
    m = fmaxf(m, v[r]);
  }
  m = j.renorm ? max16(m) : m_all;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    p[r] = part_of(v[r], m);
    z += p[r];
  }
  z = j.renorm ? sum16(z) : z_all;
#pragma unroll
  for (int r = 0; r < R; ++r) p[r] = z > 0.f ? p[r] / z : 0.f;
}

// l becomes exp(l - m), z their sum over the token.  The exponential is v_exp_f32 of a product: off
// by |l - m| 2^-24 relative, as the subtraction's own rounding of large logits is.
template <int V>
__device__ __forceinline__ void softmax_of_all(float* l, float& m, float& z) {
  m = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) m = fmaxf(m, l[v]);  // fmaxf passes over NaN
  m = max16(m);
  z = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float e = m == INFINITY ? (l[v] == INFINITY ? 1.f : 0.f)
                                  : __builtin_amdgcn_exp2f((l[v] - m) * 1.44269504f);
    l[v] = l[v] > -INFINITY ? e : 0.f;
    z += l[v];
  }
  z = sum16(z);
}

// b[] becomes the ranks s + b, s the gate's scores rounded as the weights' are; NaN where the logit is
// NaN or -inf.  16384 tokens x 256 fp32, top-8: 11.1 us with sigmoids, 12.8 with the softmax (on the
// logits 8.0): an exponential and a quotient for each of them.
template <int V>
__device__ __forceinline__ void add_scores(const RouteJob& j, const float* l, float* b) {
  float m = 0.f, z = 1.f, e[V];
  if (j.score == MOE_SOFTMAX) {
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = l[v];
    softmax_of_all<V>(e, m, z);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float s = j.score == MOE_SIGMOID ? sigmoid(l[v]) : part_of(l[v], m) / z;
    b[v] = l[v] > -INFINITY ? s + b[v] : NAN;
  }
}

// A candidate as one number: the rank's order in bits 30..61 and 511 - e below, so that the larger
// of two is the larger rank, or the lower expert of equal ones.  Read as a double it is positive
// and finite, and the order of such doubles is that of their bits: v_max_f64 compares both parts in
// one instruction.
struct Candidate {
  uint32_t hi, lo;
};
__device__ __forceinline__ Candidate larger(Candidate a, Candidate b) {
  double x = __hiloint2double((int)a.hi, (int)a.lo), r;
  const double y = __hiloint2double((int)b.hi, (int)b.lo);
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(x), "v"(y));
  return {(uint32_t)__double2hiint(r), (uint32_t)__double2loint(r)};
}
template <int CTRL>
__device__ __forceinline__ Candidate larger_dpp(Candidate a) {
  return larger(a, {dpp_u32<CTRL>(a.hi), dpp_u32<CTRL>(a.lo)});
}

__device__ __forceinline__ Candidate smaller(Candidate a, Candidate b) {
  double x = __hiloint2double((int)a.hi, (int)a.lo), r;
  const double y = __hiloint2double((int)b.hi, (int)b.lo);
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(x), "v"(y));
  return {(uint32_t)__double2hiint(r), (uint32_t)__double2loint(r)};
}
__device__ __forceinline__ void order(Candidate& a, Candidate& b) {  // the larger first
  const Candidate x = larger(a, b);
  b = smaller(a, b);
  a = x;
}

// The N largest of a row's candidates, descending, in every lane: sorting networks of N = 4 or 8.
// Two descending lists a, b have their N largest in max(a[i], b[N - 1 - i]), which rises and falls
// once and is sorted by halving.
template <int N>
__device__ __forceinline__ void sort_halving(Candidate* a) {
#pragma unroll
  for (int d = N / 2; d; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(i & d)) order(a[i], a[i + d]);
}
template <int N>
__device__ __forceinline__ void sort_all(Candidate* a) {  // odd-even merge sort
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int k = p; k; k >>= 1)
#pragma unroll
      for (int i = k & (p - 1); i + k < N; i += 2 * k)
#pragma unroll
        for (int q = 0; q < k; ++q)
          if (i + q + k < N && (i + q) / (2 * p) == (i + q + k) / (2 * p)) order(a[i + q], a[i + q + k]);
}
template <int N, int CTRL>
__device__ __forceinline__ void merge_dpp(Candidate* a) {
  Candidate m[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    m[i] = larger(a[i], {dpp_u32<CTRL>(a[N - 1 - i].hi), dpp_u32<CTRL>(a[N - 1 - i].lo)});
  sort_halving<N>(m);
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = m[i];
}
template <int V, int N>
__device__ __forceinline__ void largest_sorted(const Candidate* c, Candidate* a) {
#pragma unroll
  for (int g = 0; g < V; g += N) {
    Candidate b[N];
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = g + i < V ? c[g + i] : Candidate{0u, 0u};
    sort_all<N>(b);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = g ? larger(a[i], b[N - 1 - i]) : b[i];
    if (g) sort_halving<N>(a);
  }
  merge_dpp<N, kDppXor1>(a);
  merge_dpp<N, kDppXor2>(a);
  merge_dpp<N, kDppHalfMirror>(a);
  merge_dpp<N, kDppMirror>(a);
}

// Bound by its instructions: 16384 tokens x 256 fp32, top-8, sigmoid with bias move 18 MB (4 us) and
// take 8.0 us a call (the kernel 7.6 in the median of 20, 6.6 the fastest); K rounds of a maximum over the
// row took 10.3, and with a 32-bit maximum, a search for its lowest expert and lanes that each loaded 64
// consecutive bytes 17.0.  A small call (64 tokens) is launch and latency, the kernel 2.9 us.  K > 8 takes
// the rounds: 16384 x 512, top-10, 20 us.
// N = 4, 8: the N >= K largest by sorting networks.  N = 0 (K > 8): K rounds, each taking the row's
// largest candidate, the maximum of the lane's own and then of the 16 lanes, which its owner strikes
// out.  ON_SCORE: there is a bias, of the gate's scores and not of the logits.
template <int V, int N, bool ON_SCORE>
__global__ __launch_bounds__(kRouteT) void route_kernel(RouteJob j, const float* __restrict__ bias,
                                                        int32_t* __restrict__ expert, float* __restrict__ w) {
  constexpr int R = N ? 1 : 2;  // positions per lane
  const int t = blockIdx.x * kRouteTok + (threadIdx.x >> 4), lane = threadIdx.x & 15;
  if (t >= j.T) return;  // whole rows of 16 lanes leave; no barrier follows
  float l[V];
  Candidate c[V];
  load_logits<V>(j, t, lane, l);
  float b[V];
  if (bias) load_bias<V>(j, bias, lane, b);
  if constexpr (ON_SCORE) add_scores<V>(j, l, b);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<V>(lane, v);
    const uint32_t key = order_key(ON_SCORE ? b[v] : bias ? l[v] + b[v] : l[v]);
    c[v] = {key >> 2, key << 30 | (uint32_t)(kRouteE - 1 - e)};
  }
  Candidate mine[R];
#pragma unroll
  for (int r = 0; r < R; ++r) mine[r] = {0u, 0u};
  if constexpr (N > 0) {
    Candidate a[N];
    largest_sorted<V, N>(c, a);
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (lane == k) mine[0] = a[k];
  } else {
    for (int k = 0; k < j.K; ++k) {
      Candidate m[V];
#pragma unroll
      for (int v = 0; v < V; ++v) m[v] = c[v];
#pragma unroll
      for (int d = 1; d < V; d <<= 1)
#pragma unroll
        for (int v = 0; v + d < V; v += 2 * d) m[v] = larger(m[v], m[v + d]);
      Candidate best = larger_dpp<kDppXor1>(m[0]);
      best = larger_dpp<kDppXor2>(best);
      best = larger_dpp<kDppHalfMirror>(best);
      best = larger_dpp<kDppMirror>(best);
#pragma unroll
      for (int v = 0; v < V; ++v) c[v].hi = c[v].lo == best.lo ? 0u : c[v].hi;
      if (lane == (k & 15)) {
        if (k < 16) mine[0] = best;
        else mine[1] = best;
      }
    }
  }
  float m = 0.f, z = 0.f, lc[R];
  bool there[R];
  int ce[R];
  if (j.score == MOE_SOFTMAX && !j.renorm) softmax_of_all<V>(l, m, z);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    there[r] = mine[r].hi != 0 && lane + 16 * r < j.K;
    ce[r] = there[r] ? kRouteE - 1 - (int)(mine[r].lo & (kRouteE - 1)) : -1;
    lc[r] = there[r] ? key_value(mine[r].hi << 2 | mine[r].lo >> 30) : 0.f;
    if (bias && there[r]) lc[r] = logit_at(j, (int64_t)t * j.pitch + ce[r]);
  }
  float p[R];
  chosen_shares<R>(j, lc, there, m, z, p);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int k = lane + 16 * r;
    if (k < j.K) {
      expert[(int64_t)t * j.K + k] = ce[r];
      w[(int64_t)t * j.K + k] = j.scale * p[r];
    }
  }
}

// LDS accesses of a wave before it come before those after it (the hardware keeps them in order)
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// With p the shares and v = scale dw:
//   softmax over the chosen:  dl_j = p_j (v_j - <v, p>)
//   softmax over all:         dl_e = p_e (sum of v_j over j that name e - <v, p>)
//   sigmoid:                  dl_j = v_j p_j sigma(-l_j)
//   sigmoid over the chosen:  dl_j = p_j (v_j - <v, p>) sigma(-l_j)
template <int V, int R>
__global__ __launch_bounds__(kRouteT) void route_backward_kernel(RouteJob j, const int32_t* __restrict__ expert,
                                                                 const float* __restrict__ dw, void* dlogits,
                                                                 int64_t dpitch, int vec_out, uint32_t* err) {
  const int t = blockIdx.x * kRouteTok + (threadIdx.x >> 4), lane = threadIdx.x & 15;
  if (t >= j.T) return;
  const bool all = j.score == MOE_SOFTMAX && !j.renorm;
  int ce[R];
  float lc[R], v[R], dl[R], p[R];
  bool there[R], bad = false;
#pragma unroll
  for (int r = 0; r < R; ++r) {
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
    load_logits<V>(j, t, lane, l);
    softmax_of_all<V>(l, m, z);
  }
  chosen_shares<R>(j, lc, there, m, z, p);
  float vp = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) vp = fmaf(v[r], p[r], vp);
  vp = j.score == MOE_SIGMOID && !j.renorm ? 0.f : sum16(vp);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    dl[r] = p[r] * (all ? v[r] : v[r] - vp);
    if (j.score == MOE_SIGMOID) dl[r] *= sigmoid(-lc[r]);
  }
  float d[V];
  const float each = all && z > 0.f ? -vp / z : 0.f;
#pragma unroll
  for (int q = 0; q < V; ++q) d[q] = all ? l[q] * each : 0.f;
  // the chosen experts' part through the token's row in LDS, which only its own 16 lanes touch: each
  // position marks its expert, and where none finds another's mark no expert is named twice and
  // each writes its value (forward and gradient of 16384 x 256, top-8, softmax over all: 17.1 us; 18.9 with every position
  // held against every expert, as the other branch does)
  constexpr int W = V < 4 ? V : 4;
  __shared__ __attribute__((aligned(16))) float s_row[kRouteTok][16 * V];
  float* mine = s_row[threadIdx.x >> 4];
#pragma unroll
  for (int q = 0; q < V; q += W)
#pragma unroll
    for (int k = 0; k < W; ++k) mine[expert_of<V>(lane, q) + k] = 0.f;
  wave_order();
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (there[r]) mine[ce[r]] = (float)(1 + lane + 16 * r);
  wave_order();
  bool twice = false;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (there[r]) twice |= mine[ce[r]] != (float)(1 + lane + 16 * r);
  wave_order();
  if (__ballot(twice) == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (there[r]) mine[ce[r]] = dl[r];
    wave_order();
#pragma unroll
    for (int q = 0; q < V; ++q) d[q] += mine[expert_of<V>(lane, q)];
  } else {  // in the order of the positions
    for (int k = 0; k < j.K; ++k) {
      const int e = __shfl(k < 16 ? ce[0] : ce[R - 1], k & 15, 16);
      const float g = __shfl(k < 16 ? dl[0] : dl[R - 1], k & 15, 16);
#pragma unroll
      for (int q = 0; q < V; ++q) d[q] += e == expert_of<V>(lane, q) ? g : 0.f;
    }
  }
  const int64_t row = (int64_t)t * dpitch;
  if constexpr (V >= 4) {
    if (vec_out) {
#pragma unroll
      for (int q = 0; q < V; q += 4) {
        const int e = expert_of<V>(lane, q);
        if (e >= j.E) continue;
        if (j.dtype == MOE_F32)
          *reinterpret_cast<f32x4*>((float*)dlogits + row + e) = f32x4{d[q], d[q + 1], d[q + 2], d[q + 3]};
        else
          *reinterpret_cast<u32x2*>((uint16_t*)dlogits + row + e) =
              u32x2{pack_bf16x2(d[q], d[q + 1]), pack_bf16x2(d[q + 2], d[q + 3])};
      }
      return;
    }
  }
#pragma unroll
  for (int q = 0; q < V; ++q) {
    const int e = expert_of<V>(lane, q);
    if (e >= j.E) continue;
    if (j.dtype == MOE_F32) ((float*)dlogits)[row + e] = d[q];
    else ((uint16_t*)dlogits)[row + e] = f32_to_bf16(d[q]);
  }
}

static int check_route(int32_t T, int32_t E, int32_t K, int32_t dtype, int64_t pitch, int32_t score, int32_t renorm) {
  if (T < 0 || T > (1 << 24) || E < 1 || E > kRouteE || K < 1 || K > kRouteK || K > E || (int64_t)T * K > (1 << 24) ||
      pitch < E || pitch > ((int64_t)1 << 32))
    return MOE_EINVAL_SIZE;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EINVAL_DTYPE;
  const int32_t gate = score & ~MOE_BIAS_ON_SCORE;
  if ((gate != MOE_SOFTMAX && gate != MOE_SIGMOID) || (renorm != 0 && renorm != 1)) return MOE_EINVAL_SIZE;
  return MOE_OK;
}

static bool runs_of_four(const void* rows, int64_t pitch, int E, int esz) {
  return E % 4 == 0 && aligned_rows(rows, pitch, esz, 4 * esz);
}

static RouteJob make_route_job(int32_t T, int32_t E, int32_t K, int32_t dtype, int64_t pitch, int32_t score,
                               int32_t renorm, float scale, const void* logits) {
  const int esz = dtype_size(dtype);
  RouteJob j;
  j.T = T; j.E = E; j.K = K; j.dtype = dtype; j.score = score & ~MOE_BIAS_ON_SCORE; j.renorm = renorm;
  j.pitch = pitch; j.scale = scale; j.logits = logits;
  j.vec = runs_of_four(logits, pitch, E, esz);
  j.vec_bias = 0;
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
    const unsigned grid = (unsigned)((a->T + kRouteTok - 1) / kRouteTok);
    auto kernel = a->bias && (a->score & MOE_BIAS_ON_SCORE) ? by_k<true>(a->K) : by_k<false>(a->K);
    return launch(kernel, grid, kRouteT, stream, j, a->bias, a->expert, a->w);
  }
  template <bool ON_SCORE>
  static auto by_k(int K) {
    return K <= 4 ? route_kernel<V, 4, ON_SCORE> : K <= 8 ? route_kernel<V, 8, ON_SCORE> : route_kernel<V, 0, ON_SCORE>;
  }
};

template <int V>
struct RouteBackward {
  static int go(const RouteJob& j, const moe_route_backward_args* a, hipStream_t stream) {
    const int vec_out = runs_of_four(a->dlogits, a->dlogits_pitch, a->E, dtype_size(a->dtype));
    return launch(a->K <= 16 ? route_backward_kernel<V, 1> : route_backward_kernel<V, 2>,
                  (unsigned)((a->T + kRouteTok - 1) / kRouteTok), kRouteT, stream, j, a->expert, a->dw, a->dlogits,
                  a->dlogits_pitch, vec_out, a->err);
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
  RouteJob j = make_route_job(a->T, a->E, a->K, a->dtype, a->pitch, a->score, a->renorm, a->scale, a->logits);
  j.vec_bias = runs_of_four(a->bias, a->E, a->E, 4);
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
