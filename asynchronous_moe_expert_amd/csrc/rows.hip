// moe_sort_rows, moe_merge_rows, moe_merge_rows_backward: rows of tokens sorted by expert and
// back.  All three move rows and are bound by memory; the index is integer work on n = T K ids.
#include "home.hpp"

namespace moe {

// lane_i32 and lane_f32 stand only where every lane of the wave is active: a lane that a branch has
// switched off need not hold its value.  Loops over a row's chunks therefore run the same number of
// turns in every lane, and a lane past the row's end leaves out the loads and stores alone.
__device__ __forceinline__ int lane_i32(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

constexpr int kMaxEloc = 256, kMaxK = 32;
constexpr int kNone = kMaxEloc;  // key of a pair without a row

struct SortJob {
  int T, K, n, base, E_loc;
  const int32_t* expert;
  int32_t *perm, *pos, *counts, *offsets, *row_slot;
  uint32_t* err;
};

__device__ __forceinline__ int sort_key(const SortJob& j, int i, unsigned& bad) {
  const int g = j.expert[i];
  const int64_t e = (int64_t)g - j.base;
  if (g != -1 && e >= 0 && e < j.E_loc) return (int)e;
  if (g != -1) bad = MOE_ERR_EXPERT_NONLOCAL;
  return kNone;
}

// ------------------------------------------------------------------------------- index
// Two launches over at most kSegs segments of the pairs (a multiple of kIdx pairs each):
//   count   each workgroup counts its segment's keys into ws[segment][E_loc]
//   place   each workgroup sums the counts of the segments before its own and of all (at most
//           kSegs x E_loc values, L2-resident), scans them over the experts, and gives its own
//           pairs their rows, 1024 at a time: a pair's rank among equal keys of its wave from a
//           9-bit ballot match, the waves' counts scanned per expert
// 65536 pairs over 256 experts: 4.7 and 5.3 us, 16396 over 128: 2.6-4 and 5.0, all of it latency.  One
// launch in which every workgroup counts all keys took 8.6 us in all at 8192 pairs where these take
// 8.9, but 10.9 for 9.4 at 16384 and 28 for 14 at 65536.
constexpr int kIdx = 1024, kIdxWaves = kIdx / kWave;
constexpr int kSegs = 256;
constexpr int kCopies = 4;  // counters per expert: a favoured expert's lanes do not queue on one

__global__ __launch_bounds__(kIdx) void sort_count_kernel(SortJob j, int seg_len, int32_t* __restrict__ ws) {
  __shared__ int s_cnt[kMaxEloc * (kCopies + 1)];
  const int tid = threadIdx.x;
  for (int x = tid; x < kMaxEloc * (kCopies + 1); x += kIdx) s_cnt[x] = 0;
  __syncthreads();
  const int lo = blockIdx.x * seg_len, hi = min(j.n, lo + seg_len);
  unsigned bad = 0;
  for (int i = lo + tid; i < hi; i += kIdx) {
    const int key = sort_key(j, i, bad);
    if (key < kNone) atomicAdd(&s_cnt[key * (kCopies + 1) + (tid & (kCopies - 1))], 1);
  }
  if (bad) atomicOr(j.err, bad);
  __syncthreads();
  for (int e = tid; e < j.E_loc; e += kIdx) {
    int sum = 0;
    for (int c = 0; c < kCopies; ++c) sum += s_cnt[e * (kCopies + 1) + c];
    ws[blockIdx.x * j.E_loc + e] = sum;
  }
}

__global__ __launch_bounds__(kIdx) void sort_place_kernel(SortJob j, int segs, int seg_len,
                                                          const int32_t* __restrict__ ws) {
  __shared__ int s_run[kMaxEloc];  // next row of each expert in this segment
  __shared__ int s_all[kMaxEloc];
  __shared__ int s_wcnt[kIdxWaves][kMaxEloc + 1];
  __shared__ int s_total;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, seg = blockIdx.x;
  const int lo = seg * seg_len, hi = min(j.n, lo + seg_len);
  unsigned bad = 0;  // the count has reported these
  int key = lo + tid < hi ? sort_key(j, lo + tid, bad) : kNone;
  // column sums: thread (g, e) takes the segments g, g + 4, ..., eight loads at a time
  const int col = tid & (kMaxEloc - 1);
  int before = 0, all = 0;
  if (col < j.E_loc) {
    for (int s0 = tid / kMaxEloc; s0 < segs; s0 += 8 * (kIdx / kMaxEloc)) {
      int c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int s = s0 + u * (kIdx / kMaxEloc);
        c[u] = s < segs ? ws[s * j.E_loc + col] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        all += c[u];
        before += s0 + u * (kIdx / kMaxEloc) < seg ? c[u] : 0;
      }
    }
  }
  for (int e = tid; e < kMaxEloc; e += kIdx) s_run[e] = s_all[e] = 0;
  for (int c0 = lo; c0 < hi; c0 += kIdx) {
    const int i = c0 + tid;
    if (c0 > lo) key = i < hi ? sort_key(j, i, bad) : kNone;
    for (int x = tid; x < kIdxWaves * (kMaxEloc + 1); x += kIdx) (&s_wcnt[0][0])[x] = 0;
    uint64_t peers = ~0ull;
#pragma unroll
    for (int b = 0; b < 9; ++b) {
      const bool bit = (key >> b) & 1;
      const uint64_t bal = __ballot(bit);
      peers &= bit ? bal : ~bal;
    }
    const int rank = __popcll(peers & ((1ull << lane) - 1ull));
    __syncthreads();
    if (key < kNone && rank == 0) s_wcnt[wv][key] = __popcll(peers);
    if (c0 == lo && col < j.E_loc) {
      atomicAdd(&s_run[col], before);
      atomicAdd(&s_all[col], all);
    }
    __syncthreads();
    if (c0 == lo && wv == 0) {  // exclusive scan over the experts, four per lane
      int v[4], sum = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = s_all[lane * 4 + k];
        sum += v[k];
      }
      int incl = sum;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int t = __shfl_up(incl, d);
        if (lane >= d) incl += t;
      }
      int run = incl - sum;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = lane * 4 + k;
        if (seg == 0 && e < j.E_loc) {
          j.counts[e] = v[k];
          j.offsets[e] = run;
        }
        s_run[e] += run;
        run += v[k];
      }
      if (lane == 63) {
        s_total = incl;
        if (seg == 0) j.offsets[j.E_loc] = incl;
      }
    }
    int chunk = 0;  // this chunk's pairs of expert e = tid - 256, whose waves' counts become offsets
    if (tid >= kMaxEloc && tid < 2 * kMaxEloc) {
#pragma unroll
      for (int w = 0; w < kIdxWaves; ++w) {
        const int cnt = s_wcnt[w][tid - kMaxEloc];
        s_wcnt[w][tid - kMaxEloc] = chunk;
        chunk += cnt;
      }
    }
    __syncthreads();
    if (key < kNone) {
      const int r = s_run[key] + s_wcnt[wv][key] + rank;
      j.pos[i] = r;
      if (j.perm) j.perm[r] = i;
      if (j.row_slot) j.row_slot[r] = i / j.K;
    } else if (i < hi) {
      j.pos[i] = -1;
    }
    if (i < hi && i >= s_total) {  // rows past the last
      if (j.perm) j.perm[i] = -1;
      if (j.row_slot) j.row_slot[i] = -1;
    }
    if (c0 + kIdx >= hi) break;
    __syncthreads();
    if (tid >= kMaxEloc && tid < 2 * kMaxEloc) s_run[tid - kMaxEloc] += chunk;
  }
}

// no pairs: every count is zero
__global__ void sort_empty_kernel(SortJob j) {
  for (int e = threadIdx.x; e <= j.E_loc; e += blockDim.x) {
    if (e < j.E_loc) j.counts[e] = 0;
    j.offsets[e] = 0;
  }
}

// -------------------------------------------------------------------------- copying rows
// Threads of a workgroup that takes a row: the fewest passes of at most 512 lanes over its chunks,
// the lanes spread evenly over them.
static unsigned row_threads(int chunks) {
  const int passes = (chunks + 511) / 512, per = (chunks + passes - 1) / passes;
  return (unsigned)((per + 63) / 64 * 64);
}

struct CopyJob {
  int K, H, chunks;  // chunks of eight elements in a row
  int group_shift;   // fp8: log2 of the columns per scale, -1 for one per row
  int groups;
  const void* x;
  int64_t x_pitch;
  const float* x_scale;
  void* xs;
  int64_t xs_pitch;
};

template <int DT>
struct SortedType {
  static constexpr int out = DT == MOE_FP8_E4M3 ? MOE_BF16 : DT;
};

// A chunk of token t's row on its way: read once, written to the token's K rows (NT: by
// non-temporal stores).
template <int DT, bool NT>
struct Carried {
  static constexpr int esz = DT == MOE_F32 ? 4 : DT == MOE_BF16 ? 2 : 1;
  static constexpr int OUT = SortedType<DT>::out, osz = OUT == MOE_F32 ? 4 : 2;
  Chunk<DT> q;
  float s;
  __device__ __forceinline__ void load(const CopyJob& c, int t, int ch) {
    q.load((const char*)c.x + (int64_t)t * c.x_pitch * esz, (int64_t)ch * 8);
    if constexpr (DT == MOE_FP8_E4M3)
      s = c.x_scale[(int64_t)t * c.groups + (c.group_shift < 0 ? 0 : (ch * 8) >> c.group_shift)];
  }
  // position k's row in lane k of p; called by whole waves, `there` where the lane has a chunk
  __device__ __forceinline__ void store(const CopyJob& c, int ch, int p, bool there) const {
    float f[8];
    q.get(f);
    if constexpr (DT == MOE_FP8_E4M3) {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= s;
    }
    for (int k = 0; k < c.K; ++k) {
      const int r = lane_i32(p, k);
      if (r < 0) continue;
      char* dst = (char*)c.xs + (int64_t)r * c.xs_pitch * osz;
      if (there) {
        if constexpr (DT == MOE_BF16)
          st<NT>(reinterpret_cast<u32x4*>((uint16_t*)dst + (int64_t)ch * 8), q.r);
        else
          st8<OUT, NT>(dst, (int64_t)ch * 8, f);
      }
    }
  }
};

// A workgroup per token (blockIdx, blockIdx + gridDim, ...), in a block that covers the row in the
// fewest passes (8192 tokens to 8 rows of 4096 bf16, 604 MB: 103 us in the median of 20 launches, 5.9 TB/s,
// 97 the fastest; blocks of 128 threads 3% more).  Bound by the writes: a standalone probe that writes each 16 bytes to eight places reaches
// 5.8 TB/s.
template <int DT, bool NT>
__global__ __launch_bounds__(512) void sort_copy_kernel(CopyJob c, int T, const int32_t* __restrict__ pos) {
  const int lane = threadIdx.x & 63;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    Carried<DT, NT> x;  // on its way while the positions are looked up
    if ((int)threadIdx.x < c.chunks) x.load(c, t, threadIdx.x);
    const int p = lane < c.K ? pos[(int64_t)t * c.K + lane] : -1;
    x.store(c, threadIdx.x, p, (int)threadIdx.x < c.chunks);
    for (int c0 = blockDim.x; c0 < c.chunks; c0 += blockDim.x) {
      const int ch = c0 + threadIdx.x;
      if (ch < c.chunks) x.load(c, t, ch);
      x.store(c, ch, p, ch < c.chunks);
    }
  }
}

// Short queues: index and copy in one launch.  A pair's row is the number of pairs with a lower
// (key, pair), so each token's workgroup stages all n pairs' (key, pair) in LDS, counts those below
// each of its own K pairs (a wave takes the positions wave, wave + waves, ...) and then copies its
// row, whose first chunks are loaded meanwhile; the last workgroup writes counts, offsets and what
// lies past the last row.  No workgroup waits for another.  Every token stages and counts n pairs,
// so the work grows with T n, and past 2^22 the index launches take over.  Microseconds short / long,
// rows of 2880 bf16 (K = 8: 4096): 300 tokens x 4 4.6 / 9.0, 512 x 4 6.1 / 9.9, 1000 x 4 10.5 / 12.1,
// 2000 x 1 9.9 / 11.9, 512 x 8 11.4 / 13.5; 1500 x 4 19.9 / 14.4, 4000 x 1 23.1 / 16.8, 1000 x 8 19.9 / 18.3.
constexpr int kShort = 4096;            // pairs that the LDS staging holds
constexpr int64_t kShortWork = 1 << 22;
constexpr int kShortAny = 2048;         // pairs that are short whatever K is
static_assert((int64_t)kShortAny * kShortAny <= kShortWork, "");

template <int DT>
__global__ __launch_bounds__(512) void sort_short_kernel(SortJob j, CopyJob c) {
  __shared__ __attribute__((aligned(16))) uint32_t s_all[kShort];
  __shared__ int s_pos[kMaxK];
  __shared__ int s_cnt[kMaxEloc + 1];
  const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  unsigned bad = 0;
  if ((int)blockIdx.x < j.T) {
    const int t = blockIdx.x;
    Carried<DT, false> x;
    if (tid < c.chunks) x.load(c, t, tid);
    const int padded = (j.n + 255) & ~255;
    for (int q = tid; q < padded; q += blockDim.x)
      s_all[q] = q < j.n ? (uint32_t)sort_key(j, q, bad) << 16 | (uint32_t)q : ~0u;
    __syncthreads();
    for (int k = wv; k < j.K; k += waves) {
      const int i = t * j.K + k;
      const uint32_t mine = s_all[i];
      int before = 0;
      for (int q = lane * 4; q < padded; q += 256) {
        const u32x4 o = *reinterpret_cast<const u32x4*>(&s_all[q]);
#pragma unroll
        for (int u = 0; u < 4; ++u) before += o[u] < mine;
      }
#pragma unroll
      for (int d = 32; d; d >>= 1) before += __shfl_xor(before, d);
      const int r = (mine >> 16) < kNone ? before : -1;
      if (lane == 0) {
        s_pos[k] = r;
        j.pos[i] = r;
        if (r >= 0 && j.perm) j.perm[r] = i;
        if (r >= 0 && j.row_slot) j.row_slot[r] = t;
      }
    }
    __syncthreads();
    const int p = lane < j.K ? s_pos[lane] : -1;
    if (c.chunks) x.store(c, tid, p, tid < c.chunks);
    for (int c0 = blockDim.x; c0 < c.chunks; c0 += blockDim.x) {
      const int ch = c0 + tid;
      if (ch < c.chunks) x.load(c, t, ch);
      x.store(c, ch, p, ch < c.chunks);
    }
    return;
  }
  for (int e = tid; e <= kMaxEloc; e += blockDim.x) s_cnt[e] = 0;
  __syncthreads();
  for (int q = tid; q < j.n; q += blockDim.x) atomicAdd(&s_cnt[sort_key(j, q, bad)], 1);
  if (bad) atomicOr(j.err, bad);
  __syncthreads();
  if (wv != 0) return;
  int v[4], sum = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = s_cnt[lane * 4 + k];
    sum += v[k];
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(incl, d);
    if (lane >= d) incl += u;
  }
  int run = incl - sum;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int e = lane * 4 + k;
    if (e < j.E_loc) {
      j.counts[e] = v[k];
      j.offsets[e] = run;
    }
    run += v[k];
  }
  const int total = lane_i32(incl, 63);
  if (lane == 0) j.offsets[j.E_loc] = total;
  for (int r = total + lane; r < j.n; r += 64) {
    if (j.perm) j.perm[r] = -1;
    if (j.row_slot) j.row_slot[r] = -1;
  }
}

// -------------------------------------------------------------------------- merging rows
struct MergeJob {
  int T, K, H, chunks;
  const void* rows;
  int64_t row_pitch, n_rows;
  const int32_t* pos;
  const float* w;
  void* out;
  int64_t out_pitch;
  uint32_t* err;
};

template <int DT>
__device__ __forceinline__ const char* row_at(const void* rows, int64_t r, int64_t pitch) {
  return (const char*)rows + r * pitch * (DT == MOE_F32 ? 4 : DT == MOE_BF16 ? 2 : 1);
}

// Position k of token t in lane k: its row or -1, and its weight.
struct Named {
  int p;
  float w;
};
__device__ __forceinline__ Named named_rows(const int32_t* pos, const float* w, uint32_t* err, int t, int K,
                                            int64_t n_rows, int lane) {
  Named r{-1, 0.f};
  if (lane < K) {
    const int64_t at = (int64_t)t * K + lane;
    r.p = pos[at];
    r.w = w ? w[at] : 1.f;
  }
  if (r.p < 0 || r.p >= n_rows) {
    if (r.p != -1) atomicOr(err, MOE_ERR_ROW_RANGE);
    r.p = -1;
  }
  return r;
}

// A workgroup per token, KB positions at a time: their loads are all issued before the first is
// used.  Each lane sums its chunk over the positions in order.  Bound by the reads: 8192 tokens from 8
// rows of 4096 bf16, 604 MB, 100 us (6.0 TB/s; 120 with plain loads; blocks of 256 threads 105, of 128
// 140).  A standalone probe that reads eight places at once reaches 6.3 TB/s.
template <int RT, int OT, int KB, int S>
__global__ __launch_bounds__(512) void merge_kernel(MergeJob m) {
  const int lane = threadIdx.x & 63;
  for (int t = blockIdx.x; t < m.T; t += gridDim.x) {
    const Named r = named_rows(m.pos, m.w, m.err, t, m.K, m.n_rows, lane);
    char* out = (char*)m.out + (int64_t)t * m.out_pitch * (OT == MOE_F32 ? 4 : 2);
    for (int c0 = 0; c0 < m.chunks; c0 += blockDim.x) {
      const int ch = c0 + threadIdx.x;
      const bool there = ch < m.chunks;
      float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      for (int k0 = 0; k0 < m.K; k0 += KB) {
        int p[KB];
        float w[KB];
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          p[k] = lane_i32(r.p, k0 + k);
          w[k] = lane_f32(r.w, k0 + k);
        }
        if (there) {
          Chunk<RT> q[KB];
#pragma unroll
          for (int k = 0; k < KB; ++k)
            if (p[k] >= 0) q[k].template load<(S >= kReadOnce)>(row_at<RT>(m.rows, p[k], m.row_pitch), (int64_t)ch * 8);
#pragma unroll
          for (int k = 0; k < KB; ++k) {
            if (p[k] < 0) continue;
            float f[8];
            q[k].get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[k], f[e], acc[e]);
          }
        }
      }
      if (there) st8<OT, S == kThrough>(out, (int64_t)ch * 8, acc);
    }
  }
}

struct MergeBackJob {
  int T, K, H, chunks;
  const void* dout;
  int64_t dout_pitch;
  const void* rows;
  int64_t row_pitch, n_rows;
  const int32_t* pos;
  const float* w;
  void* drows;
  int64_t drows_pitch;
  float* dw;
  uint32_t* err;
};

// A workgroup per token, KB positions at a time; a position's dot product runs through the lane's
// chunks, the wave's lanes and the waves.  6554 tokens x 4 rows of 2880 bf16, 325 MB: 60 us (5.4 TB/s; 77
// with one position after the other and a barrier for each).
template <int DT, int RT, int KB, int S>
__global__ __launch_bounds__(512) void merge_backward_kernel(MergeBackJob m) {
  __shared__ float s_dot[2][8][KB];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, waves = blockDim.x >> 6;
  int par = 0;
  for (int t = blockIdx.x; t < m.T; t += gridDim.x) {
    const char* dout = row_at<DT>(m.dout, t, m.dout_pitch);
    const Named r = named_rows(m.pos, m.w, m.err, t, m.K, m.n_rows, lane);
    for (int k0 = 0; k0 < m.K; k0 += KB, par ^= 1) {
      float dot[KB], w[KB];
      int p[KB];
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        dot[k] = 0.f;
        p[k] = lane_i32(r.p, k0 + k);
        w[k] = lane_f32(r.w, k0 + k);
      }
      for (int ch = threadIdx.x; ch < m.chunks; ch += blockDim.x) {
        Chunk<RT> q[KB];
        Chunk<DT> d;
        d.template load<(S >= kReadOnce)>(dout, (int64_t)ch * 8);
        if (m.dw) {
#pragma unroll
          for (int k = 0; k < KB; ++k)
            if (p[k] >= 0) q[k].template load<(S >= kReadOnce)>(row_at<RT>(m.rows, p[k], m.row_pitch), (int64_t)ch * 8);
        }
        float g[8];
        d.get(g);
        if (m.drows) {
#pragma unroll
          for (int k = 0; k < KB; ++k) {
            if (p[k] < 0) continue;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = g[e] * w[k];
            st8<RT, S == kThrough>((char*)m.drows + (int64_t)p[k] * m.drows_pitch * (RT == MOE_F32 ? 4 : 2), (int64_t)ch * 8, f);
          }
        }
        if (m.dw) {
#pragma unroll
          for (int k = 0; k < KB; ++k) {
            if (p[k] < 0) continue;
            float f[8];
            q[k].get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) dot[k] = fmaf(g[e], f[e], dot[k]);
          }
        }
      }
      if (!m.dw) continue;
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const float s = wave_sum(dot[k]);
        if (lane == 0) s_dot[par][wv][k] = s;
      }
      __syncthreads();
      if (threadIdx.x < KB && k0 + (int)threadIdx.x < m.K) {
        float s = 0.f;
        for (int v = 0; v < waves; ++v) s += s_dot[par][v][threadIdx.x];
        m.dw[(int64_t)t * m.K + k0 + threadIdx.x] = s;
      }
    }
  }
}

template <int RT, int OT, int KB>
static int merge_launch(const MergeJob& m, hipStream_t stream) {
  const int64_t bytes = (int64_t)m.T * m.H * (m.K * dtype_size(RT) + dtype_size(OT));
  const unsigned grid = grid_of(m.T), block = row_threads(m.chunks);
  switch (stream_kind(bytes)) {
    case kThrough: return launch(merge_kernel<RT, OT, KB, kThrough>, grid, block, stream, m);
    case kReadOnce: return launch(merge_kernel<RT, OT, KB, kReadOnce>, grid, block, stream, m);
    default: return launch(merge_kernel<RT, OT, KB, kNear>, grid, block, stream, m);
  }
}
template <int RT, int OT>
static int merge_by_k(const MergeJob& m, hipStream_t stream) {
  if (m.K <= 2) return merge_launch<RT, OT, 2>(m, stream);
  if (m.K <= 4) return merge_launch<RT, OT, 4>(m, stream);
  return merge_launch<RT, OT, 8>(m, stream);
}
template <int DT, int RT, int KB>
static int merge_backward_launch(const MergeBackJob& m, hipStream_t stream) {
  const int sides = (m.dw != nullptr) + (m.drows != nullptr);
  const int64_t bytes = (int64_t)m.T * m.H * (m.K * sides * dtype_size(RT) + dtype_size(DT));
  const unsigned grid = grid_of(m.T), block = row_threads(m.chunks);
  switch (stream_kind(bytes)) {
    case kThrough: return launch(merge_backward_kernel<DT, RT, KB, kThrough>, grid, block, stream, m);
    case kReadOnce: return launch(merge_backward_kernel<DT, RT, KB, kReadOnce>, grid, block, stream, m);
    default: return launch(merge_backward_kernel<DT, RT, KB, kNear>, grid, block, stream, m);
  }
}
template <int DT, int RT>
static int merge_backward_by_k(const MergeBackJob& m, hipStream_t stream) {
  if (m.K <= 2) return merge_backward_launch<DT, RT, 2>(m, stream);
  if (m.K <= 4) return merge_backward_launch<DT, RT, 4>(m, stream);
  return merge_backward_launch<DT, RT, 8>(m, stream);
}

constexpr int64_t kMaxPitch = (int64_t)1 << 32;

static bool row_size_ok(int32_t T, int32_t K, int32_t H) {
  return T >= 0 && T <= (1 << 24) && K >= 1 && K <= kMaxK && (int64_t)T * K <= (1 << 24) && H >= 1 && H <= kHMaxRows;
}
static bool pitch_ok(int64_t pitch, int32_t H) { return pitch >= H && pitch <= kMaxPitch; }
static bool f32_or_bf16(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }

}  // namespace moe

using namespace moe;

extern "C" size_t moe_sort_rows_workspace_size(int32_t n_max) {
  return n_max > kShortAny ? (size_t)kSegs * kMaxEloc * sizeof(int32_t) : 0;
}

static int check_sort(const moe_sort_rows_args* a) {
  if (!row_size_ok(a->T, a->K, a->H) || a->E_loc < 1 || a->E_loc > kMaxEloc) return MOE_EINVAL_SIZE;
  if (a->xs) {
    if (a->x_dtype != MOE_FP8_E4M3 && !f32_or_bf16(a->x_dtype)) return MOE_EINVAL_DTYPE;
    if (a->H % 8) return MOE_EINVAL_SHAPE;
    if (!pitch_ok(a->x_pitch, a->H) || !pitch_ok(a->xs_pitch, a->H)) return MOE_EINVAL_SIZE;
    if (a->x_dtype == MOE_FP8_E4M3 && a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128)
      return MOE_EINVAL_SIZE;
  }
  if (!a->counts || !a->offsets || !a->err) return MOE_EINVAL_NULL;
  if (a->T == 0) return MOE_OK;
  if (!a->expert || !a->pos) return MOE_EINVAL_NULL;
  if (a->xs) {
    if (!a->x || (a->x_dtype == MOE_FP8_E4M3 && !a->x_scale)) return MOE_EINVAL_NULL;
    const int out = a->x_dtype == MOE_F32 ? MOE_F32 : MOE_BF16;
    if (!aligned_rows(a->x, a->x_pitch, dtype_size(a->x_dtype), chunk_align(a->x_dtype)) ||
        !aligned_rows(a->xs, a->xs_pitch, dtype_size(out), 16))
      return MOE_EINVAL_ALIGN;
  }
  const size_t need = moe_sort_rows_workspace_size(a->T * a->K);
  if (need) {
    if (!a->workspace || a->workspace_bytes < need) return MOE_EWORKSPACE;
    if (!aligned16(a->workspace)) return MOE_EINVAL_ALIGN;
  }
  return MOE_OK;
}

static CopyJob make_copy_job(const moe_sort_rows_args* a) {
  CopyJob c;
  c.K = a->K; c.H = a->H;
  c.chunks = a->xs ? a->H / 8 : 0;
  c.group_shift = a->group ? __builtin_ctz((unsigned)a->group) : -1;
  c.groups = a->group ? (a->H + a->group - 1) / a->group : 1;
  c.x = a->x; c.x_pitch = a->x_pitch; c.x_scale = a->x_scale;
  c.xs = a->xs; c.xs_pitch = a->xs_pitch;
  return c;
}

template <int DT>
static int sort_rows(const moe_sort_rows_args* a, const SortJob& j, hipStream_t stream) {
  const CopyJob c = make_copy_job(a);
  const unsigned block = c.chunks ? row_threads(c.chunks) : 256;
  if (j.n <= kShort && (int64_t)j.T * j.n <= kShortWork) {
    const unsigned b = block < 256 ? 256 : block;
    return launch(sort_short_kernel<DT>, (unsigned)j.T + 1, b, stream, j, c);
  }
  const int per = (j.n + kSegs - 1) / kSegs, seg_len = (per + kIdx - 1) / kIdx * kIdx;
  const int segs = (j.n + seg_len - 1) / seg_len;
  int rc = launch(sort_count_kernel, (unsigned)segs, kIdx, stream, j, seg_len, (int32_t*)a->workspace);
  if (rc == MOE_OK)
    rc = launch(sort_place_kernel, (unsigned)segs, kIdx, stream, j, segs, seg_len, (const int32_t*)a->workspace);
  if (rc != MOE_OK || !c.chunks) return rc;
  // NT stores from where the rows do not stay near (stream_kind), but plain loads: x is a Kth of the
  // bytes and was written just before (NT loads too took 104 us where plain ones take 91).  Rows of
  // 2880 bf16 to four experts each, microseconds plain / NT stores, alone and with a reader of xs
  // after it: 16384 rows 30.0 / 25.1 and 48.0 / 52.0, 32768 rows 51.7 / 42.5 and 94.3 / 92.8, 65536 rows
  // 95.6 / 87.1 and 181.4 / 173.9.
  const int64_t bytes = ((int64_t)j.n * (DT == MOE_F32 ? 4 : 2) + (int64_t)j.T * dtype_size(DT)) * a->H;
  return launch(stream_kind(bytes) == kThrough ? sort_copy_kernel<DT, true> : sort_copy_kernel<DT, false>,
                grid_of(j.T), block, stream,
                c, j.T, (const int32_t*)a->pos);
}

extern "C" int moe_sort_rows(const moe_sort_rows_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  const int rc = check_sort(a);
  if (rc != MOE_OK) return rc;
  const int n = a->T * a->K;
  SortJob j;
  j.T = a->T; j.K = a->K; j.n = n; j.base = a->expert_base; j.E_loc = a->E_loc;
  j.expert = a->expert; j.perm = a->perm; j.pos = a->pos; j.counts = a->counts; j.offsets = a->offsets;
  j.row_slot = a->row_slot; j.err = a->err;
  if (n == 0) return launch(sort_empty_kernel, 1, 256, stream, j);
  if (!a->xs || a->x_dtype == MOE_BF16) return sort_rows<MOE_BF16>(a, j, stream);
  if (a->x_dtype == MOE_F32) return sort_rows<MOE_F32>(a, j, stream);
  return sort_rows<MOE_FP8_E4M3>(a, j, stream);
}

extern "C" int moe_merge_rows(const moe_merge_rows_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  if (!row_size_ok(a->T, a->K, a->H) || a->n_rows < 0) return MOE_EINVAL_SIZE;
  if (!f32_or_bf16(a->row_dtype) || !f32_or_bf16(a->out_dtype)) return MOE_EINVAL_DTYPE;
  if (a->H % 8) return MOE_EINVAL_SHAPE;
  if (!pitch_ok(a->row_pitch, a->H) || !pitch_ok(a->out_pitch, a->H)) return MOE_EINVAL_SIZE;
  if (!a->err) return MOE_EINVAL_NULL;
  if (a->T == 0) return MOE_OK;
  if (!a->pos || !a->out || (a->n_rows > 0 && !a->rows)) return MOE_EINVAL_NULL;
  if (!aligned_rows(a->rows, a->row_pitch, dtype_size(a->row_dtype), 16) ||
      !aligned_rows(a->out, a->out_pitch, dtype_size(a->out_dtype), 16))
    return MOE_EINVAL_ALIGN;
  MergeJob m;
  m.T = a->T; m.K = a->K; m.H = a->H; m.chunks = a->H / 8;
  m.rows = a->rows; m.row_pitch = a->row_pitch; m.n_rows = a->n_rows;
  m.pos = a->pos; m.w = a->w; m.out = a->out; m.out_pitch = a->out_pitch; m.err = a->err;
  if (a->row_dtype == MOE_F32)
    return a->out_dtype == MOE_F32 ? merge_by_k<MOE_F32, MOE_F32>(m, stream) : merge_by_k<MOE_F32, MOE_BF16>(m, stream);
  return a->out_dtype == MOE_F32 ? merge_by_k<MOE_BF16, MOE_F32>(m, stream) : merge_by_k<MOE_BF16, MOE_BF16>(m, stream);
}

extern "C" int moe_merge_rows_backward(const moe_merge_rows_backward_args* a, hipStream_t stream) {
  if (!a) return MOE_EINVAL_NULL;
  if (!row_size_ok(a->T, a->K, a->H) || a->n_rows < 0) return MOE_EINVAL_SIZE;
  if (!f32_or_bf16(a->row_dtype) || !f32_or_bf16(a->dout_dtype)) return MOE_EINVAL_DTYPE;
  if (a->H % 8) return MOE_EINVAL_SHAPE;
  if (!pitch_ok(a->dout_pitch, a->H) || (a->dw && !pitch_ok(a->row_pitch, a->H)) ||
      (a->drows && !pitch_ok(a->drows_pitch, a->H)))
    return MOE_EINVAL_SIZE;
  if (!a->err) return MOE_EINVAL_NULL;
  if (a->T == 0) return MOE_OK;
  if (!a->drows && !a->dw) return MOE_EINVAL_NULL;
  if (!a->dout || !a->pos || (a->dw && a->n_rows > 0 && !a->rows)) return MOE_EINVAL_NULL;
  if (!aligned_rows(a->dout, a->dout_pitch, dtype_size(a->dout_dtype), 16) ||
      (a->dw && !aligned_rows(a->rows, a->row_pitch, dtype_size(a->row_dtype), 16)) ||
      (a->drows && !aligned_rows(a->drows, a->drows_pitch, dtype_size(a->row_dtype), 16)))
    return MOE_EINVAL_ALIGN;
  MergeBackJob m;
  m.T = a->T; m.K = a->K; m.H = a->H; m.chunks = a->H / 8;
  m.dout = a->dout; m.dout_pitch = a->dout_pitch; m.rows = a->rows; m.row_pitch = a->row_pitch;
  m.n_rows = a->n_rows; m.pos = a->pos; m.w = a->w; m.drows = a->drows; m.drows_pitch = a->drows_pitch;
  m.dw = a->dw; m.err = a->err;
  if (a->dout_dtype == MOE_F32)
    return a->row_dtype == MOE_F32 ? merge_backward_by_k<MOE_F32, MOE_F32>(m, stream)
                                   : merge_backward_by_k<MOE_F32, MOE_BF16>(m, stream);
  return a->row_dtype == MOE_F32 ? merge_backward_by_k<MOE_BF16, MOE_F32>(m, stream)
                                 : merge_backward_by_k<MOE_BF16, MOE_BF16>(m, stream);
}
