// The experts' products for few rows of each expert: a pass over the weights.
#include <type_traits>

#include "product_copy.hpp"

namespace moe {

// A workgroup of NW waves takes up to 16 MT rows and 32 NW columns of C and walks along k with S steps in a ring of
// LDS, S - 1 of them on their way while one is multiplied.  Such a product is a pass over the weights, whose rate is
// what the chip has on its way over the latency (2 to 2.5 us when HBM is busy), so the shapes are chosen to have
// much on its way on all CUs:
//   WK = 1, NW = 4, S = 3: two workgroups to a CU, for calls of many of them;
//   WK = 1, NW = 4, 6 or 8, S = 6, 4 or 3: one to a CU and more steps, for calls whose workgroups all run at
//           once; run_narrow chooses the NW that leaves the fewest CUs idle;
//   WK = 4: 32 columns, a step is four times as long, each wave takes its quarter and the waves' sums are added at
//           the end: for calls that would leave most CUs idle.
// Fragments lie in LDS as the tiles' do (product_tiles.hip).  256 rows of 8 experts, 5760 x 2880, other weights each
// time: 45 us in bf16 (the weights at 6.0 TB/s), 34 in 8 bits (4.0: rows of 2880 bytes, whose steps are parts of two
// lines each), back to back 42 and 25 (some of the weights are still in the last-level cache then); 128 experts
// of two rows, 2880 x 2880 bf16: 352 (6.0).
template <int MODE, int DT, int WK, int NW, int S>
struct Narrow {
  static constexpr int es = esize<DT>();
  static constexpr int kWaves = NW, kStages = S;
  static constexpr int kQ = 32 * NW / WK;         // columns
  static constexpr int kMT = WK == 1 ? 4 : 2;     // 16 rows each, at most
  static constexpr bool kAlong = MODE == kForward, kScaled = esize<DT>() == 1;
  static constexpr int kQBytes = 4096 * NW;
  static constexpr int kStage = kQBytes + WK * kMT * 2048;  // bytes: Q, then P
  static_assert(kAlong || NW == 4, "blocks of 64 columns are shared out among four waves");
  static_assert(WK == 1 || NW == WK, "");
};

template <typename T, int MODE, int DT, int WK, int MT>
__device__ __forceinline__ void narrow_tile(const ProductJob& j, const Place& at, char* ring, float* scales, const float* wsc,
                                            int wv, int lane, bool once) {
  constexpr int es = T::es, NW = T::kWaves, kStages = T::kStages;
  constexpr int kP = WK == 1 ? (2 * MT + NW - 1) / NW : 2 * MT, kCopies = 4 + kP + (T::kScaled ? 1 : 0);
  static_assert((kStages - 2) * kCopies < 64, "a wave's copies are counted in six bits");
  const int g = lane >> 4, l16 = lane & 15, sub = WK == 1 ? 0 : wv;
  const int pieces = j.D * es / 16, steps = (pieces + 8 * WK - 1) / (8 * WK);

  // ---- copies.  P: instruction c of a wave fills rows 8 i .. 8 i + 7, i = NW c + wv (WK = 4: of its own quarter, i =
  // c); where the waves do not share them out evenly some are made twice
  auto p_rows = [&](int c) { return WK == 1 ? (NW * c + wv) % (2 * MT) : c; };
  uint32_t poff[kP], nosrc = 0;
  int ppiece[kP];
#pragma unroll
  for (int c = 0; c < kP; ++c) {
    const int r = 8 * p_rows(c) + (lane >> 3);
    const int row = min(at.p0 + r, at.pend - 1);
    int64_t slot = row;
    if (j.row_slot) {
      slot = j.row_slot[row];
      if (slot < 0 || slot >= j.x_rows) {
        atomicOr(j.err, MOE_ERR_SLOT_RANGE);
        slot = 0;
        nosrc |= 1u << c;
      }
    }
    ppiece[c] = (lane & 7) ^ ((r >> 1) & 7);
    poff[c] = (uint32_t)(slot * (j.x_pitch * es / 16) + ppiece[c]);
  }
  const float* sptr = nullptr;
  if constexpr (T::kScaled) {
    const int row = min(at.p0 + min(lane, 16 * MT - 1), at.pend - 1);
    const int64_t slot = j.row_slot ? j.row_slot[row] : row;
    if (slot >= 0 && slot < j.x_rows) sptr = j.x_scale + slot * ((j.D + 127) / 128);
  }
  uint32_t qoff[2];
  int qpiece = 0;
  const char* q = (const char*)j.w + (at.e * j.w_stride + (T::kAlong ? (int64_t)at.q0 * j.w_pitch : 0)) * es;
  if constexpr (T::kAlong) {  // rows 8 i .., i = NW c + wv (WK = 4: i = c): bits 3 and 4 of the row are i's lowest
    qoff[0] = (uint32_t)((lane >> 3) * (int)j.w_pitch * es);
  } else {  // blocks of 64 columns, rows 8 (i % 8) .. of block i / 8
    const int k = 8 * wv + (lane >> 3), f = ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
    qpiece = (lane & 7) ^ (2 * f);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int first = at.q0 + 64 * b < j.N ? at.q0 + 64 * b : at.q0;
      qoff[b] = (uint32_t)(k * (int)j.w_pitch * es + (first + min(qpiece * 8, j.N - 8 - first)) * es);
    }
  }
  auto copy = [&](int step) {
    const int slot = step % kStages;
    const uint32_t dst = lds_at(ring) + slot * T::kStage;
    const int first = (step * WK + sub) * 8;  // this wave's first piece of a row
    const bool whole = first + 8 <= pieces;
    if constexpr (T::kAlong) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int i = WK == 1 ? NW * c + wv : c, r = 8 * i;
        const int piece = (lane & 7) ^ (((lane >> 4) & 1) | 2 * (i & 3));
        const char* from = uniform_ptr(q + (int64_t)first * 16 + (at.q0 + r < j.N ? r : 0) * j.w_pitch * es);
        const uint32_t to = dst + (WK == 1 ? i : 4 * wv + c) * 1024;
        if (whole && once) copy16_once(from, qoff[0] + piece * 16, to);
        else if (whole) copy16(from, qoff[0] + piece * 16, to);
        else copy16(first + piece < pieces ? from + (qoff[0] + piece * 16) : (const char*)&g_zeros, to);
      }
    } else {
      const char* from = uniform_ptr(q + (int64_t)step * kStep * j.w_pitch * es);
      const char* odd = uniform_ptr(from + 32 * j.w_pitch * es);
      const int k = step * kStep + 8 * wv + (lane >> 3);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t to = dst + (4 * c + wv) * 1024;
        if ((step + 1) * kStep <= j.D) copy16(c & 1 ? odd : from, qoff[c >> 1], to);
        else copy16(k + 32 * (c & 1) < j.D ? (c & 1 ? odd : from) + qoff[c >> 1] : (const char*)&g_zeros, to);
      }
    }
    const char* p = uniform_ptr((const char*)j.x + (int64_t)first * 16);
#pragma unroll
    for (int c = 0; c < kP; ++c) {
      const uint32_t to = dst + T::kQBytes + (WK == 1 ? p_rows(c) * 1024 : wv * (T::kMT * 2048) + c * 1024);
      copy16(first + ppiece[c] < pieces && !(nosrc >> c & 1) ? p + (uint64_t)poff[c] * 16 : (const char*)&g_zeros, to);
    }
    if constexpr (T::kScaled)
      copy4(sptr && first < pieces ? (const char*)(sptr + step * WK + sub) : (const char*)&g_zeros,
            lds_at(scales) + (slot * WK + sub) * 256);
  };

  // ---- fragments
  const int pr = l16 * 128 + ((g ^ ((l16 >> 1) & 7)) << 4);
  const int qcol = WK == 1 ? wv * 32 : 0;  // this wave's columns
  const int qr = qcol * 128 + (8 * (l16 >> 2) + (l16 & 3)) * 128 + ((g ^ (((l16 >> 1) & 1) | ((l16 >> 1) & 6))) << 4);
  const int tr = (qcol >> 6) * 8192 + (8 * g + (l16 >> 2)) * 128 + ((((l16 >> 3) & 1) | (g & 1) << 1) << 5) + (l16 & 3) * 8;
  f32x4 acc[MT][2];
#pragma unroll
  for (int a = 0; a < MT; ++a) acc[a][0] = acc[a][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](int step) {
    const char* st = ring + (step % kStages) * T::kStage;
    const char* qs = st + (WK == 1 ? 0 : wv * 4096);
    const char* ps = st + T::kQBytes + (WK == 1 ? 0 : wv * (T::kMT * 2048));
    u32x4 qf[2][2], pf[MT][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if constexpr (T::kAlong) {
          qf[b][s] = *reinterpret_cast<const u32x4*>(qs + (qr ^ (s * 64)) + b * 512);
        } else {
          const char* from = qs + (tr ^ (((qcol & 32) >> 4) + b) << 5) + s * 4096;
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(from));
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(from + 512));
          __builtin_memcpy(&qf[b][s], &lo, 8);
          __builtin_memcpy((char*)&qf[b][s] + 8, &hi, 8);
        }
      }
#pragma unroll
      for (int a = 0; a < MT; ++a) pf[a][s] = *reinterpret_cast<const u32x4*>(ps + (pr ^ (s * 64)) + a * 2048);
    }
    if constexpr (T::kScaled) {
      const float sw = wsc[(((at.q0 + qcol) >> 7) - (at.q0 >> 7)) * kMaxBlocks + step * WK + sub];
      const float* ss = scales + ((step % kStages) * WK + sub) * 64;
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        const float s = ss[a * 16 + l16] * sw;
        i32x8 p;
        __builtin_memcpy(&p, &pf[a][0], 32);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          i32x8 w;
          __builtin_memcpy(&w, &qf[b][0], 32);
          const f32x4 v = dot128<DT>(w, p);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[a][b][i] = fmaf(v[i], s, acc[a][b][i]);
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            bf16x8 p, w;
            __builtin_memcpy(&p, &pf[a][s], 16);
            __builtin_memcpy(&w, &qf[b][s], 16);
            acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, p, acc[a][b], 0, 0, 0);
          }
    }
  };

  // ---- The copies of step i + S - 1 go where step i - 1 was, which every wave has read when it has met the others
  // at step i (each wave has copied and read its own quarter where WK = 4).  Steps past the end copy zeros: the
  // counts that the waits go by stay the same.
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) copy(i);
#pragma clang loop unroll(disable)
  for (int i = 0; i < steps; ++i) {
    wait_copies<(kStages - 2) * kCopies>();
    wait_lds();
    if constexpr (WK == 1) meet();
    else asm volatile("" ::: "memory");
    copy(i + kStages - 1);
    multiply(i);
    asm volatile("" ::: "memory");
  }
  wait_copies<0>();

  if constexpr (WK > 1) {  // the waves' sums, added in their order
    __syncthreads();
    f32x4* part = reinterpret_cast<f32x4*>(ring);
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) part[((a * 2 + b) * 4 + wv) * 64 + lane] = acc[a][b];
    __syncthreads();
    if (wv < 2 * MT) {
      f32x4 v = part[wv * 4 * 64 + lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) v += part[(wv * 4 + w) * 64 + lane];
      const int p = at.p0 + (wv >> 1) * 16 + l16, col = at.q0 + 8 * g + 4 * (wv & 1);
      if (p < at.pend && col < j.N) put4(j, p * j.out_pitch + col, v);
    }
    return;
  }
#pragma unroll
  for (int a = 0; a < MT; ++a) {
    const int p = at.p0 + a * 16 + l16;
    if (j.out_f32) {
      if (p >= at.pend) continue;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int col = at.q0 + qcol + (T::kAlong ? 8 * g + 4 * b : 16 * b + 4 * g);
        if (col < j.N) put4(j, p * j.out_pitch + col, acc[a][b]);
      }
    } else {
      u32x4 v = {pack_bf16x2(acc[a][0][0], acc[a][0][1]), pack_bf16x2(acc[a][0][2], acc[a][0][3]),
                 pack_bf16x2(acc[a][1][0], acc[a][1][1]), pack_bf16x2(acc[a][1][2], acc[a][1][3])};
      if constexpr (!T::kAlong) neighbours(v);
      const int col = at.q0 + qcol + 8 * g;
      if (p < at.pend && col < j.N) *reinterpret_cast<u32x4*>((uint16_t*)j.out + p * j.out_pitch + col) = v;
    }
  }
}

template <int MODE, int DT, int WK, int NW, int S>
__global__ __launch_bounds__(64 * NW) void narrow_kernel(ProductJob j) {
  using T = Narrow<MODE, DT, WK, NW, S>;
  __shared__ __attribute__((aligned(1024))) char ring[S * T::kStage];
  __shared__ float scales[T::kScaled ? S * WK * 64 : 1], wsc[T::kScaled ? 2 * kMaxBlocks : 1];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kRows = 16 * T::kMT;
  const int ct = (j.N + T::kQ - 1) / T::kQ;
  const RowTiles<kRows> all(j, lane);
  const int total = all.total() * ct;
  // an XCD's workgroups take a contiguous part of the tiles: an expert's row tiles of one column block after the
  // other, so that the weights of the second one are found in its L2
  const int xcd = blockIdx.x % 8, u0 = (int)((int64_t)total * xcd / 8), u1 = (int)((int64_t)total * (xcd + 1) / 8);
  // the grid has a workgroup for every tile but where offsets give rows to several experts (without the loop such tiles
  // would be left out; 256 rows of 8 experts, 5760 x 2880: 44 us without, 45 with it)
  for (int u = u0 + (int)(blockIdx.x / 8); u < u1; u += (int)(gridDim.x / 8)) {
    if (u >= u0 + (int)(gridDim.x / 8)) __syncthreads();  // the tile before is out of LDS
    int e, base, n;
    all.find(u, ct, e, base, n);
    int r0, r1;
    expert_rows(j, e, r0, r1);
    const int v = u - base * ct;
    Place at;
    at.e = e;
    at.p0 = __builtin_amdgcn_readfirstlane(r0 + v % n * kRows);
    at.q0 = v / n * T::kQ;
    at.pend = __builtin_amdgcn_readfirstlane(min(r1, at.p0 + kRows));
    at.k0 = 0;
    at.kend = j.D;
    if constexpr (T::kScaled) {  // the scales of the one block of columns, or of the two that the columns lie in
      const int kb = (j.D + 127) / 128, nb = (j.N + 127) / 128;
#pragma unroll
      for (int b = 0; b < (128 % T::kQ ? 2 : 1); ++b) {
        const float* from = j.w_scale + ((int64_t)e * nb + min((at.q0 >> 7) + b, nb - 1)) * kb;
        for (int k = threadIdx.x; k < (kb + WK - 1) / WK * WK; k += 64 * NW)  // (quarters past the end: times 0)
          wsc[b * kMaxBlocks + k] = k < kb ? from[k] : 0.f;
      }
      __syncthreads();
    }
    // Weights that no other workgroup reads pass through the caches without staying (256 rows of 8 experts, 5760 x 2880
    // bf16 from HBM: 50 us with cached copies, 44 so), unless a step's 128 bytes of a row are parts of two lines, which
    // the next step wants again (the same in 8 bits, rows of 2880 bytes: 31 us cached, 33 so).
    const bool once = n == 1 && (j.w_pitch * T::es) % 128 == 0 && (j.w_stride * T::es) % 128 == 0 && ((uint64_t)j.w & 127) == 0;
    const int rows = at.pend - at.p0;
    if (rows <= kRows / 2) narrow_tile<T, MODE, DT, WK, T::kMT / 2>(j, at, ring, scales, wsc, wv, lane, once);
    else narrow_tile<T, MODE, DT, WK, T::kMT>(j, at, ring, scales, wsc, wv, lane, once);
  }
}

template <int MODE, int DT, int WK, int NW, int S>
static int launch_narrow(const ProductJob& j, hipStream_t stream) {
  using T = Narrow<MODE, DT, WK, NW, S>;
  const int64_t rt = j.n / (16 * T::kMT) + (j.n < j.E ? j.n : j.E), ct = (j.N + T::kQ - 1) / T::kQ;
  return launch(narrow_kernel<MODE, DT, WK, NW, S>, (unsigned)((rt * ct + 7) / 8 * 8), 64u * NW, stream, j);
}

// The number of workgroups is guessed from as many experts with rows as there can be, a row tile to each.
template <int MODE, int DT>
static int choose_narrow(const ProductJob& j, int64_t cus, hipStream_t stream) {
  const int64_t experts = j.n < j.E ? j.n : j.E;
  const auto units = [&](int nw) { return experts * ((j.N + 32 * nw - 1) / (32 * nw)); };
  if constexpr (MODE == kForward) {
    if (2 * units(4) <= cus) return launch_narrow<MODE, DT, 4, 4, 3>(j, stream);
    // one workgroup to a CU: the least work on the busiest one, the widest of equals
    int best = 8;
    int64_t cost = (units(8) + cus - 1) / cus * 8;
    for (int nw : {6, 4}) {
      const int64_t c = (units(nw) + cus - 1) / cus * nw;
      if (c < cost) {
        best = nw;
        cost = c;
      }
    }
    if (units(best) <= cus) {
      if (best == 8) return launch_narrow<MODE, DT, 1, 8, 3>(j, stream);
      if (best == 6) return launch_narrow<MODE, DT, 1, 6, 4>(j, stream);
      return launch_narrow<MODE, DT, 1, 4, 6>(j, stream);
    }
  }
  return launch_narrow<MODE, DT, 1, 4, 3>(j, stream);
}

int run_narrow(const ProductJob& j, int dtype, int mode, int cus, hipStream_t stream) {
  if (dtype == MOE_FP8_E4M3)
    return j.out_f32 ? choose_narrow<kForward, kFp8Wide>(j, cus, stream) : choose_narrow<kForward, MOE_FP8_E4M3>(j, cus, stream);
  if (mode == kRowsGrad) return choose_narrow<kRowsGrad, MOE_BF16>(j, cus, stream);
  return choose_narrow<kForward, MOE_BF16>(j, cus, stream);
}

}  // namespace moe
