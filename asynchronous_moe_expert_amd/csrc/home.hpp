// Device helpers of the home rank's operators (route.hip, rows.hip, norm.hip): eight elements of
// a row as fp32 in registers, sums and maxima over lanes, and launches that report their own error.
#pragma once

#include "common.hpp"

namespace moe {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

// Loads and stores of rows come in two kinds.  NT (non-temporal) ones pass through the caches
// without staying: they move large arrays faster, but what they wrote is not near for a next kernel.
template <bool NT, typename V>
__device__ __forceinline__ V ld(const V* p) {
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool NT, typename V>
__device__ __forceinline__ void st(V* p, V v) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// A row is handled in chunks of eight elements: 16 bytes of bf16, two 16-byte runs of fp32, 8
// bytes of fp8.  load and st8 take the element offset of the chunk from the row's start.
template <int DT>
struct Chunk;

template <>
struct Chunk<MOE_BF16> {
  u32x4 r;
  template <bool NT = false>
  __device__ __forceinline__ void load(const void* row, int64_t at) {
    r = ld<NT>(reinterpret_cast<const u32x4*>((const uint16_t*)row + at));
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(r[k] << 16);
      f[2 * k + 1] = __uint_as_float(r[k] & 0xffff0000u);
    }
  }
};

template <>
struct Chunk<MOE_F32> {
  f32x4 a, b;
  template <bool NT = false>
  __device__ __forceinline__ void load(const void* row, int64_t at) {
    a = ld<NT>(reinterpret_cast<const f32x4*>((const float*)row + at));
    b = ld<NT>(reinterpret_cast<const f32x4*>((const float*)row + at + 4));
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k] = a[k];
      f[4 + k] = b[k];
    }
  }
};

template <>
struct Chunk<MOE_FP8_E4M3> {
  u32x2 r;
  template <bool NT = false>
  __device__ __forceinline__ void load(const void* row, int64_t at) {
    r = ld<NT>(reinterpret_cast<const u32x2*>((const uint8_t*)row + at));
  }
  __device__ __forceinline__ void get(float* f) const {  // exact: every code is a bf16 value
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(r[0], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(r[0], true);
    const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(r[1], false), d = __builtin_amdgcn_cvt_pk_f32_fp8(r[1], true);
    f[0] = a[0]; f[1] = a[1]; f[2] = b[0]; f[3] = b[1];
    f[4] = c[0]; f[5] = c[1]; f[6] = d[0]; f[7] = d[1];
  }
};

// One rounding to the stored type, to nearest even.
template <int DT, bool NT = false>
__device__ __forceinline__ void st8(void* row, int64_t at, const float* f) {
  if constexpr (DT == MOE_F32) {
    float* p = (float*)row + at;
    st<NT>(reinterpret_cast<f32x4*>(p), f32x4{f[0], f[1], f[2], f[3]});
    st<NT>(reinterpret_cast<f32x4*>(p + 4), f32x4{f[4], f[5], f[6], f[7]});
  } else if constexpr (DT == MOE_BF16) {
    st<NT>(reinterpret_cast<u32x4*>((uint16_t*)row + at),
           u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])});
  } else {
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
    st<NT>(reinterpret_cast<u32x2*>((uint8_t*)row + at), u32x2{(uint32_t)lo, (uint32_t)hi});
  }
}

// Lane exchange inside rows of 16 lanes as DPP operands: lane ^ 1, lane ^ 2, then the mirrored
// lane of 8 and of 16 (which equal the other half's value once 4, then 8 lanes agree).
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v)));
}

// every lane of a row of 16 gets the row's sum / maximum / minimum (fixed order of additions)
__device__ __forceinline__ float sum16(float v) {
  v += dpp_f32<kDppXor1>(v);
  v += dpp_f32<kDppXor2>(v);
  v += dpp_f32<kDppHalfMirror>(v);
  v += dpp_f32<kDppMirror>(v);
  return v;
}
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, dpp_f32<kDppXor1>(v));
  v = fmaxf(v, dpp_f32<kDppXor2>(v));
  v = fmaxf(v, dpp_f32<kDppHalfMirror>(v));
  v = fmaxf(v, dpp_f32<kDppMirror>(v));
  return v;
}
__device__ __forceinline__ uint32_t max16u(uint32_t v) {
  v = max(v, dpp_u32<kDppXor1>(v));
  v = max(v, dpp_u32<kDppXor2>(v));
  v = max(v, dpp_u32<kDppHalfMirror>(v));
  v = max(v, dpp_u32<kDppMirror>(v));
  return v;
}
__device__ __forceinline__ uint32_t min16u(uint32_t v) {
  v = min(v, dpp_u32<kDppXor1>(v));
  v = min(v, dpp_u32<kDppXor2>(v));
  v = min(v, dpp_u32<kDppHalfMirror>(v));
  v = min(v, dpp_u32<kDppMirror>(v));
  return v;
}

__device__ __forceinline__ float lane_f32(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
// every lane of the wave gets its sum / maximum
__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  return (lane_f32(v, 0) + lane_f32(v, 16)) + (lane_f32(v, 32) + lane_f32(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
  v = max16(v);
  return fmaxf(fmaxf(lane_f32(v, 0), lane_f32(v, 16)), fmaxf(lane_f32(v, 32), lane_f32(v, 48)));
}

// A launch whose own return value is the status (an error left by an earlier call of someone
// else's is neither reported nor cleared).
template <typename... P, typename... A>
inline int launch(void (*kernel)(P...), unsigned grid, unsigned block, hipStream_t stream, A... args) {
  static_assert(sizeof...(P) == sizeof...(A), "one argument for each parameter");
  return [&](P... p) {
    void* list[] = {(void*)&p...};
    return hipLaunchKernel((const void*)kernel, dim3(grid), dim3(block), list, 0, stream) == hipSuccess ? MOE_OK
                                                                                                       : MOE_ELAUNCH;
  }(args...);
}

// Workgroups for as many units of work: kernels step by the grid, which has to stay below 2^32
// threads.
inline unsigned grid_of(int64_t units) { return (unsigned)(units < (1 << 20) ? units : 1 << 20); }

// a pointer and the bytes between its rows are multiples of `to`
inline bool aligned_rows(const void* p, int64_t pitch, int esz, int to) {
  return (uintptr_t)p % (unsigned)to == 0 && (pitch * esz) % to == 0;
}
// rows are read and written in chunks of eight elements, by 16 bytes where a chunk has as many
inline int chunk_align(int dt) { return dt == MOE_FP8_E4M3 ? 8 : 16; }

// How a call that reads and writes so many bytes of rows goes through the caches: kNear plain,
// kReadOnce with NT loads, kThrough with NT loads and stores.  Measured, microseconds alone / with a
// kernel after it that reads the output (merge: four rows of 2880 bf16 per token; norm: 4096 bf16 with
// its residual in and out):
//                              kNear          kReadOnce      kThrough
//   merge      56 MiB moved    11.9 /  19.0   13.7 /  21.1   12.5 /  23.0
//             112 MiB          26.7 /  33.3   24.9 /  32.5   23.3 /  34.6
//             225 MiB          49.4 /  60.1   46.4 /  56.7   44.1 /  57.4
//             450 MiB          94.5 / 115.1   90.9 / 109.8   85.7 / 109.5
//   its      101 MiB           23.0 /  31.9   20.9 /  31.5   21.7 /  35.2
//   gradient 202 MiB           44.1 /  64.4   37.0 /  56.9   41.0 /  64.8
//            405 MiB           85.0 / 120.7   84.4 / 119.4   80.2 / 123.4
//   norm       64 MiB          12.4 /  20.9   14.5 /  23.0   13.5 /  24.9
//             128 MiB          26.4 /  37.0   25.0 /  36.4   24.0 /  37.5
//             256 MiB          48.2 /  63.9   48.6 /  60.1   44.5 /  60.9
//             512 MiB          93.3 / 122.7   91.6 / 116.7   85.5 / 116.2
// Below 96 MiB what was written lately is still near and a plain load finds it; from about 256 MiB on,
// which the last-level cache holds, an output does not stay near anyway.
enum { kNear = 0, kReadOnce = 1, kThrough = 2 };
inline int stream_kind(int64_t bytes) {
  return bytes >= (220ll << 20) ? kThrough : bytes >= (96ll << 20) ? kReadOnce : kNear;
}

constexpr int kHMaxRows = 1 << 16;  // longest row of the row operators

}  // namespace moe
