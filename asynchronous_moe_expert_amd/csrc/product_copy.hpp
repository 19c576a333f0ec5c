// What the kernels that copy their operands straight into LDS share (product_tiles.hip, product_narrow.hip).
#pragma once

#include <type_traits>
#include <utility>

#include "products.hpp"

namespace moe {

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;

constexpr int kStep = 64;  // a step's k: 64 bf16 or 128 codes, 128 bytes of a row either way
constexpr int kMaxBlocks = kHMaxRows / 128;  // scales of a row
static __device__ u32x4 g_zeros;  // what lanes past a contraction's end copy

// A wave's copy of 64 x 16 (or 64 x 4) bytes to LDS, lane after lane from dst on.  In inline assembly, so that
// the compiler does not put waits of its own before every LDS read that might meet a copy (it tells the copies of
// a few instructions apart, and a tile has more); the waits are wait_copies and meet below.  The address is
// read when the copy is issued, and nothing is returned to a register.  m0, which the copies take their place in LDS
// from, is named as written so that none of them comes between a value that the compiler puts there and its use (it
// warns that it would not keep one in m0 across the statement, which is as well).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ uint32_t lds_at(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
template <int AT = 0>
__device__ __forceinline__ void copy16(const char* src, uint32_t dst) {
  asm volatile("s_add_u32 m0, %1, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(dst), "n"(AT)
               : "memory", "scc", "m0");
}
template <int AT = 0>
__device__ __forceinline__ void copy16(const char* base, uint32_t off, uint32_t dst) {  // base in scalar registers
  asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(dst), "n"(AT)
               : "memory", "scc", "m0");
}
__device__ __forceinline__ void copy16_once(const char* base, uint32_t off, uint32_t dst) {  // non-temporal
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(off), "s"(base), "s"(dst)
               : "memory", "m0");
}
__device__ __forceinline__ void copy4(const char* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(dst) : "memory", "m0");
}
#pragma clang diagnostic pop
template <typename F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {  // f(0) .. f(N - 1), with constants
  each_of(f, std::make_integer_sequence<int, N>{});
}

template <int N>
__device__ __forceinline__ void wait_copies() {  // at most N of this wave's copies are still on their way
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8)); }
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// A 16 x 16 block's sums over 128 columns of codes.  The matrix unit adds 8-bit products (in the form for 32 columns as
// in that for 128) eight at a time and cuts each 13 bits below the largest of the eight; those sums it adds in fp32 (found
// by sums of 2^16, -2^16 and 2^(16 - d): exact to d = 13 within eight columns, to d = 23 beyond).  With 7 terms cut by less
// than 2^-13 of the largest, an element is off by less than 2^-10 of the sum of its terms' sizes; codes of normal numbers
// leave 1.3e-6 of that sum and 1.3e-5 of the outputs' norm, whatever D is, one column of 128 that is 300 times as large as
// the others 8e-5 of the sum.  For bf16 outputs, whose own rounding is 1.7e-3 of the norm, that is taken for its rate; for
// fp32 ones the codes are widened to bf16, which is exact, and multiplied as such, summed in fp32 (3.5e-8 to 1.1e-7 of the
// norm).  32 experts of 512 rows, 4096 x 4096: 321 to 370 us by the codes' values, and 676; 8 of 32, 5760 x 2880: 25 and 29.
template <int DT>
__device__ __forceinline__ f32x4 dot128(i32x8 a, i32x8 b) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if constexpr (DT == MOE_FP8_E4M3) {
    v = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, v, 0, 0, 0, 0, 0, 0);
  } else {
    const auto widened = [](i32x8 c, int i) {  // codes 8 i .. 8 i + 7
      u32x4 w;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const auto lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)c[2 * i + k], 1.f, false);
        const auto hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)c[2 * i + k], 1.f, true);
        __builtin_memcpy((char*)&w + 8 * k, &lo, 4);
        __builtin_memcpy((char*)&w + 8 * k + 4, &hi, 4);
      }
      bf16x8 r;
      __builtin_memcpy(&r, &w, 16);
      return r;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widened(a, i), widened(b, i), v, 0, 0, 0);
  }
  return v;
}

// One tile's place: rows of C p0 .. pend - 1 of expert e (-1: no tile) from column q0, contraction k0 .. kend - 1; mt: the
// 16 rows of C that each half of the workgroup takes, as many times.
struct Place {
  int e, p0, pend, q0, k0, kend, mt;
};

__device__ __forceinline__ const char* uniform_ptr(const char* p) {
  const uint64_t v = (uint64_t)p;
  return (const char*)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v) |
                       (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32);
}

// Lane groups g hold columns 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3 of a row, two values to a register; after it
// they hold columns 8 g .. 8 g + 7, 16 bytes that can be stored at once.
__device__ __forceinline__ void neighbours(u32x4& v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto h = __builtin_amdgcn_permlane32_swap(v[i], v[2 + i], false, false);
    const auto r = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
    v[i] = r[0];
    v[2 + i] = r[1];
  }
}

// NB blocks of 64 columns of an operand whose rows lie across k: byte offsets of this lane's copies from row k0 of
// the matrix, two copies to a block, of row() and of the row 32 further.  Columns past the end are read at others.
template <int NB>
struct Across {
  uint32_t off[NB];
  __device__ __forceinline__ void set(int wq, int lane, int col0, int cols, int64_t pitch, int es) {
    const int k = row(wq, lane), f = ((k >> 1) & 1) | ((k >> 3) & 1) << 1, piece = (lane & 7) ^ (2 * f);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int first = col0 + 64 * b < cols ? col0 + 64 * b : col0 < cols ? col0 : 0;
      off[b] = (uint32_t)(k * (int)pitch * es + (first + min(piece * 8, cols - 8 - first)) * es);
    }
  }
  static __device__ __forceinline__ int row(int wq, int lane) { return 8 * wq + (lane >> 3); }
  // step `step` of the contraction's rows 0 .. end - 1, which begin at base
  __device__ __forceinline__ void copy(const char* base, int64_t pitch_bytes, uint32_t dst, int step, int end, int wq,
                                       int lane) const {
    const char* from = uniform_ptr(base + (int64_t)step * kStep * pitch_bytes);
    const char* odd = uniform_ptr(from + 32 * pitch_bytes);
    if ((step + 1) * kStep <= end) {
      each<2 * NB>([&](auto c) { copy16<c() * 4096>(c() & 1 ? odd : from, off[c() >> 1], dst); });
    } else {
      const int k = step * kStep + row(wq, lane);
      each<2 * NB>([&](auto c) {
        const char* src = (c() & 1 ? odd : from) + off[c() >> 1];
        copy16<c() * 4096>(k + 32 * (c() & 1) < end ? src : (const char*)&g_zeros, dst);
      });
    }
  }
};

// Lanes 2 r and 2 r + 1 hold a 16-byte piece of the first 64 bytes (a) and of the second (b) of rows 2 r and 2 r + 1;
// after it a is a piece of row 2 r and b of row 2 r + 1, of the first 64 bytes in even lanes and of the second in odd
// ones, so that eight lanes store a line of 128 bytes at once.
template <typename V>
__device__ __forceinline__ void pair_rows(V& a, V& b, bool odd) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x, y;
    __builtin_memcpy(&x, (const char*)&a + 4 * i, 4);
    __builtin_memcpy(&y, (const char*)&b + 4 * i, 4);
    const uint32_t got = dpp_u32<kDppXor1>(odd ? x : y);
    x = odd ? got : x;
    y = odd ? y : got;
    __builtin_memcpy((char*)&a + 4 * i, &x, 4);
    __builtin_memcpy((char*)&b + 4 * i, &y, 4);
  }
}

}  // namespace moe
