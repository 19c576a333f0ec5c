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
// read when the copy is issued, and nothing is returned to a register.
__device__ __forceinline__ uint32_t lds_at(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
template <int AT = 0>
__device__ __forceinline__ void copy16(const char* src, uint32_t dst) {
  asm volatile("s_add_u32 m0, %1, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(dst), "n"(AT)
               : "memory", "scc");
}
template <int AT = 0>
__device__ __forceinline__ void copy16(const char* base, uint32_t off, uint32_t dst) {  // base in scalar registers
  asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(dst), "n"(AT)
               : "memory", "scc");
}
__device__ __forceinline__ void copy16_once(const char* base, uint32_t off, uint32_t dst) {  // non-temporal
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(off), "s"(base), "s"(dst)
               : "memory");
}
__device__ __forceinline__ void copy4(const char* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(dst) : "memory");
}
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

}  // namespace moe
