// Values held in 8 bits: the codes of a cache and the 16-bit operands that they become.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/attn_paged.h"

namespace attn {

// Four codes (one word, lowest byte first) as two pairs of f16 operands, exactly:
// int8 and e4m3 both fit its 11 bits and its range.  A0, A1 are the bytes that the first
// pair holds, B0, B1 the second.
template <int FMT>
struct F16Codes;

template <>
struct F16Codes<ATTN_CODES_INT8> {
  static constexpr int A0 = 0, A1 = 2, B0 = 1, B1 = 3;
  // 0x6400 | (x + 128) is the f16 number 1024 + 128 + x
  static __device__ __forceinline__ uint32_t pair(uint32_t bytes) {
    uint32_t y, z;
    // (bytes & mask) ^ bias: one operation, where two constants in C became two
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(y) : "r"(bytes), "r"(0x00ff00ffu), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(z) : "r"(y), "r"(0x64806480u));
    return z;
  }
  static __device__ __forceinline__ void unpack(uint32_t w, uint32_t &p0, uint32_t &p1) {
    p0 = pair(w);
    p1 = pair(w >> 8);
  }
  static constexpr uint32_t LOW = 0x5410, HIGH = 0x7632;      // a0 a1 b0 b1, a2 a3 b2 b3
};

template <>
struct F16Codes<ATTN_CODES_E4M3> {
  static constexpr int A0 = 0, A1 = 1, B0 = 2, B1 = 3;
  static __device__ __forceinline__ void unpack(uint32_t w, uint32_t &p0, uint32_t &p1) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(p0), "=r"(p1)
        : "r"(w));
  }
  static constexpr uint32_t LOW = 0x5140, HIGH = 0x7362;      // a0 b0 a1 b1, a2 b2 a3 b3
};

// Four codes each of two rows: p[i] is the pair (a's i-th, b's i-th).
template <int FMT>
__device__ __forceinline__ void across(uint32_t a, uint32_t b, uint32_t (&p)[4]) {
  using C = F16Codes<FMT>;
  C::unpack(__byte_perm(a, b, C::LOW), p[0], p[1]);
  C::unpack(__byte_perm(a, b, C::HIGH), p[2], p[3]);
}

}  // namespace attn
