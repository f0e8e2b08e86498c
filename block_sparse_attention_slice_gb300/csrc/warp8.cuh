// Steps of the warp-level kernels over pages in 8 bits.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace attn {

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds4(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
// An 8 x 8 matrix of 16-bit values, two neighbours of a row a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float pow2_of(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }   // -126 <= e <= 127

// A row's weights w = p vs become f16 times 2^lc, -113 <= lc <= 126, and O holds 2^lc times
// their sums.  p <= 2^8, so w is formed first, in f32, where it is finite for every vs up to 2^119; the
// power of two comes last, once it suits: 2^lc vs alone would leave f32 where lc was raised for
// tiny values and large ones follow.
// The largest w that 2^lc suits: 2^(15 - lc), infinity at -113.
__device__ __forceinline__ float most_at(int lc) { return __uint_as_float(static_cast<uint32_t>(142 - lc) << 23); }
// Fits lc to w, the largest weight of the keys at hand, and `top`, the largest that was looked at
// before, less what the row's maximum has grown by since: down where w is too large, up where
// both are below 2^-lc; the larger then comes to 2^7 .. 2^8.  Rising by what O holds as well as by
// w keeps O in range: it never comes to more than 2^23 times codes and keys.  Returns O's factor.
__device__ __forceinline__ float refit(float w, float &top, int &lc) {
  const float t = fmaxf(top, w);
  float f = 1.f;
  if (w > most_at(lc) || (t > 0.f && t < pow2_of(-lc))) {
    int by = min(max(134 - static_cast<int>(__float_as_uint(t) >> 23), -113), 126) - lc;
    if (top > 0.f) by = min(by, 126);        // 0: O is 0, or below 2^-24 of what comes
    f = by < -126 ? 0.f : pow2_of(min(by, 126));
    lc += by;
  }
  top = t;
  return f;
}

}  // namespace attn
