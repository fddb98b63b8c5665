// What both attention kernels of the paged cache read a block with: the words
// of codes and of (scale, zero), and the way from a word to fp16 pairs.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace vqk {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) {
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ __half2 bits_h2(uint32_t u) {
  return *reinterpret_cast<const __half2 *>(&u);
}

// (w & mask) | 0x64006400 in one instruction: 0x6400 | c is 1024 + c
template <uint32_t mask>
__device__ __forceinline__ __half2 field(uint32_t w) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "n"(mask), "r"(0x64006400u));
  return bits_h2(d);
}

// the (scale, zero) words of a token pair, all groups
template <int NG>
__device__ __forceinline__ void load_meta(const unsigned char *p, uint2 (&m)[NG]) {
  if constexpr (NG == 1) {
    m[0] = *reinterpret_cast<const uint2 *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) {
      const uint4 x = reinterpret_cast<const uint4 *>(p)[i];
      m[2 * i] = make_uint2(x.x, x.y);
      m[2 * i + 1] = make_uint2(x.z, x.w);
    }
  }
}

template <int I>
__device__ __forceinline__ void load_words(const unsigned char *p, uint32_t (&w)[I]) {
  if constexpr (I == 4) {
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    w[0] = x.x; w[1] = x.y;
  }
}

}  // namespace vqk
