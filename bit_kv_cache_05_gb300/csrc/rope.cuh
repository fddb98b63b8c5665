// Rows of heads: 16-byte loads and stores of fp16 / bf16 / fp32, the RMS norm
// of a head and its rotation by position.  Shared by the norm-and-rotate
// kernel (rope.cu) and the paged append (paged_append.cu).
//
// Lanes: a row of D channels is held by LPR lanes (D / 16 of them active),
// each with two chunks of 8 channels chosen so that both channels of a
// rotated pair sit in one lane:
//   half split   chunks at 8 l and half + 8 l (pairs (i, i + half))
//   interleaved  chunks at 16 l and 16 l + 8 (pairs (2 i, 2 i + 1))
// and the channels behind the rotated ones in 16-channel runs.
//
// Angles: a pair's frequency is a fraction of a turn per position in 64-bit
// fixed point (turns * 2^64), so position * frequency mod 1 is one 64-bit
// integer product, exact for every position: the error of an angle is
// position * 2^-65 turns, where position * inv_freq in fp32 loses the angle
// at positions in the thousands (2^-24 relative).  Cosine and sine of the
// fraction are Taylor series on an eighth of a turn either side of a quarter,
// summed so that little more than their last rounding is left: a key next to
// an fp16 rounding border, or a code next to a tie, falls on its own side as
// often as fp32 allows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

namespace vqk {

// one tensor's heads: element strides, last dimension contiguous
struct HeadRows {
  const void *x = nullptr;
  void *out = nullptr;
  const void *weight = nullptr;   // [D], nullptr: no norm
  int64_t x_token = 0, x_head = 0, out_token = 0, out_head = 0;
  int heads = 0;
};

struct RopeArgs {
  const unsigned long long *turns = nullptr;   // [half]
  const uint8_t *axis = nullptr;               // [half] or nullptr (axis 0)
  const void *pos = nullptr;                   // [axes][tokens]
  int64_t pos_stride = 0;                      // elements between axes
  int half = 0;                                // rotated pairs (0: none)
  int interleaved = 0;
  int pos64 = 0;                               // positions are int64
  int axes = 1;
  float scale = 1.f;                           // factor of cos and sin
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 (&r)[sizeof(T) == 4 ? 2 : 1],
                                        float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[4 * i] = __uint_as_float(r[i].x);
      v[4 * i + 1] = __uint_as_float(r[i].y);
      v[4 * i + 2] = __uint_as_float(r[i].z);
      v[4 * i + 3] = __uint_as_float(r[i].w);
    }
  } else {
    const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      } else {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
}

// the 8 channels at p, still as stored
template <typename T>
__device__ __forceinline__ void load8(const T *p, uint4 (&r)[sizeof(T) == 4 ? 2 : 1]) {
#pragma unroll
  for (int i = 0; i < (sizeof(T) == 4 ? 2 : 1); ++i)
    r[i] = reinterpret_cast<const uint4 *>(p)[i];
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// channels of lane l's two chunks
__device__ __forceinline__ void chunk_places(const RopeArgs &r, int l, int &p0, int &p1) {
  if (8 * l < r.half && !r.interleaved) {
    p0 = 8 * l;
    p1 = r.half + 8 * l;
  } else {
    p0 = 16 * l;   // behind the rotated channels too: half / 8 lanes hold 2 half
    p1 = p0 + 8;
  }
}

// cos and sin of a / 2^64 turns
__device__ __forceinline__ void turn_cos_sin(unsigned long long a, float &c, float &s) {
  // the nearest quarter, and what is left of it: r in [-1/8, 1/8) turns
  const unsigned quarter = (unsigned)((a + (1ull << 61)) >> 62);
  const long long r = (long long)(a - ((unsigned long long)quarter << 62));
  // x = 2 pi r / 2^64 as xh + xl
  const int top = (int)(r >> 32);
  const float f = (float)top;
  const float g = (float)(top - (int)f) + (float)(unsigned)r * 2.3283064365386963e-10f;
  constexpr float kh = 1.4629180792671596e-09f;    // 2 pi / 2^32 in fp32
  constexpr float kl = -4.0709404e-17f;            // and what is left of it
  const float xh = f * kh;
  const float xl = fmaf(f, kh, -xh) + fmaf(g, kh, f * kl);
  const float z = xh * xh, zl = fmaf(xh, xh, -z) + 2.f * xh * xl;
  float p = fmaf(z, -2.5052108e-8f, 2.7557319e-6f);          // -1/11!, 1/9!
  p = fmaf(z, p, -1.9841270e-4f);                            // -1/7!
  p = fmaf(z, p, 8.3333333e-3f);                             // 1/5!
  p = fmaf(z, p, -1.6666667e-1f);                            // -1/3!
  const float sx = xh + fmaf(xh * z, p, fmaf(xl, -0.5f * z, xl));
  float q = fmaf(z, 2.0876757e-9f, -2.7557319e-7f);          // 1/12!, -1/10!
  q = fmaf(z, q, 2.4801587e-5f);                             // 1/8!
  q = fmaf(z, q, -1.3888889e-3f);                            // -1/6!
  q = fmaf(z, q, 4.1666667e-2f);                             // 1/4!
  const float w = fmaf(z, -0.5f, 1.f);
  const float cx = w + fmaf(z * z, q, fmaf(zl, -0.5f, fmaf(z, -0.5f, 1.f - w)));
  c = quarter & 1u ? sx : cx;
  s = quarter & 1u ? cx : sx;
  if (quarter == 1u || quarter == 2u) c = -c;
  if (quarter & 2u) s = -s;
}

// cos and sin of the 8 pairs 8 l ... 8 l + 7 of a lane (1 and 0 behind the
// rotated pairs).  The 32 / LPR rows of a warp share a token and so their
// angles: each lane works out its share and the warp exchanges them.
// `at(axis)` is the token's position on an axis.
template <int LPR, typename At>
__device__ __forceinline__ void rope_angles(const RopeArgs &r, At at, int lane, float (&c)[8],
                                            float (&s)[8]) {
  constexpr int RPW = 32 / LPR, PER = 8 / RPW;
  const int sub = lane / LPR, l = lane % LPR;
  float mc[PER], ms[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int f = 8 * l + sub * PER + j;
    mc[j] = 1.f;
    ms[j] = 0.f;
    if (f < r.half) {
      turn_cos_sin((unsigned long long)at(r.axis ? (int)r.axis[f] : 0) * r.turns[f], mc[j],
                   ms[j]);
      mc[j] *= r.scale;
      ms[j] *= r.scale;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c[e] = __shfl_sync(0xffffffffu, mc[e % PER], (e / PER) * LPR + l);
    s[e] = __shfl_sync(0xffffffffu, ms[e % PER], (e / PER) * LPR + l);
  }
}

// RMS norm of a row held by LPR lanes (all lanes of the warp take part).  Of
// fp16 rows the product with the weight is exact in fp32 (22 bits, no
// overflow) and comes first; bf16 and fp32 rows could leave its range.
template <typename T, int LPR>
__device__ __forceinline__ void norm_row(float (&x0)[8], float (&x1)[8], const float (&w0)[8],
                                         const float (&w1)[8], int D, float eps) {
  // four short sums, so that a square meets few roundings
  float p[4] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e & 3] = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], p[e & 3]));
  float ss = (p[0] + p[1]) + (p[2] + p[3]);
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  // one Newton step with its residual in two parts: the factor of a whole row
  // is off by little more than its last rounding
  const float m = ss / (float)D + eps, r = rsqrtf(m);
  const float h = m * r, rest = fmaf(-h, r, 1.f) - fmaf(m, r, -h) * r;
  const float inv = m > 0.f && r > 0.f ? fmaf(0.5f * r, rest, r) : r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (std::is_same<T, __half>::value) {
      x0[e] = x0[e] * w0[e] * inv;
      x1[e] = x1[e] * w1[e] * inv;
    } else {
      x0[e] = x0[e] * inv * w0[e];
      x1[e] = x1[e] * inv * w1[e];
    }
  }
}

__device__ __forceinline__ void rotate_row(bool interleaved, const float (&c)[8],
                                           const float (&s)[8], float (&x0)[8],
                                           float (&x1)[8]) {
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = x0[2 * j], b = x0[2 * j + 1];
      x0[2 * j] = a * c[j] - b * s[j];
      x0[2 * j + 1] = b * c[j] + a * s[j];
      const float d = x1[2 * j], e = x1[2 * j + 1];
      x1[2 * j] = d * c[4 + j] - e * s[4 + j];
      x1[2 * j + 1] = e * c[4 + j] + d * s[4 + j];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = x0[e], b = x1[e];
      x0[e] = a * c[e] - b * s[e];
      x1[e] = b * c[e] + a * s[e];
    }
  }
}

}  // namespace vqk
