// Append to the paged 4-bit cache with the norms and the rotation on the way
// (vq_kivi_paged_append), and the stored tokens read back
// (vq_kivi_paged_dequantize).
//
// Per new token: queries normed, rotated and written out; keys normed,
// rotated, rounded to fp16 and quantized; values rounded to fp16 and
// quantized.  Groups of g channels of one token, as the value groups of the
// contiguous cache: scale = (max - min) / 15 and code = rint((x - min) /
// scale) in fp32, scale and min stored in fp16.
//
// LPR = D / 16 lanes hold a row.  A rotated key row passes through shared
// memory so that its lanes hold 16 neighbouring channels, as a value row's
// do: a group is then g / 16 neighbouring lanes, whatever the rotation.
#include "paged.cuh"
#include "paged_words.cuh"
#include "vqk_internal.cuh"

namespace vqk {
namespace {

constexpr int kThreads = 128;
constexpr unsigned kFull = 0xffffffffu;

// two fp16 of two fp32; values beyond the type's range (infinities too) become
// its largest, NaN stays NaN
__device__ __forceinline__ uint32_t half2_sat(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ __half2 as_half2(uint32_t u) {
  return *reinterpret_cast<const __half2 *>(&u);
}

// 8 channels as stored in fp16, saturated as above
template <typename T>
__device__ __forceinline__ void to_half8(const uint4 &r, uint32_t (&h)[4]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __half>::value) {
      const __half2 top = as_half2(0x7bff7bffu), low = as_half2(0xfbfffbffu);
      const __half2 x = __hmax2_nan(__hmin2_nan(as_half2(w[i]), top), low);
      h[i] = *reinterpret_cast<const uint32_t *>(&x);
    } else {
      h[i] = half2_sat(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
}

// smallest and largest of a group, whose 16-channel pieces lie in g / 16
// neighbouring lanes; NaN where one of its values is
__device__ __forceinline__ __half2 group_range(const uint32_t (&h)[8], int g) {
  __half2 lo = as_half2(h[0]), hi = lo;
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    lo = __hmin2_nan(lo, as_half2(h[e]));
    hi = __hmax2_nan(hi, as_half2(h[e]));
  }
  __half l = __hmin_nan(__low2half(lo), __high2half(lo));
  __half u = __hmax_nan(__low2half(hi), __high2half(hi));
  for (int o = 1; o < (g >> 4); o <<= 1) {
    const __half2 x = __shfl_xor_sync(kFull, __halves2half2(l, u), o);
    l = __hmin_nan(l, __low2half(x));
    u = __hmax_nan(u, __high2half(x));
  }
  return __halves2half2(l, u);
}

// Codes of 16 channels of a group from lo in steps of `scale`, 4 bits each,
// the first lowest: rint((x - lo) / scale) with the quotient rounded to fp32.
// The product with the reciprocal is off by less than 2^-21 of a quotient of
// at most 15; only where it comes within 2^-12 of a tie (|t - rint(t)| near
// 1/2) can the two round to different codes, and there the division decides.
__device__ __forceinline__ void codes16(const uint32_t (&x)[8], float lo, float scale,
                                        uint32_t (&w)[2]) {
  constexpr float kMagic = 12582912.f;      // 1.5 * 2^23: its sum's low bits are rint
  const float inv = __fdividef(1.f, scale);
  const float2 lo2 = make_float2(-lo, -lo), inv2 = make_float2(inv, inv);
  const float2 up2 = make_float2(kMagic, kMagic), down2 = make_float2(-kMagic, -kMagic);
  float off = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t acc = 0u;
#pragma unroll
    for (int e = 3; e >= 0; --e) {
      const float2 d = __fadd2_rn(__half22float2(as_half2(x[4 * h + e])), lo2);
      const float2 t = __fmul2_rn(d, inv2);
      const float2 r = __fadd2_rn(t, up2);
      const float2 i = __fadd2_rn(r, down2);
      off = fmaxf(off, fmaxf(fabsf(t.x - i.x), fabsf(t.y - i.y)));
      acc = acc * 16u + __float_as_uint(r.y);
      acc = acc * 16u + __float_as_uint(r.x);
    }
    // 0x4B400000 (kMagic's bits) times 1 + 16 + ... + 16^7, modulo 2^32
    w[h] = acc - 0x3f400000u;
  }
  if (off > 0.5f - 0.000244140625f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t acc = 0u;
#pragma unroll
      for (int e = 3; e >= 0; --e) {
        const float2 v = __half22float2(as_half2(x[4 * h + e]));
        acc = acc * 16u + (uint32_t)(int)rintf((v.y - lo) / scale);
        acc = acc * 16u + (uint32_t)(int)rintf((v.x - lo) / scale);
      }
      w[h] = acc;
    }
  }
}

// One row's 16 neighbouring channels x per lane, quantized and stored in the
// block `blk` at token tl.  `poison`: the token's key or
// value row holds a NaN.  A key row then gets NaN zeros, so that the scores
// of every query that sees the token are NaN; a value row is stored as
// zeros, because a masked token's weight of 0 times NaN would reach rows
// that do not see it.
template <int D, bool VALUES>
__device__ __forceinline__ void quantize_row(const uint32_t (&x)[8], __half2 range, int g, int l,
                                             bool poison, uint8_t *blk, int tl) {
  const float lo = __low2float(range) + 0.f;            // -0 to +0
  const float scale = (__high2float(range) - lo) / 15.f;
  uint32_t w[2] = {0u, 0u};
  if (scale > 0.f && !poison) codes16(x, lo, scale, w);
  __half s = __float2half_rn(scale), z = __float2half_rn(lo);
  // code 15 must stay inside fp16's range (it rounds to infinity from 65520)
  if (fmaf(15.f, __half2float(s), lo) >= 65520.f)
    s = __ushort_as_half((unsigned short)(__half_as_ushort(s) - 1));
  if (poison) {
    s = __float2half_rn(0.f);
    z = VALUES ? s : __ushort_as_half((unsigned short)0x7fff);
  }
  constexpr int I = D / 32;
  if (VALUES) {
    // quads 4 (l % 2) ... + 3 of the 32-channel span l / 2
    uint8_t *p = blk + off_vc(D, g) + 2 * (tl & 1) +
                 4 * (((8 * (tl >> 3) + 4 * (l & 1)) * 4 + ((tl & 7) >> 1)) * I + (l >> 1));
#pragma unroll
    for (int n = 0; n < 4; ++n)
      *reinterpret_cast<uint16_t *>(p + 16 * I * n) =
          (uint16_t)(w[n >> 1] >> (16 * (n & 1)));
  } else {
    // words 2 l and 2 l + 1 of the row: span l / 2, quarter 2 (l % 2) and next
    uint32_t *p = reinterpret_cast<uint32_t *>(blk + tl * (D / 2)) + 2 * (l & 1) * I + (l >> 1);
    p[0] = w[0];
    p[I] = w[1];
  }
  if ((l & ((g >> 4) - 1)) == 0) {
    __half *m = reinterpret_cast<__half *>(blk + (VALUES ? off_vm(D, g) : off_km(D))) +
                ((tl >> 1) * (D / g) + 16 * l / g) * 4 + (tl & 1);
    m[0] = s;
    m[2] = z;
  }
}

// A warp serves a token (with few tokens `parts` warps do), 32 / LPR rows at a
// time: first the query rows, then the key and value rows of as many kv
// heads.  The next rows' loads are in flight while these are worked on, and
// the first ones while the token's place is looked up.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 5)
k_paged_append(PagedArgs a, HeadRows q, HeadRows k, HeadRows v, RopeArgs r,
               bool rotate_by_place, float eps, int parts) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  __shared__ __align__(16) __half rows[kThreads / 32][RPW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR, l = lane % LPR;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + warp;
  const int64_t t = w / parts;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int p0, p1;
  chunk_places(r, l, p0, p1);
  const int gq = (q.heads + RPW - 1) / RPW, gk = (a.H_kv + RPW - 1) / RPW;
  uint4 xa[1] = {}, xb[1] = {}, va[1] = {}, vb[1] = {};
  auto fetch = [&](int gi) {
    const bool isk = gi >= gq;
    const HeadRows &h = isk ? k : q;
    const int row = (isk ? gi - gq : gi) * RPW + sub;
    if (t < a.tokens && gi < gq + gk && row < h.heads) {
      const T *x = static_cast<const T *>(h.x) + t * h.x_token + row * h.x_head;
      load8<T>(x + p0, xa);
      load8<T>(x + p1, xb);
      if (isk) {
        const T *y = static_cast<const T *>(v.x) + t * v.x_token + row * v.x_head + 16 * l;
        load8<T>(y, va);
        load8<T>(y + 8, vb);
      }
    }
  };
  int gi = (int)(w % parts);
  fetch(gi);
  const Place at = find_place(a, t, t < a.tokens ? -1 : 32 * (w - a.tokens * parts) + lane);
  if (at.pos < 0) return;
  // the token's page, looked up while the rows arrive
  const bool stores = gi + (gq + gk - 1 - gi) / parts * parts >= gq;
  const int page = stores ? a.table[(int64_t)at.b * a.table_stride + (at.pos >> a.page_log2)] : 0;
  float c[8], s[8];
  rope_angles<LPR>(r, [&](int ax) -> long long {
    if (rotate_by_place) return at.pos;
    const int64_t i = (int64_t)ax * r.pos_stride + t;
    return r.pos64 ? static_cast<const long long *>(r.pos)[i]
                   : (long long)static_cast<const int *>(r.pos)[i];
  }, lane, c, s);
  const bool good = (unsigned)page < (unsigned)a.n_pages;
  if (!good && lane == 0) atomicOr(a.status, kBadPage);

  const void *held = nullptr;
  uint4 wa[1] = {}, wb[1] = {};
  for (; gi < gq + gk; gi += parts) {
    const bool isk = gi >= gq;
    const HeadRows &h = isk ? k : q;
    const int row = (isk ? gi - gq : gi) * RPW + sub;
    const bool valid = row < h.heads;
    float x0[8], x1[8];
    unpack8<T>(xa, x0);
    unpack8<T>(xb, x1);
    uint32_t y[8];
    if (isk) {
      uint32_t y0[4], y1[4];
      to_half8<T>(va[0], y0);
      to_half8<T>(vb[0], y1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] = y0[e];
        y[4 + e] = y1[e];
      }
    }
    fetch(gi + parts);
    if (h.weight) {
      if (held != h.weight) {
        held = h.weight;
        load8<T>(static_cast<const T *>(h.weight) + p0, wa);
        load8<T>(static_cast<const T *>(h.weight) + p1, wb);
      }
      float w0[8], w1[8];
      unpack8<T>(wa, w0);
      unpack8<T>(wb, w1);
      norm_row<T, LPR>(x0, x1, w0, w1, D, eps);
    }
    if (8 * l < r.half) rotate_row(r.interleaved, c, s, x0, x1);
    if (!isk) {
      if (valid) {
        T *o = static_cast<T *>(q.out) + t * q.out_token + row * q.out_head;
        store8<T>(o + p0, x0);
        store8<T>(o + p1, x1);
      }
      continue;
    }
    // the key row's lanes change from rotated pairs to neighbouring channels
    __syncwarp();
    *reinterpret_cast<uint4 *>(&rows[warp][sub][p0]) =
        make_uint4(half2_sat(x0[0], x0[1]), half2_sat(x0[2], x0[3]), half2_sat(x0[4], x0[5]),
                   half2_sat(x0[6], x0[7]));
    *reinterpret_cast<uint4 *>(&rows[warp][sub][p1]) =
        make_uint4(half2_sat(x1[0], x1[1]), half2_sat(x1[2], x1[3]), half2_sat(x1[4], x1[5]),
                   half2_sat(x1[6], x1[7]));
    __syncwarp();
    const uint4 k0 = *reinterpret_cast<const uint4 *>(&rows[warp][sub][16 * l]),
                k1 = *reinterpret_cast<const uint4 *>(&rows[warp][sub][16 * l + 8]);
    const uint32_t x[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
    const __half2 xr = group_range(x, a.g), yr = group_range(y, a.g);
    // a NaN of any group of the token's key or value row
    const unsigned mask = ((1u << LPR) - 1u) << (sub * LPR);
    const bool poison =
        (__ballot_sync(kFull, __hisnan(__low2half(xr)) || __hisnan(__low2half(yr))) & mask) != 0u;
    uint8_t *blk = nullptr;
    if (valid && good)
      blk = a.pool + ((((int64_t)page * a.H_kv + row) << (a.page_log2 - 4)) +
                      ((at.pos & ((1 << a.page_log2) - 1)) >> 4)) *
                         paged_block_bytes(D, a.g);
    if (!blk) continue;
    quantize_row<D, false>(x, xr, a.g, l, poison, blk, at.pos & 15);
    quantize_row<D, true>(y, yr, a.g, l, poison, blk, at.pos & 15);
  }
}

// the 8 values of a word of codes, lowest nibble first: code * s + z, each
// rounded once (1024 + code and 1024 + 16 code are one logic operation from the
// word, both steps to the code are exact)
__device__ __forceinline__ uint4 word_row(uint32_t w, __half2 s, __half2 z) {
  const __half2 k1024 = bits_h2(0x64006400u), k16 = bits_h2(0x2c002c00u),
                k64 = bits_h2(0xd400d400u);
  uint32_t v[4];                      // values (r, r + 4)
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    v[2 * j] = h2_bits(__hfma2(__hsub2(field<0x000f000fu>(w), k1024), s, z));
    v[2 * j + 1] = h2_bits(__hfma2(__hfma2(field<0x00f000f0u>(w), k16, k64), s, z));
    w >>= 8;
  }
  return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                    __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

// Four lanes a token, eight tokens a warp: lane t4 has the words t4 of the key
// row and, of the value words, the token's halves of two neighbouring quads of
// channels, which together read as a key word does; so channels 32 i + 8 t4 ...
// of both rows, 16 bytes a store.  Neighbouring tokens share the value words'
// sectors.  Bound: HBM, four bytes out per byte in, and the latency of the
// loads (16384 tokens of 8 kv heads, D = 128, g = 64: 86 MB in 15.8 us; with a
// token's halves loaded one by one 25.3).
template <int D, int NG>
__global__ void __launch_bounds__(kThreads)
k_paged_dequantize(PagedArgs a, __half *K, __half *V, int parts) {
  constexpr int I = D / 32, G = D / NG, BLK = paged_block_bytes(D, G);
  const int lane = threadIdx.x & 31, t4 = lane & 3;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t groups = (a.tokens + 7) / 8, t = w / parts * 8 + (lane >> 2);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Place at{-1, -1};
  if (w >= groups * parts) at = find_place(a, a.tokens, 32 * (w - groups * parts) + lane);
  else if (t < a.tokens) at = find_place(a, t, -1);
  if (at.pos < 0) return;
  const uint8_t *blk = find_block(a, at.b, at.pos, 0, BLK);
  if (!blk) return;
  const int tl = at.pos & 15;
  const unsigned half = (tl & 1) ? 0x7632u : 0x5410u, twice = (tl & 1) ? 0x3232u : 0x1010u;
  const int64_t head = (int64_t)BLK << (a.page_log2 - 4);
#pragma unroll 2
  for (int h = (int)(w % parts); h < a.H_kv; h += parts) {
    const uint8_t *b = blk + h * head;
    uint32_t k[I], v0[I], v1[I];
    uint2 km[NG], vm[NG];
    const uint8_t *vw = b + off_vc(D, G) +
                        ((8 * (tl >> 3) + 2 * t4) * 4 + ((tl & 7) >> 1)) * (4 * I);
    load_words<I>(b + tl * (D / 2) + t4 * (4 * I), k);
    load_meta<NG>(b + off_km(D) + (tl >> 1) * (8 * NG), km);
    load_words<I>(vw, v0);
    load_words<I>(vw + 16 * I, v1);
    load_meta<NG>(b + off_vm(D, G) + (tl >> 1) * (8 * NG), vm);
    const int64_t row = (t * a.H_kv + h) * D + 8 * t4;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const uint2 m = km[32 * i / G], n = vm[32 * i / G];
      *reinterpret_cast<uint4 *>(K + row + 32 * i) =
          word_row(k[i], bits_h2(__byte_perm(m.x, 0u, twice)), bits_h2(__byte_perm(m.y, 0u, twice)));
      *reinterpret_cast<uint4 *>(V + row + 32 * i) =
          word_row(__byte_perm(v0[i], v1[i], half), bits_h2(__byte_perm(n.x, 0u, twice)),
                   bits_h2(__byte_perm(n.y, 0u, twice)));
    }
  }
}

// warps per token: enough for about 16 per SM, at most one per row group
int parts_for(int64_t tokens, int groups, int sm_count) {
  int64_t p = (int64_t)sm_count * 16 / (tokens > 0 ? tokens : 1);
  return (int)(p < 1 ? 1 : (p > groups ? groups : p));
}

// those and the ones that only look at sequences (find_place)
int64_t warps_for(const PagedArgs &a, int parts) {
  return a.tokens * parts + (a.cu ? (a.B + 31) / 32 : 0);
}

template <typename T, int D>
cudaError_t launch_append(const PagedArgs &a, const HeadRows &q, const HeadRows &k,
                          const HeadRows &v, const RopeArgs &r, bool by_place, float eps,
                          int sm_count, cudaStream_t st) {
  constexpr int RPW = 32 / (D / 16);
  const int groups = (q.heads + RPW - 1) / RPW + (a.H_kv + RPW - 1) / RPW;
  const int parts = parts_for(a.tokens, groups, sm_count);
  const int64_t wpc = kThreads / 32;
  cudaError_t e = launch_pdl(k_paged_append<T, D>,
                             dim3((unsigned)((warps_for(a, parts) + wpc - 1) / wpc)),
                             dim3(kThreads), 0, st, a, q, k, v, r, by_place, eps, parts);
  count_launch();
  return e;
}

}  // namespace

cudaError_t launch_paged_append(int dtype, const PagedArgs &a, const HeadRows &q,
                                const HeadRows &k, const HeadRows &v, const RopeArgs &r,
                                bool by_place, int D, float eps, int sm_count,
                                cudaStream_t st) {
  if (dtype == VQ_F16)
    return D == 64 ? launch_append<__half, 64>(a, q, k, v, r, by_place, eps, sm_count, st)
                   : launch_append<__half, 128>(a, q, k, v, r, by_place, eps, sm_count, st);
  return D == 64
             ? launch_append<__nv_bfloat16, 64>(a, q, k, v, r, by_place, eps, sm_count, st)
             : launch_append<__nv_bfloat16, 128>(a, q, k, v, r, by_place, eps, sm_count, st);
}

template <int D, int NG>
static cudaError_t dequantize_d(const PagedArgs &a, __half *K, __half *V, int sm_count,
                                cudaStream_t st) {
  const int64_t groups = (a.tokens + 7) / 8, wpc = kThreads / 32;
  int64_t parts = (int64_t)sm_count * 32 / groups;
  parts = parts < 1 ? 1 : (parts > a.H_kv ? a.H_kv : parts);
  // and warps that only look at sequences (find_place)
  const int64_t warps = groups * parts + (a.cu ? (a.B + 31) / 32 : 0);
  cudaError_t e = launch_pdl(k_paged_dequantize<D, NG>, dim3((unsigned)((warps + wpc - 1) / wpc)),
                             dim3(kThreads), 0, st, a, K, V, (int)parts);
  count_launch();
  return e;
}

cudaError_t launch_paged_dequantize(const PagedArgs &a, __half *K, __half *V, int D,
                                    int sm_count, cudaStream_t st) {
  const int ng = D / a.g;
  if (D == 64)
    return ng == 1 ? dequantize_d<64, 1>(a, K, V, sm_count, st)
                   : dequantize_d<64, 2>(a, K, V, sm_count, st);
  return ng == 1   ? dequantize_d<128, 1>(a, K, V, sm_count, st)
         : ng == 2 ? dequantize_d<128, 2>(a, K, V, sm_count, st)
                   : dequantize_d<128, 4>(a, K, V, sm_count, st);
}

}  // namespace vqk
