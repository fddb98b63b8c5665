// Attention of few new tokens per sequence over the paged 4-bit cache: up to
// 8 (new token, query head) pairs per kv head (vq_kivi_paged_attend).
//
//   out = sum_t softmax_t(scale q.k_hat_t) v_hat_t,  t <= the row's own token
//
// The work is one line of 16-token blocks over (sequence, kv head, block),
// cut evenly among the resident warps, whatever the lengths: no plan on the
// host, so a captured call follows the lengths that it finds.  A warp copies
// its blocks (one bulk copy each) into its own ring of shared-memory stages
// and keeps one online softmax per row; a second kernel merges the warps'
// partials of a (sequence, kv head).
//
// Products on mma.m16n8k16 with fp32 accumulators.  Scores: A = queries
// (rows 0-7), B = k_hat of 8 tokens; output: A = weights, B = v_hat.  The
// weights enter as fp16 hi (rows 0-7) plus the remainder lo (rows 8-15, free
// in a 16-row product), so only the output is rounded to 16 bits.  k_hat and
// v_hat are fp16 by definition; a bf16 query row is scaled by a power of two
// to a maximum near 2^14 and taken as fp16, which keeps every bit of values
// down to 2^-28 of the row's largest.
//
// The bound is HBM: a block is read once (160 bytes per token and kv head at
// D = 128, g = 32).
#include "bulk_pipe.cuh"
#include "paged.cuh"
#include "vqk_internal.cuh"

namespace vqk {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kMinBlocks = 2;      // blocks a warp takes at least
constexpr float kLazy = 8.f;       // a maximum is raised when it grows by more

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) {
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ __half2 bits_h2(uint32_t u) {
  return *reinterpret_cast<const __half2 *>(&u);
}

// the four fp16 pairs of a word: nibbles r of its two halves, times s plus z
__device__ __forceinline__ void word_values(uint32_t w, __half2 s, __half2 z, uint32_t (&v)[4]) {
  const __half2 k1024 = bits_h2(0x64006400u), k16 = bits_h2(0x2c002c00u),
                k64 = bits_h2(0xd400d400u);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    // 0x6400 | c is 1024 + c, 0x6400 | 16 c is 1024 + 16 c: both exact
    const __half2 c0 = __hsub2(bits_h2((w & 0x000f000fu) | 0x64006400u), k1024);
    const __half2 c1 = __hfma2(bits_h2((w & 0x00f000f0u) | 0x64006400u), k16, k64);
    v[2 * j] = h2_bits(__hfma2(c0, s, z));
    v[2 * j + 1] = h2_bits(__hfma2(c1, s, z));
    w >>= 8;
  }
}

// Blocks of every sequence as a running sum over (sequence, kv head), in
// shared memory; one entry per sequence.  Faulty lengths count as empty.
struct Lengths {
  int len, n;   // tokens, new tokens (rows)
};

__device__ __forceinline__ Lengths lengths_of(const PagedArgs &a, int b, int max_new) {
  Lengths r{a.lens[b], 1};
  int first = b;
  if (a.cu) {
    first = a.cu[b];
    r.n = a.cu[b + 1] - first;
  }
  if (r.len < 0 || r.len > ((int64_t)a.max_pages << a.page_log2) || r.n < 0 || r.n > max_new ||
      first < 0 || (int64_t)first + r.n > a.tokens) {
    atomicOr(a.status, kBadLength);
    r.len = r.n = 0;
  }
  return r;
}

__device__ __forceinline__ int blocks_of(const Lengths &r) {
  return r.n > 0 ? (r.len + kBlk - 1) / kBlk : 0;
}

// prefix[b] = blocks of sequences 0 ... b - 1 times H_kv, for b <= B
__device__ void block_prefix(const PagedArgs &a, int max_new, int *prefix, int *warp_sum) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + nt - 1) / nt;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < a.B) sum += blocks_of(lengths_of(a, b, max_new)) * a.H_kv;
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int base = inc - sum;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < a.B) {
      prefix[b] = base;
      base += blocks_of(lengths_of(a, b, max_new)) * a.H_kv;
      if (b == a.B - 1) prefix[a.B] = base;
    }
  }
  __syncthreads();
}

// warps that share `units` blocks, and the first block of warp w
__device__ __forceinline__ int warps_used(int units, int warps_max) {
  const int w = (units + kMinBlocks - 1) / kMinBlocks;
  return w < warps_max ? w : warps_max;
}
__device__ __forceinline__ int first_unit(int units, int warps, int w) {
  return (int)((int64_t)units * w / warps);
}
// the warp that owns block u
__device__ __forceinline__ int owner(int units, int warps, int u) {
  return (int)((((int64_t)u + 1) * warps - 1) / units);
}

template <int D>
struct Part {   // a partial: rows x (D outputs, maximum, sum, padding)
  static constexpr int ROW = D + 4;
};

template <int D, int NG>
struct DecSmem {
  static constexpr int BLK = 16 * D + 128 * NG;
  static constexpr int STAGES = D == 128 ? 4 : 6;
  static constexpr int PER_WARP = STAGES * BLK;          // a multiple of 128
  static constexpr int BAR = kWarps * PER_WARP;
  static constexpr int PREFIX = BAR + kWarps * STAGES * 8;
  static_assert(BLK % 128 == 0, "stages stay 128-byte aligned");
};

template <typename T, int D, int NG>
__global__ void __launch_bounds__(kThreads, 4)
k_paged_decode(PagedArgs a, PagedAttend t, int warps_max) {
  using SM = DecSmem<D, NG>;
  constexpr int I = D / 32, BLK = SM::BLK, ST = SM::STAGES, G = D / NG;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int wsum[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n8 = lane >> 2, t4 = lane & 3;
  unsigned char *stage = smem + warp * SM::PER_WARP;
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + SM::BAR) + warp * ST;
  int *prefix = reinterpret_cast<int *>(smem + SM::PREFIX);
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&bar[i]);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  block_prefix(a, t.max_new, prefix, wsum);

  const int units = prefix[a.B];
  const int warps = warps_used(units, warps_max);
  // neighbouring pieces of the line go to different SMs
  const int w = warp * gridDim.x + blockIdx.x;
  if (w >= warps) return;
  int u = first_unit(units, warps, w);
  const int u_end = first_unit(units, warps, w + 1);
  const int H = a.H_kv, GQ = a.H_q / a.H_kv;

  // the sequence of block u
  int b = 0;
  {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= u) lo = mid; else hi = mid;
    }
    b = lo;
  }
  // cursor of the copies: block iu of sequence ib, head ih, at place ik
  int iu = u, ib = b, inb, ih, ik;
  auto enter = [&](int bb, int uu, int &nb, int &h, int &k) {
    nb = (prefix[bb + 1] - prefix[bb]) / H;
    h = (uu - prefix[bb]) / nb;
    k = (uu - prefix[bb]) - h * nb;
  };
  enter(ib, iu, inb, ih, ik);
  const int bpp = a.page_log2 - 4;                     // log2 blocks of a page
  unsigned ok_mask = 0u;                               // stages with a good page
  auto issue = [&](int s) {
    const int p = a.table[(int64_t)ib * a.table_stride + (ik >> bpp)];
    const bool good = (unsigned)p < (unsigned)a.n_pages;
    ok_mask = good ? ok_mask | (1u << s) : ok_mask & ~(1u << s);
    if (lane == 0) {
      if (good) {
        const int64_t blk = (((int64_t)p * H + ih) << bpp) + (ik & ((1 << bpp) - 1));
        mbar_expect_tx(&bar[s], BLK);
        bulk_g2s(stage + s * BLK, a.pool + blk * BLK, BLK, &bar[s]);
      } else {
        atomicOr(a.status, kBadPage);
      }
    }
    ++iu;
    if (++ik == inb) {
      ik = 0;
      if (++ih == H) {
        ih = 0;
        do { ++ib; } while (ib < a.B && prefix[ib + 1] == prefix[ib]);
        if (ib < a.B) inb = (prefix[ib + 1] - prefix[ib]) / H;
      }
    }
  };
#pragma unroll
  for (int s = 0; s < ST; ++s)
    if (iu < u_end) issue(s);

  int s = 0;
  unsigned phases = 0u;
  bool dead = false;
  while (u < u_end && !dead) {
    // one (sequence, kv head)
    int nb, h, k;
    enter(b, u, nb, h, k);
    const Lengths L = lengths_of(a, b, t.max_new);
    const int row0 = a.cu ? a.cu[b] : b, rows = L.n * GQ;
    const int tok = n8 / GQ;
    // the newest token this lane's row sees (rows without a query: none)
    const int last = n8 < rows ? L.len - L.n + tok : -1;
    const int all_see = L.len - L.n;      // tokens up to here are seen by all rows
    uint32_t qa[I][4];
    float sl2 = t.scale;
    {
      uint4 raw[I];
      const T *q = static_cast<const T *>(t.q) + (row0 + tok) * t.q_token +
                   (h * GQ + n8 % GQ) * t.q_head;
#pragma unroll
      for (int i = 0; i < I; ++i)
        raw[i] = n8 < rows ? *reinterpret_cast<const uint4 *>(q + 32 * i + 8 * t4)
                           : make_uint4(0u, 0u, 0u, 0u);
      if constexpr (!std::is_same<T, __half>::value) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            m = fmaxf(m, fabsf(__uint_as_float(x[e] << 16)));
            m = fmaxf(m, fabsf(__uint_as_float(x[e] & 0xffff0000u)));
          }
        }
        m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
        m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
        // factor 2^f, f = 14 - exponent, within what fp32 can hold
        int f = 14 - ((int)(__float_as_uint(m) >> 23) - 127);
        f = m > 0.f ? (f > 126 ? 126 : f) : 0;
        f = f < -100 ? -100 : f;
        const float up = __uint_as_float((uint32_t)(127 + f) << 23);
        sl2 *= __uint_as_float((uint32_t)(127 - f) << 23);
#pragma unroll
        for (int i = 0; i < I; ++i) {
          uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = h2_bits(__floats2half2_rn(__uint_as_float(x[e] << 16) * up,
                                             __uint_as_float(x[e] & 0xffff0000u) * up));
          raw[i] = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < I; ++i) {
        // pairs (r, r + 4) of the 8 channels, as the codes' words give them
        qa[i][0] = __byte_perm(raw[i].x, raw[i].z, 0x5410);
        qa[i][1] = __byte_perm(raw[i].x, raw[i].z, 0x7632);
        qa[i][2] = __byte_perm(raw[i].y, raw[i].w, 0x5410);
        qa[i][3] = __byte_perm(raw[i].y, raw[i].w, 0x7632);
      }
    }
    float m = -INFINITY, l = 0.f;
    float o[I][4][4];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][r][e] = 0.f;

    const int k_end = min(nb, k + (u_end - u));
    u += k_end - k;
    for (; k < k_end; ++k) {
      const bool good = (ok_mask >> s) & 1u;
      if (good) {
        const bool ok = mbar_wait(&bar[s], (phases >> s) & 1u);
        phases ^= 1u << s;
        if (!__all_sync(kFull, ok)) {
          if (lane == 0) atomicOr(a.status, kGaveUp);
          dead = true;
          break;
        }
        const unsigned char *st = stage + s * BLK;
        const int t0 = k * kBlk;
        float sc[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int tl = 8 * nt + n8;
          uint32_t kw[I];
          if constexpr (I == 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(st + tl * (D / 2) + t4 * 16);
            kw[0] = x.x; kw[1] = x.y; kw[2] = x.z; kw[3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(st + tl * (D / 2) + t4 * 8);
            kw[0] = x.x; kw[1] = x.y;
          }
          const uint2 *km = reinterpret_cast<const uint2 *>(st + off_km(D)) + (tl >> 1) * NG;
          const unsigned sel = (tl & 1) ? 0x3232u : 0x1010u;
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
          __half2 ks, kz;
#pragma unroll
          for (int i = 0; i < I; ++i) {
            if ((32 * i) % G == 0) {
              const uint2 x = km[32 * i / G];
              ks = bits_h2(__byte_perm(x.x, 0u, sel));
              kz = bits_h2(__byte_perm(x.y, 0u, sel));
            }
            uint32_t v[4];
            word_values(kw[i], ks, kz, v);
            mma16816(sc[nt], qa[i][0], 0u, qa[i][1], 0u, v[0], v[1]);
            mma16816(sc[nt], qa[i][2], 0u, qa[i][3], 0u, v[2], v[3]);
          }
        }
        // scores of row n8: tokens 2 t4, 2 t4 + 1 of both octets
        float x[4] = {sc[0][0] * sl2, sc[0][1] * sl2, sc[1][0] * sl2, sc[1][1] * sl2};
        const bool tail = t0 + kBlk - 1 > all_see;
        if (tail) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (t0 + 8 * (e >> 1) + 2 * t4 + (e & 1) > last) x[e] = -INFINITY;
        }
        const float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        if (__any_sync(kFull, mx > m + kLazy)) {
          float mn = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
          mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, 2));
          mn = fmaxf(m, mn);
          const float f = m == -INFINITY ? 0.f : ex2(m - mn);
          m = mn;
          l *= f;
#pragma unroll
          for (int i = 0; i < I; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[i][r][e] *= f;
        }
        const float base = m == -INFINITY ? 0.f : m;
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = ex2(x[e] - base);
          l += p[e];
        }
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const __half2 hh = __floats2half2_rn(p[2 * e], p[2 * e + 1]);
          const float2 hf = __half22float2(hh);
          hi[e] = h2_bits(hh);
          lo[e] = h2_bits(__floats2half2_rn(p[2 * e] - hf.x, p[2 * e + 1] - hf.y));
        }
        uint32_t vw[2][I];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const unsigned char *vp = st + off_vc(D, G) + (32 * hf + lane) * (4 * I);
          if constexpr (I == 4) {
            const uint4 y = *reinterpret_cast<const uint4 *>(vp);
            vw[hf][0] = y.x; vw[hf][1] = y.y; vw[hf][2] = y.z; vw[hf][3] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2 *>(vp);
            vw[hf][0] = y.x; vw[hf][1] = y.y;
          }
        }
        const uint2 *vm = reinterpret_cast<const uint2 *>(st + off_vm(D, G)) + t4 * NG;
        // tokens behind the sequence hold anything: their values become 0
        unsigned keep[2] = {kFull, kFull};
        if (tail) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int tp = t0 + 8 * hf + 2 * t4;
            keep[hf] = (tp < L.len ? 0x0000ffffu : 0u) | (tp + 1 < L.len ? 0xffff0000u : 0u);
          }
        }
        __half2 vs[2], vz[2];
#pragma unroll
        for (int i = 0; i < I; ++i) {
          if ((32 * i) % G == 0) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint2 y = vm[4 * hf * NG + 32 * i / G];
              vs[hf] = bits_h2(y.x & keep[hf]);
              vz[hf] = bits_h2(y.y & keep[hf]);
            }
          }
          uint32_t v0[4], v1[4];
          word_values(vw[0][i], vs[0], vz[0], v0);
          word_values(vw[1][i], vs[1], vz[1], v1);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            mma16816(o[i][r], hi[0], lo[0], hi[1], lo[1], v0[r], v1[r]);
        }
      }
      // every lane has read the stage
      __syncwarp();
      if (iu < u_end) issue(s);
      s = s + 1 == ST ? 0 : s + 1;
    }
    // the partial of this (sequence, kv head): row n8's channels 32 i + 8 t4 ...
    l += __shfl_xor_sync(kFull, l, 1);
    l += __shfl_xor_sync(kFull, l, 2);
    if (n8 < rows) {
      float *part = t.ws + ((int64_t)(w + b * H + h) * (t.max_new * GQ) + n8) * Part<D>::ROW;
#pragma unroll
      for (int i = 0; i < I; ++i) {
        float4 c0, c1;
        c0 = make_float4(o[i][0][0] + o[i][0][2], o[i][1][0] + o[i][1][2],
                         o[i][2][0] + o[i][2][2], o[i][3][0] + o[i][3][2]);
        c1 = make_float4(o[i][0][1] + o[i][0][3], o[i][1][1] + o[i][1][3],
                         o[i][2][1] + o[i][2][3], o[i][3][1] + o[i][3][3]);
        reinterpret_cast<float4 *>(part + 32 * i + 8 * t4)[0] = c0;
        reinterpret_cast<float4 *>(part + 32 * i + 8 * t4)[1] = c1;
      }
      if (t4 == 0) *reinterpret_cast<float2 *>(part + D) = make_float2(m, l);
    }
    // the next head or sequence with blocks
    if (h + 1 == H) {
      do { ++b; } while (b < a.B && prefix[b + 1] == prefix[b]);
    }
  }
  if (dead) {
    // let the copies in flight land before the CTA's memory is given up
    for (int i = 0; i < ST; ++i)
      if ((ok_mask >> i) & 1u) mbar_wait(&bar[i], (phases >> i) & 1u);
  }
}

// Merge of the partials of a (sequence, kv head): one CTA per output row;
// each warp takes every kMergeWarps-th partial, its lanes the channels.
constexpr int kMergeWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps)
k_paged_merge(PagedArgs a, PagedAttend t, int warps_max) {
  constexpr int CPL = D / 32;
  __shared__ float red[kMergeWarps][D];
  __shared__ float rl[kMergeWarps], rm[kMergeWarps];
  extern __shared__ int prefix[];
  __shared__ int wsum[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  block_prefix(a, t.max_new, prefix, wsum);
  const int H = a.H_kv, GQ = a.H_q / H, R = t.max_new * GQ;
  const int row = blockIdx.x % R, seg = blockIdx.x / R, b = seg / H, h = seg % H;
  const Lengths L = lengths_of(a, b, t.max_new);
  if (row >= L.n * GQ) return;
  const int64_t tokrow = (a.cu ? a.cu[b] : b) + row / GQ;
  T *out = static_cast<T *>(t.out) + (tokrow * a.H_q + h * GQ + row % GQ) * D;
  const int units = prefix[a.B], nb = (prefix[b + 1] - prefix[b]) / H;
  float acc[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
  float lsum = 0.f, mw = -INFINITY;
  if (nb > 0) {
    const int warps = warps_used(units, warps_max);
    const int u0 = prefix[b] + h * nb;
    const int w0 = owner(units, warps, u0), w1 = owner(units, warps, u0 + nb - 1);
    // this warp's partials: the maximum first, then the weighted sums
    const float *base = t.ws + ((int64_t)(w0 + seg) * R + row) * Part<D>::ROW;
    const int64_t step = (int64_t)R * Part<D>::ROW;
    const int count = w1 - w0 + 1;
    for (int i = warp + kMergeWarps * lane; i < count; i += 32 * kMergeWarps)
      mw = fmaxf(mw, base[i * step + D]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mw = fmaxf(mw, __shfl_xor_sync(kFull, mw, o));
#pragma unroll 4
    for (int i = warp; i < count; i += kMergeWarps) {
      const float *p = base + i * step;
      const float2 ml = *reinterpret_cast<const float2 *>(p + D);
      const float f = ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.f) : ex2(ml.x - mw);
      float v[CPL];
      if constexpr (CPL == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p + 4 * lane);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2 *>(p + 2 * lane);
        v[0] = x.x; v[1] = x.y;
      }
      lsum = fmaf(f, ml.y, lsum);
#pragma unroll
      for (int e = 0; e < CPL; ++e) acc[e] = fmaf(f, v[e], acc[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < CPL; ++e) red[warp][CPL * lane + e] = acc[e];
  if (lane == 0) {
    rl[warp] = lsum;
    rm[warp] = mw;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float M = rm[0];
#pragma unroll
    for (int i = 1; i < kMergeWarps; ++i) M = fmaxf(M, rm[i]);
    float v = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kMergeWarps; ++i) {
      const float f = rm[i] == -INFINITY ? 1.f : ex2(rm[i] - M);
      v = fmaf(f, red[i][threadIdx.x], v);
      sum = fmaf(f, rl[i], sum);
    }
    // no token seen: a row of zeros
    const float y = sum == 0.f ? 0.f : v / sum;
    if constexpr (std::is_same<T, __half>::value) out[threadIdx.x] = __float2half_rn(y);
    else out[threadIdx.x] = __float2bfloat16_rn(y);
  }
}

int decode_ctas(int sm_count) { return 4 * sm_count; }

template <typename T, int D, int NG>
cudaError_t launch_dec(const PagedArgs &a, const PagedAttend &t, int sm_count,
                       cudaStream_t st) {
  using SM = DecSmem<D, NG>;
  const size_t smem = SM::PREFIX + sizeof(int) * (a.B + 1);
  cudaError_t e = cudaFuncSetAttribute(k_paged_decode<T, D, NG>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int ctas = decode_ctas(sm_count), warps_max = ctas * kWarps;
  e = launch_pdl(k_paged_decode<T, D, NG>, dim3(ctas), dim3(kThreads), smem, st, a, t,
                 warps_max);
  count_launch();
  if (e != cudaSuccess) return e;
  const int rows = t.max_new * (a.H_q / a.H_kv);
  e = launch_pdl(k_paged_merge<T, D>, dim3(a.B * a.H_kv * rows), dim3(32 * kMergeWarps),
                 sizeof(int) * (a.B + 1), st, a, t, warps_max);
  count_launch();
  return e;
}

template <typename T>
cudaError_t launch_t(const PagedArgs &a, const PagedAttend &t, int D, int sm_count,
                     cudaStream_t st) {
  const int ng = D / a.g;
  if (D == 64)
    return ng == 1 ? launch_dec<T, 64, 1>(a, t, sm_count, st)
                   : launch_dec<T, 64, 2>(a, t, sm_count, st);
  return ng == 1   ? launch_dec<T, 128, 1>(a, t, sm_count, st)
         : ng == 2 ? launch_dec<T, 128, 2>(a, t, sm_count, st)
                   : launch_dec<T, 128, 4>(a, t, sm_count, st);
}

}  // namespace

size_t paged_decode_ws(int B, int H_kv, int D, int rows, int sm_count) {
  return ((size_t)decode_ctas(sm_count) * kWarps + (size_t)B * H_kv) * rows * (D + 4) *
         sizeof(float);
}

cudaError_t launch_paged_decode(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                                int sm_count, cudaStream_t st) {
  return dtype == VQ_F16 ? launch_t<__half>(a, t, D, sm_count, st)
                         : launch_t<__nv_bfloat16>(a, t, D, sm_count, st);
}

}  // namespace vqk
