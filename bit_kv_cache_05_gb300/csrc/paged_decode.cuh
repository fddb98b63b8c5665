// Attention of few new tokens per sequence over the paged 4-bit cache: up to
// 16 (new token, query head) pairs per kv head (vq_kivi_paged_attend,
// vq_kivi_paged_attend_tree, vq_kivi_paged_attend_weights).
//
//   out = sum_t softmax_t(scale q.k_hat_t) v_hat_t,  t <= the row's own token,
//                  or t before the new tokens or named by the row's mask
//
// The work is one line of 32-token steps (two blocks) over (sequence, kv head,
// step), cut evenly among the resident warps, whatever the lengths: no plan
// on the host, so a captured call follows the lengths that it finds.  A warp
// copies its steps (one bulk copy each, two where a page holds one block) into
// its own ring of shared-memory stages and keeps one online softmax per row; a
// second kernel merges the warps' partials of a (sequence, kv head).
//
// Products on mma.m16n8k16 with fp32 accumulators.  Scores: A = k_hat of 16
// tokens (row n the even token of pair n, row 8 + n the odd one, so that a
// pair's scales are the halves of one word), B = up to 8 query rows; output:
// A = weights, turned over by movmatrix, B = v_hat.  The weights enter as
// fp16 hi (rows 0-7) plus the remainder lo (rows 8-15, free in a 16-row
// product).  With 9 to 16 rows (drafts) the second 8 take those rows, and the
// weights of all are rounded to fp16 once, as the tensor-memory kernel rounds
// them.  Both operands that change are made where the product reads them: no
// register is moved.  k_hat and v_hat are fp16 by definition; a bf16
// query row is scaled by a power of two to a maximum near 2^14 and taken as
// fp16, which keeps every bit of values down to 2^-28 of the row's largest.
//
// What a weight loses: below 2^-14 fp16 has steps of 2^-24, no longer small
// beside the weight, while the weights' sum is kept in fp32; a long tail of
// small weights behind a large one would be lost from the output alone.  So a
// row's largest weight is 2^7 or 2^12 (Weights below), not 1, and may grow to
// 2^15.  With hi + lo the remainder is taken times 2^12 (exact) into sums of
// its own and is off by 2^-22 of the weight or 2^-37, which is 2^-44 of the
// row's largest: only the output is rounded to 16 bits.  Rounded once (9 to
// 16 rows) a weight is off by 2^-11 of itself, as an fp16 output, or by 2^-25,
// which is 2^-37 of the row's largest.
//
// The bound is HBM: a block is read once (160 bytes per token and kv head at
// D = 128, g = 32).
#pragma once

#include "bulk_pipe.cuh"
#include "paged.cuh"
#include "paged_words.cuh"
#include "stage_ring.h"
#include "vqk_internal.cuh"

namespace vqk {
namespace {

// What a row sees and what is left beside the outputs: kCausal the tokens up to
// its own; kTree those before the new tokens and the ones that its mask names;
// kWeigh as kCausal, each score left for k_paged_merge_weigh.
enum Form { kCausal, kTree, kWeigh };

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kStep = 32;          // tokens of a step: two blocks
constexpr int kMinSteps = 1;       // steps a warp takes at least

// A fresh maximum's weight is 2^top; a maximum is raised when a weight would
// pass 2^most.  hi + lo need no more range than 7 bits give; single fp16
// weights get all but 3.
template <int ROWS>
struct Weights {
  static constexpr float top = ROWS == 8 ? 7.f : 12.f, most = 15.f;
};
constexpr float kLo = 4096.f;      // the remainders' factor

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// an 8 x 8 matrix of 16-bit values, a row per four lanes, turned over
__device__ __forceinline__ uint32_t turn(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// the four fp16 pairs of a word: nibbles r of its two halves, times s plus z
__device__ __forceinline__ void word_values(uint32_t w, __half2 s, __half2 z, uint32_t (&v)[4]) {
  const __half2 k1024 = bits_h2(0x64006400u), k16 = bits_h2(0x2c002c00u),
                k64 = bits_h2(0xd400d400u);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    // 1024 + c and 1024 + 16 c: both steps to c are exact
    const __half2 c0 = __hsub2(field<0x000f000fu>(w), k1024);
    const __half2 c1 = __hfma2(field<0x00f000f0u>(w), k16, k64);
    v[2 * j] = h2_bits(__hfma2(c0, s, z));
    v[2 * j + 1] = h2_bits(__hfma2(c1, s, z));
    w >>= 8;
  }
}

__device__ __forceinline__ int steps_of(const Seq &r) {
  return r.n > 0 ? (r.len + kStep - 1) / kStep : 0;
}

// prefix[b] = steps of sequences 0 ... b - 1 times H_kv, for b <= B
__device__ void step_prefix(const PagedArgs &a, int max_new, int *prefix, int *warp_sum) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + nt - 1) / nt;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < a.B) sum += steps_of(sequence_of(a, b, max_new)) * a.H_kv;
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
      base += steps_of(sequence_of(a, b, max_new)) * a.H_kv;
      if (b == a.B - 1) prefix[a.B] = base;
    }
  }
  __syncthreads();
}

// warps that share `units` steps, and the first step of warp w
__device__ __forceinline__ int warps_used(int units, int warps_max) {
  const int w = (units + kMinSteps - 1) / kMinSteps;
  return w < warps_max ? w : warps_max;
}
// (pieces differ by one step at most)
struct Cut {
  int each, more;
  __device__ Cut(int units, int warps) : each(units / warps), more(units % warps) {}
  __device__ int first(int w) const { return each * w + min(w, more); }
  // the warp that owns step u
  __device__ int owner(int u) const {
    const int big = more * (each + 1);
    return u < big ? u / (each + 1) : more + (u - big) / each;
  }
};

template <int D>
struct Part {   // a partial: rows x (D outputs, maximum, sum, padding)
  static constexpr int ROW = D + 4;
};

// CTAs of 4 warps on an SM: what the registers allow (64 accumulators a thread
// at D = 128, the second 8 rows' queries and scores with 16 rows; 16 sequences
// of about 6000 tokens, 16 rows: 53.6 us with two CTAs, 62 with three and
// spills)
__host__ __device__ constexpr int decode_ctas(int D, int rows) {
  return D == 64 ? 4 : (rows > 8 ? 2 : 3);
}

template <int D, int NG, int ROWS>
struct DecSmem {
  static constexpr int BLK = 16 * D + 128 * NG;
  static constexpr int STEP = 2 * BLK;
  static constexpr int CTAS = decode_ctas(D, ROWS);
  static constexpr int STAGES = CTAS == 3 ? 3 : 4;
  static constexpr int PER_WARP = STAGES * STEP;         // a multiple of 128
  static constexpr int BAR = kWarps * PER_WARP;
  static constexpr int PREFIX = BAR + kWarps * STAGES * 8;
  static_assert(BLK % 128 == 0, "stages stay 128-byte aligned");
};

// ROWS: 8, or 16 for calls with more rows
template <typename T, int D, int NG, int ROWS, int FORM>
__global__ void __launch_bounds__(kThreads, DecSmem<D, NG, ROWS>::CTAS)
k_paged_decode(PagedArgs a, PagedAttend t, int warps_max, int *prefixes, float *scores) {
  using SM = DecSmem<D, NG, ROWS>;
  using W = Weights<ROWS>;
  constexpr int I = D / 32, BLK = SM::BLK, STEP = SM::STEP, ST = SM::STAGES, G = D / NG;
  constexpr int NR = ROWS / 8;      // groups of 8 rows
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
  step_prefix(a, t.max_new, prefix, wsum);

  if (blockIdx.x == 0)   // for the merge
    for (int i = threadIdx.x; i <= a.B; i += kThreads) prefixes[i] = prefix[i];
  const int units = prefix[a.B];
  const int warps = warps_used(units, warps_max);
  // neighbouring pieces of the line go to different SMs
  const int w = warp * gridDim.x + blockIdx.x;
  if (w >= warps) return;
  const Cut cut(units, warps);
  int u = cut.first(w);
  const int u_end = cut.first(w + 1);
  const int H = a.H_kv, GQ = a.H_q / a.H_kv;

  auto find = [&](int uu) {   // the sequence of step uu
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= uu) lo = mid; else hi = mid;
    }
    return lo;
  };
  auto enter = [&](int bb, int uu, int &nb, int &h, int &k) {
    nb = (prefix[bb + 1] - prefix[bb]) / H;
    h = (uu - prefix[bb]) / nb;
    k = (uu - prefix[bb]) - h * nb;
  };
  int b = find(u);
  const int bpp = a.page_log2 - 4;                     // log2 blocks of a page
  // The copies of 32 steps are prepared at once, lane j those of step ibase +
  // j: where its blocks lie and whether their pages are in the pool.
  int iu = u, ibase = u;
  const uint8_t *src0 = nullptr, *src1 = nullptr;
  unsigned g0 = 0u, g1 = 0u;                           // of the 32 steps
  auto prepare = [&]() {
    ibase = iu;
    const int v = iu + lane;
    bool ok0 = false, ok1 = false;
    if (v < u_end) {
      int nb, h, k;
      const int bb = find(v);
      enter(bb, v, nb, h, k);
      const int32_t *row = a.table + (int64_t)bb * a.table_stride;
      const int blk = 2 * k, nblk = (a.lens[bb] + kBlk - 1) / kBlk;
      const int p0 = row[blk >> bpp];
      ok0 = (unsigned)p0 < (unsigned)a.n_pages;
      src0 = a.pool + ((((int64_t)p0 * H + h) << bpp) + (blk & ((1 << bpp) - 1))) * BLK;
      bool bad = !ok0;
      if (blk + 1 < nblk) {
        const int p1 = bpp ? p0 : row[blk + 1];
        ok1 = (unsigned)p1 < (unsigned)a.n_pages;
        src1 = bpp ? src0 + BLK : a.pool + ((int64_t)p1 * H + h) * BLK;
        bad = bad || !ok1;
      }
      if (bad) atomicOr(a.status, kBadPage);
    }
    g0 = __ballot_sync(kFull, ok0);
    g1 = __ballot_sync(kFull, ok1);
  };
  prepare();
  StageRing ring;
  auto issue = [&](int s) {
    if (iu - ibase == 32) prepare();
    const int j = iu - ibase;
    const unsigned gd = ((g0 >> j) & 1u) | (((g1 >> j) & 1u) << 1);
    ring.issued(s, gd);
    if (lane == j && gd) {
      unsigned char *dst = stage + s * STEP;
      mbar_expect_tx(&bar[s], gd == 3u ? STEP : BLK);
      if (bpp && gd == 3u) {
        bulk_g2s(dst, src0, STEP, &bar[s]);
      } else {
        if (gd & 1u) bulk_g2s(dst, src0, BLK, &bar[s]);
        if (gd & 2u) bulk_g2s(dst + BLK, src1, BLK, &bar[s]);
      }
    }
    ++iu;
  };
#pragma unroll
  for (int s = 0; s < ST; ++s)
    if (iu < u_end) issue(s);

  int s = 0;
  bool dead = false;
  while (u < u_end && !dead) {
    // one (sequence, kv head)
    int nb, h, k;
    enter(b, u, nb, h, k);
    const Seq L = sequence_of(a, b, t.max_new);
    const int row0 = L.first, rows = L.n * GQ;
    // tokens up to here are seen by all rows
    const int all_see = L.len - L.n - (FORM == kTree ? 1 : 0);
    // of rows 8 g + 2 t4 and the next: the newest tokens they see (rows
    // without a query: none), the scores' factors, maxima and sums
    int2 see[NR];
    float2 sc[NR], m[NR], l[NR];
    uint32_t qa[NR][I][4];
#pragma unroll
    for (int g = 0; g < NR; ++g) {
      const int r0 = 8 * g + 2 * t4, row = 8 * g + n8;
      see[g] = make_int2(r0 < rows ? L.len - L.n + r0 / GQ : -1,
                         r0 + 1 < rows ? L.len - L.n + (r0 + 1) / GQ : -1);
      m[g] = make_float2(-INFINITY, -INFINITY);
      l[g] = make_float2(0.f, 0.f);
      float sl2 = t.scale;
      uint4 raw[I];
      const T *q = static_cast<const T *>(t.q) + (int64_t)(row0 + row / GQ) * t.q_token +
                   (int64_t)(h * GQ + row % GQ) * t.q_head;
#pragma unroll
      for (int i = 0; i < I; ++i)
        raw[i] = row < rows ? *reinterpret_cast<const uint4 *>(q + 32 * i + 8 * t4)
                            : make_uint4(0u, 0u, 0u, 0u);
      if constexpr (!std::is_same<T, __half>::value) {
        float mq = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            mq = fmaxf(mq, fabsf(__uint_as_float(x[e] << 16)));
            mq = fmaxf(mq, fabsf(__uint_as_float(x[e] & 0xffff0000u)));
          }
        }
        mq = fmaxf(mq, __shfl_xor_sync(kFull, mq, 1));
        mq = fmaxf(mq, __shfl_xor_sync(kFull, mq, 2));
        const RowScale rs = row_scale(__float_as_uint(mq), t.scale);
        const float up = rs.up;
        sl2 = rs.back;
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
        qa[g][i][0] = __byte_perm(raw[i].x, raw[i].z, 0x5410);
        qa[g][i][1] = __byte_perm(raw[i].x, raw[i].z, 0x7632);
        qa[g][i][2] = __byte_perm(raw[i].y, raw[i].w, 0x5410);
        qa[g][i][3] = __byte_perm(raw[i].y, raw[i].w, 0x7632);
      }
      sc[g] = make_float2(__shfl_sync(kFull, sl2, 8 * t4), __shfl_sync(kFull, sl2, 8 * t4 + 4));
    }
    float o[I][4][4];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][r][e] = 0.f;

    // this step's scores, row by row
    float *left = nullptr;
    if constexpr (FORM == kWeigh)
      left = scores + (int64_t)(prefix[b] + h * nb + k) * (t.max_new * GQ * kStep) + 2 * n8;
    const int k_end = min(nb, k + (u_end - u));
    u += k_end - k;
    for (; k < k_end; ++k) {
      const unsigned gd = ring.blocks(s);
      if (gd) {
        const bool ok = bounded_wait(&bar[s], ring.parity(s));
        if (!__all_sync(kFull, ok)) {
          if (lane == 0) atomicOr(a.status, kGaveUp);
          dead = true;
          break;
        }
        ring.landed(s);
        const unsigned char *st = stage + s * STEP;
        const int t0 = k * kStep;
        // raw scores of rows 8 g + 2 t4 and the next: tokens 16 bk + 2 n8 and
        // the next
        float x[NR][2][4];
#pragma unroll
        for (int bk = 0; bk < 2; ++bk) {
          const unsigned char *blk = st + bk * BLK;
          uint32_t k0[I], k1[I];
          uint2 km[NG];
          load_words<I>(blk + 2 * n8 * (D / 2) + t4 * (4 * I), k0);
          load_words<I>(blk + (2 * n8 + 1) * (D / 2) + t4 * (4 * I), k1);
          load_meta<NG>(blk + off_km(D) + n8 * (8 * NG), km);
#pragma unroll
          for (int g = 0; g < NR; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[g][bk][e] = 0.f;
#pragma unroll
          for (int i = 0; i < I; ++i) {
            const __half2 s2 = bits_h2(km[32 * i / G].x), z2 = bits_h2(km[32 * i / G].y);
            uint32_t v0[4], v1[4];
            word_values(k0[i], __low2half2(s2), __low2half2(z2), v0);
            word_values(k1[i], __high2half2(s2), __high2half2(z2), v1);
#pragma unroll
            for (int g = 0; g < NR; ++g) {
              mma16816(x[g][bk], v0[0], v1[0], v0[1], v1[1], qa[g][i][0], qa[g][i][1]);
              mma16816(x[g][bk], v0[2], v1[2], v0[3], v1[3], qa[g][i][2], qa[g][i][3]);
            }
          }
        }
        const bool special = t0 + kStep - 1 > all_see || gd != 3u;
        if (special) {
#pragma unroll
          for (int g = 0; g < NR; ++g) {
            // the masks of a tree's rows are read where they are needed: few
            // steps have new tokens
            TreeRow tree[2];
            if constexpr (FORM == kTree) {
              tree[0] = tree_row(t.tree, L, (8 * g + 2 * t4) / GQ, see[g].x);
              tree[1] = tree_row(t.tree, L, (8 * g + 2 * t4 + 1) / GQ, see[g].y);
            }
#pragma unroll
            for (int bk = 0; bk < 2; ++bk)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int tk = t0 + 16 * bk + 2 * n8 + (e >> 1);
                bool hidden;
                if constexpr (FORM == kTree) hidden = !tree[e & 1].sees(tk);
                else hidden = tk > ((e & 1) ? see[g].y : see[g].x);
                if (hidden || !((gd >> bk) & 1u)) x[g][bk][e] = -INFINITY;
              }
          }
        }
        // The scaled scores are rounded before a maximum is taken from them,
        // so that a score's distance from it is exact: in one fma with the
        // maximum it would be off by the maximum's own rounding, whole bits
        // from 2^24 on (the fma takes 77.7 us, this 78.8: 65536 tokens, 32 kv
        // heads).
        float2 mx[NR];
        bool raise = false;
#pragma unroll
        for (int g = 0; g < NR; ++g) {
#pragma unroll
          for (int bk = 0; bk < 2; ++bk)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 z = __fmul2_rn(make_float2(x[g][bk][2 * e], x[g][bk][2 * e + 1]), sc[g]);
              x[g][bk][2 * e] = z.x;
              x[g][bk][2 * e + 1] = z.y;
            }
          mx[g].x = fmaxf(fmaxf(x[g][0][0], x[g][0][2]), fmaxf(x[g][1][0], x[g][1][2]));
          mx[g].y = fmaxf(fmaxf(x[g][0][1], x[g][0][3]), fmaxf(x[g][1][1], x[g][1][3]));
          raise = raise || mx[g].x + (W::top - m[g].x) > W::most ||
                  mx[g].y + (W::top - m[g].y) > W::most;
          if constexpr (FORM == kWeigh) {
            const int r0 = 8 * g + 2 * t4;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (r0 + e < rows)
#pragma unroll
                for (int bk = 0; bk < 2; ++bk)
                  *reinterpret_cast<float2 *>(left + (r0 + e) * kStep + 16 * bk) =
                      make_float2(x[g][bk][e], x[g][bk][2 + e]);
          }
        }
        if (__any_sync(kFull, raise)) {
#pragma unroll
          for (int g = 0; g < NR; ++g) {
            float2 mn = mx[g];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              mn.x = fmaxf(mn.x, __shfl_xor_sync(kFull, mn.x, d));
              mn.y = fmaxf(mn.y, __shfl_xor_sync(kFull, mn.y, d));
            }
            mn.x = fmaxf(m[g].x, stand_in(mn.x, W::top));
            mn.y = fmaxf(m[g].y, stand_in(mn.y, W::top));
            const float f0 = m[g].x == -INFINITY ? 0.f : ex2(m[g].x - mn.x);
            const float f1 = m[g].y == -INFINITY ? 0.f : ex2(m[g].y - mn.y);
            m[g] = mn;
            l[g].x *= f0;
            l[g].y *= f1;
            // row 8 g + n8's factor; with 8 rows, of both its parts
            const float g0 = __shfl_sync(kFull, f0, n8 >> 1),
                        g1 = __shfl_sync(kFull, f1, n8 >> 1);
            const float f = (n8 & 1) ? g1 : g0;
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                if (NR == 1 || g == 0) {
                  o[i][r][0] *= f;
                  o[i][r][1] *= f;
                }
                if (NR == 1 || g == 1) {
                  o[i][r][2] *= f;
                  o[i][r][3] *= f;
                }
              }
          }
        }
#pragma unroll
        for (int bk = 0; bk < 2; ++bk) {
          // weights of the even (0) and the odd (1) tokens: of the 8 rows as
          // fp16 hi + lo, or of both groups of rows
          uint32_t wt[2][2];
#pragma unroll
          for (int g = 0; g < NR; ++g) {
            const float2 base = make_float2(m[g].x == -INFINITY ? 0.f : W::top - m[g].x,
                                            m[g].y == -INFINITY ? 0.f : W::top - m[g].y);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 y = __fadd2_rn(make_float2(x[g][bk][2 * e], x[g][bk][2 * e + 1]), base);
              const float2 p = make_float2(ex2(y.x), ex2(y.y));
              l[g] = __fadd2_rn(l[g], p);
              const __half2 hh = __floats2half2_rn(p.x, p.y);
              wt[g][e] = turn(h2_bits(hh));
              if constexpr (NR == 1) {
                const float2 hf = __half22float2(hh);
                const float2 lo = __fmul2_rn(make_float2(p.x - hf.x, p.y - hf.y),
                                             make_float2(kLo, kLo));
                wt[1][e] = turn(h2_bits(__floats2half2_rn(lo.x, lo.y)));
              }
            }
          }
          // row n8's (and 8 + n8's) weights of token pairs 2 t4 and 2 t4 + 1
          const uint32_t a0 = __byte_perm(wt[0][0], wt[0][1], 0x5410),
                         a1 = __byte_perm(wt[1][0], wt[1][1], 0x5410),
                         a2 = __byte_perm(wt[0][0], wt[0][1], 0x7632),
                         a3 = __byte_perm(wt[1][0], wt[1][1], 0x7632);
          const unsigned char *blk = st + bk * BLK;
          uint32_t vw[2][I];
          uint2 vm[2][NG];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int pair = 2 * t4 + j;
            load_words<I>(blk + off_vc(D, G) + ((8 * (pair >> 2) + n8) * 4 + (pair & 3)) * (4 * I),
                          vw[j]);
            load_meta<NG>(blk + off_vm(D, G) + pair * (8 * NG), vm[j]);
          }
          if (special) {
            // tokens behind the sequence hold anything: their values become 0
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int tp = t0 + 16 * bk + 2 * (2 * t4 + j);
              unsigned keep = (tp < L.len ? 0x0000ffffu : 0u) | (tp + 1 < L.len ? 0xffff0000u : 0u);
              if (!((gd >> bk) & 1u)) keep = 0u;
#pragma unroll
              for (int g = 0; g < NG; ++g) {
                vm[j][g].x &= keep;
                vm[j][g].y &= keep;
              }
            }
          }
#pragma unroll
          for (int i = 0; i < I; ++i) {
            uint32_t v0[4], v1[4];
            word_values(vw[0][i], bits_h2(vm[0][32 * i / G].x), bits_h2(vm[0][32 * i / G].y), v0);
            word_values(vw[1][i], bits_h2(vm[1][32 * i / G].x), bits_h2(vm[1][32 * i / G].y), v1);
#pragma unroll
            for (int r = 0; r < 4; ++r) mma16816(o[i][r], a0, a1, a2, a3, v0[r], v1[r]);
          }
        }
      } else if constexpr (FORM == kWeigh) {
        // no block of this step is in the pool
        for (int r = t4; r < rows; r += 4)
#pragma unroll
          for (int bk = 0; bk < 2; ++bk)
            *reinterpret_cast<float2 *>(left + r * kStep + 16 * bk) =
                make_float2(-INFINITY, -INFINITY);
      }
      if constexpr (FORM == kWeigh) left += t.max_new * GQ * kStep;
      // every lane has read the stage
      __syncwarp();
      if (iu < u_end) issue(s);
      s = s + 1 == ST ? 0 : s + 1;
    }
    // the partial of this (sequence, kv head): channels 32 i + 8 t4 ... of row
    // n8 (and 8 + n8)
    float *first = t.ws + (int64_t)(w + b * H + h) * (t.max_new * GQ) * Part<D>::ROW;
#pragma unroll
    for (int g = 0; g < NR; ++g) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l[g].x += __shfl_xor_sync(kFull, l[g].x, d);
        l[g].y += __shfl_xor_sync(kFull, l[g].y, d);
      }
      const int r0 = 8 * g + 2 * t4 + n8;
      if (n8 < 2 && r0 < rows)
        *reinterpret_cast<float2 *>(first + r0 * Part<D>::ROW + D) =
            n8 ? make_float2(m[g].y, l[g].y) : make_float2(m[g].x, l[g].x);
      if (8 * g + n8 < rows) {
        float *part = first + (8 * g + n8) * Part<D>::ROW;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float4 y;
            if constexpr (NR == 1)
              y = make_float4(fmaf(o[i][0][2 + c], 1.f / kLo, o[i][0][c]),
                              fmaf(o[i][1][2 + c], 1.f / kLo, o[i][1][c]),
                              fmaf(o[i][2][2 + c], 1.f / kLo, o[i][2][c]),
                              fmaf(o[i][3][2 + c], 1.f / kLo, o[i][3][c]));
            else
              y = make_float4(o[i][0][2 * g + c], o[i][1][2 * g + c], o[i][2][2 * g + c],
                              o[i][3][2 * g + c]);
            reinterpret_cast<float4 *>(part + 32 * i + 8 * t4)[c] = y;
          }
      }
    }
    // the next head or sequence with steps
    if (h + 1 == H && u < u_end) {
      do { ++b; } while (prefix[b + 1] == prefix[b]);
    }
  }
  if (dead) {
    // let the copies in flight land before the CTA's memory is given up
    for (int i = 0; i < ST; ++i)
      if (ring.blocks(i)) bounded_wait(&bar[i], ring.parity(i));
  }
}

// a partial's factor beside the maximum M; one without a seen token weighs
// nothing (NaN sums stay)
__device__ __forceinline__ float part_factor(float2 ml, float M) {
  return ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.f) : ex2(ml.x - M);
}

// Merge of the partials of a (sequence, kv head): one CTA per output row;
// each warp takes every WARPS-th partial, its lanes the channels.
template <typename T, int D, int WARPS>
__device__ __forceinline__ void merge_row(const PagedArgs &a, const PagedAttend &t, int warps_max,
                                          const int *prefix) {
  constexpr int CPL = D / 32;
  __shared__ float red[WARPS][D];
  __shared__ float rl[WARPS], rm[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int H = a.H_kv, GQ = a.H_q / H, R = t.max_new * GQ;
  const int row = blockIdx.x % R, seg = blockIdx.x / R, b = seg / H, h = seg % H;
  const Seq L = sequence_of(a, b, t.max_new);
  const int units = prefix[a.B], p0 = prefix[b], nb = (prefix[b + 1] - p0) / H;
  if (row >= L.n * GQ) return;
  const int64_t tokrow = (a.cu ? a.cu[b] : b) + row / GQ;
  T *out = static_cast<T *>(t.out) + (tokrow * a.H_q + h * GQ + row % GQ) * D;
  float acc[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
  float lsum = 0.f, mw = -INFINITY;
  if (nb > 0) {
    const Cut cut(units, warps_used(units, warps_max));
    const int u0 = p0 + h * nb, w0 = cut.owner(u0), w1 = cut.owner(u0 + nb - 1);
    // this warp's partials: the maximum first, then the weighted sums
    const float *base = t.ws + ((int64_t)(w0 + seg) * R + row) * Part<D>::ROW;
    const int64_t step = (int64_t)R * Part<D>::ROW;
    const int count = w1 - w0 + 1;
    for (int i = warp + WARPS * lane; i < count; i += 32 * WARPS)
      mw = fmaxf(mw, base[i * step + D]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mw = fmaxf(mw, __shfl_xor_sync(kFull, mw, o));
#pragma unroll 4
    for (int i = warp; i < count; i += WARPS) {
      const float *p = base + i * step;
      const float2 ml = *reinterpret_cast<const float2 *>(p + D);
      const float f = part_factor(ml, mw);
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
    for (int i = 1; i < WARPS; ++i) M = fmaxf(M, rm[i]);
    float v = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
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

template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(32 * WARPS)
k_paged_merge(PagedArgs a, PagedAttend t, int warps_max, const int *prefix) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  merge_row<T, D, WARPS>(a, t, warps_max, prefix);
}

// The merge, and beside it, in CTAs of their own behind those of the output's
// rows, weights[token] += sum over the rows of 2^(score + top - maximum) / sum
// from the scores that the attention left.  Such a CTA takes 8 WARPS steps of a
// (sequence, kv head): it finds its rows' maxima and sums from the partials, as
// the merge does, then eight lanes take a step, four tokens each.  A token is one
// thread's, so that no two threads add to one place and the order of a sum is
// fixed.
//
// The scores are kept (4 bytes a row and token, written and read) rather than
// computed a second time: with 4 rows that is 32 bytes against the 80 of the
// key's codes at D = 128, g = 32, and no product.  Bound: latency.  In a kernel
// behind the merge, with the merge's maxima: 56.9 us a call where this takes
// 53.2 (16 sequences of 8192, 8 kv heads, 4 rows).
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(32 * WARPS)
k_paged_merge_weigh(PagedArgs a, PagedAttend t, int warps_max, const int *prefix,
                    const float *scores, PagedWeights w, float top, int out_rows, int chunks) {
  constexpr int STEPS = 8 * WARPS;
  __shared__ float2 stats[16];        // of each row: top - maximum, 1 / sum
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x < out_rows) {
    merge_row<T, D, WARPS>(a, t, warps_max, prefix);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int H = a.H_kv, R = t.max_new * (a.H_q / H);
  const int at = blockIdx.x - out_rows, seg = at / chunks, k0 = (at - seg * chunks) * STEPS,
            b = seg / H, h = seg - b * H;
  const int units = prefix[a.B], p0 = prefix[b], nb = (prefix[b + 1] - p0) / H;
  if (k0 >= nb) return;
  const Seq L = sequence_of(a, b, t.max_new);
  const int rows = L.n * (a.H_q / H), u0 = p0 + h * nb;
  const Cut cut(units, warps_used(units, warps_max));
  const int w0 = cut.owner(u0), count = cut.owner(u0 + nb - 1) - w0 + 1;
  for (int r = warp; r < rows; r += WARPS) {
    const float *ml = t.ws + ((int64_t)(w0 + seg) * R + r) * Part<D>::ROW + D;
    const int64_t step = (int64_t)R * Part<D>::ROW;
    float M = -INFINITY, sum = 0.f;
    for (int i = lane; i < count; i += 32) M = fmaxf(M, ml[i * step]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    for (int i = lane; i < count; i += 32) {
      const float2 x = *reinterpret_cast<const float2 *>(ml + i * step);
      sum = fmaf(part_factor(x, M), x.y, sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0)
      stats[r] = make_float2(M == -INFINITY ? 0.f : top - M, sum == 0.f ? 0.f : 1.f / sum);
  }
  __syncthreads();
  for (int k = k0 + 4 * warp + (lane >> 3); k < min(nb, k0 + STEPS); k += 4 * WARPS) {
    const int tok = k * kStep + 4 * (lane & 7);
    const float4 *x = reinterpret_cast<const float4 *>(scores + (int64_t)(u0 + k) * (R * kStep)) +
                      (lane & 7);
    float *to = w.at + b * w.seq + h * w.head + tok;
    const int n = min(4, L.len - tok);            // (none where the step ends behind the sequence)
    const bool wide = n == 4 && reinterpret_cast<uintptr_t>(to) % 16 == 0;
    float old[4], sum[4] = {0.f, 0.f, 0.f, 0.f};
    if (wide) {
      const float4 y = *reinterpret_cast<const float4 *>(to);
      old[0] = y.x; old[1] = y.y; old[2] = y.z; old[3] = y.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) old[i] = i < n ? to[i] : 0.f;
    }
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
      const float4 y = x[r * (kStep / 4)];
      const float2 f = stats[r];
      const float s[4] = {y.x, y.y, y.z, y.w};
      // a token that the row does not see gets nothing, whatever the others are
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += s[i] == -INFINITY ? 0.f : ex2(s[i] + f.x) * f.y;
    }
    if (wide) {
      *reinterpret_cast<float4 *>(to) =
          make_float4(old[0] + sum[0], old[1] + sum[1], old[2] + sum[2], old[3] + sum[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) to[i] = old[i] + sum[i];
    }
  }
}

// a partial per warp and per (sequence, kv head)
size_t part_floats(int B, int H_kv, int D, int rows, int sm_count) {
  return ((size_t)decode_ctas(D, rows) * sm_count * kWarps + (size_t)B * H_kv) * rows * (D + 4);
}

// workspace: partials, the prefixes; for kWeigh the scores of all steps that the
// tables have room for
size_t prefix_at(int B, int H_kv, int D, int rows, int sm_count) {
  return part_floats(B, H_kv, D, rows, sm_count) * sizeof(float);
}
size_t scores_at(int B, int H_kv, int D, int rows, int sm_count) {
  return (prefix_at(B, H_kv, D, rows, sm_count) + (B + 1) * sizeof(int) + 127) / 128 * 128;
}

template <int FORM, typename T, int D, int NG, int ROWS>
cudaError_t launch_dec(const PagedArgs &a, const PagedAttend &t, const PagedWeights *w,
                       int sm_count, cudaStream_t st) {
  using SM = DecSmem<D, NG, ROWS>;
  const size_t smem = SM::PREFIX + sizeof(int) * (a.B + 1);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_paged_decode<T, D, NG, ROWS, FORM>,
                             SM::PREFIX + (int)sizeof(int) * (kMaxSeqs + 1), done);
  if (e != cudaSuccess) return e;
  const int ctas = SM::CTAS * sm_count, warps_max = ctas * kWarps;
  const int rows = t.max_new * (a.H_q / a.H_kv);
  char *ws = reinterpret_cast<char *>(t.ws);
  int *prefixes = reinterpret_cast<int *>(ws + prefix_at(a.B, a.H_kv, D, rows, sm_count));
  float *scores = reinterpret_cast<float *>(ws + scores_at(a.B, a.H_kv, D, rows, sm_count));
  e = launch_pdl(k_paged_decode<T, D, NG, ROWS, FORM>, dim3(ctas), dim3(kThreads), smem, st, a,
                 t, warps_max, prefixes, FORM == kWeigh ? scores : nullptr);
  count_launch();
  if (e != cudaSuccess) return e;
  // many rows have few partials each (about warps_max over the number of
  // sequences and kv heads): 512 rows of 14, 4 warps 49.4 us a call, 16 warps
  // 51.4; 128 rows of 57, 8 warps 98.3 us, 16 warps 97.8
  const int out_rows = a.B * a.H_kv * rows;
  auto merge = [&](auto warps) {
    constexpr int W = decltype(warps)::value;
    if constexpr (FORM == kWeigh) {
      const int64_t steps = (((int64_t)a.max_pages << a.page_log2) + kStep - 1) / kStep,
                    chunks = (steps + 8 * W - 1) / (8 * W);
      return launch_pdl(k_paged_merge_weigh<T, D, W>,
                        dim3((unsigned)(out_rows + a.B * a.H_kv * chunks)), dim3(32 * W), 0, st,
                        a, t, warps_max, (const int *)prefixes, (const float *)scores, *w,
                        Weights<ROWS>::top, out_rows, (int)chunks);
    } else {
      return launch_pdl(k_paged_merge<T, D, W>, dim3(out_rows), dim3(32 * W), 0, st, a, t,
                        warps_max, (const int *)prefixes);
    }
  };
  e = out_rows >= 2 * sm_count ? merge(std::integral_constant<int, 4>{})
                               : merge(std::integral_constant<int, 16>{});
  count_launch();
  return e;
}

template <int FORM, typename T, int D, int NG>
cudaError_t launch_rows(const PagedArgs &a, const PagedAttend &t, const PagedWeights *w,
                        int sm_count, cudaStream_t st) {
  return t.max_new * (a.H_q / a.H_kv) <= 8
             ? launch_dec<FORM, T, D, NG, 8>(a, t, w, sm_count, st)
             : launch_dec<FORM, T, D, NG, 16>(a, t, w, sm_count, st);
}

template <int FORM, typename T>
cudaError_t launch_t(const PagedArgs &a, const PagedAttend &t, const PagedWeights *w, int D,
                     int sm_count, cudaStream_t st) {
  const int ng = D / a.g;
  if (D == 64)
    return ng == 1 ? launch_rows<FORM, T, 64, 1>(a, t, w, sm_count, st)
                   : launch_rows<FORM, T, 64, 2>(a, t, w, sm_count, st);
  return ng == 1   ? launch_rows<FORM, T, 128, 1>(a, t, w, sm_count, st)
         : ng == 2 ? launch_rows<FORM, T, 128, 2>(a, t, w, sm_count, st)
                   : launch_rows<FORM, T, 128, 4>(a, t, w, sm_count, st);
}

template <int FORM>
cudaError_t launch_form(int dtype, const PagedArgs &a, const PagedAttend &t,
                        const PagedWeights *w, int D, int sm_count, cudaStream_t st) {
  return dtype == VQ_F16 ? launch_t<FORM, __half>(a, t, w, D, sm_count, st)
                         : launch_t<FORM, __nv_bfloat16>(a, t, w, D, sm_count, st);
}

}  // namespace
}  // namespace vqk
