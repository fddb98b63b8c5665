// Causal attention of any number of new tokens over the paged 4-bit cache
// (vq_kivi_paged_attend), on tcgen05 with tensor-memory accumulators.
//
//   out = sum_t softmax_t(scale q.k_hat_t) v_hat_t,  t <= the row's own token
//
// Rows: 128 (new token, query head) pairs of a kv head make a query tile, two
// tiles a pair; a pair walks its keys 128 at a time.  The work is one line of
// key tiles over (sequence, kv head, pair, key tile), cut evenly among one CTA
// per SM whatever the lengths, so no plan on the host; a pair that is cut
// leaves partial rows, which a second kernel merges.
//
// A CTA works in two slots, so that one is multiplied while the other is in
// its softmax: the two query tiles of a pair, or, where the second would be
// empty, the even and the odd key tiles of one query tile (joined at the
// end).  Its warps:
//   0-3, 4-7   softmax of slot 0 and 1, one row a thread: scores from tensor
//              memory, online softmax in fp32, weights back to tensor memory
//              in fp16 (the A operand of the second product), the output
//              read out at the end.  Rounding a weight to fp16 moves it by
//              2^-11 of itself at most, as one rounding of an fp16 output
//              does, or by 2^-25 where fp16 has no smaller steps: 2^-34 of
//              the row's largest weight, which is 2^9 or more.
//   8-11       rebuild k_hat (fp16 by definition) from the codes into two
//   12-15      128-byte-swizzled stages, and v_hat likewise
//   16         issues the products: S = Q k_hat^T, then O += P v_hat
//   17, 18     copy the key and the value halves of the blocks (one bulk copy
//              each), 64 tokens a stage
// The running maximum of a row is a whole number (base 2), its weight 2^10,
// and it is raised only when a score passes it by more than 5: a weight stays
// within 2^15, which fp16 holds, one pass over a tile's scores is enough, and
// what was weighed with the old maximum is brought to a new one by an exact
// power of two.  More of fp16's range for the small weights means more raises
// (2 x 512 tokens at 33280: 464 us with 7 or 5 bits of headroom, 480 with 3).
//
// k_hat's channels lie in the order 0 4 1 5 2 6 3 7 within each 8, in which
// a code word gives its fp16 pairs; the queries are laid out the same.
// Every wait is bounded; a CTA that gives up sets the status word, drains and
// frees its tensor memory.
#include "bulk_pipe.cuh"
#include "paged.cuh"
#include "paged_words.cuh"
#include "vqk_internal.cuh"

namespace vqk {
namespace chunk {

constexpr int kThreads = 640;
constexpr int kTile = 128;           // keys of a tile, rows of a query tile
constexpr int kRaw = 3;              // stages of 64 tokens as stored
constexpr unsigned kFull = 0xffffffffu;
// exponents of a fresh maximum's weight and of the largest one (see above)
constexpr float kTop = 10.f, kMost = 15.f;
constexpr int kNear = 64;            // sequences whose prefix fits in shared memory
constexpr int kMinTiles = 2;         // key tiles a CTA takes at least
constexpr int kSliceRows = 16;       // rows that a CTA of the merge takes, one a warp

// ---- barriers ----------------------------------------------------------------

__device__ __forceinline__ void bar_init(uint64_t *b, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(count));
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(b)) : "memory");
}
// given up by its own limit, or soon after another role has
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, volatile int *dead) {
  if (bounded_wait(b, parity, dead)) return true;
  *dead = 1;
  return false;
}

// ---- tcgen05 -----------------------------------------------------------------

// 128-byte-swizzled K-major operand whose 8-row atoms (1024 B) follow one
// another: address >> 4, stride 1024 B between atoms, version 1, swizzle 2
__device__ __forceinline__ uint64_t desc128(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16, fp16 operands, fp32 accumulator, both K-major
__host__ __device__ constexpr uint32_t idesc(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// The issuing warp runs as a whole (its operands are then known to be uniform
// and stay in uniform registers); one elected lane issues the products of a
// tile, K in steps of 16.  One election a tile: one per product cost the warp
// more than the products take.  A step adds 32 bytes to an operand's start,
// 64 channels or tokens the next block of 128-byte rows.
#define VQK_SS(e, off)                                                            \
  " add.s64 x, %1, " #off ";\n add.s64 y, %2, " #off ";\n"                         \
  " @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, " e ";\n"
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
  if constexpr (D == 128)
    asm volatile(
        "{\n .reg .pred n, t, q;\n .reg .b64 x, y;\n setp.ne.b32 n, 0, 0;\n"
        " setp.eq.b32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n"
        VQK_SS("n", 0) VQK_SS("t", 2) VQK_SS("t", 4) VQK_SS("t", 6)
        VQK_SS("t", 1024) VQK_SS("t", 1026) VQK_SS("t", 1028) VQK_SS("t", 1030) "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred n, t, q;\n .reg .b64 x, y;\n setp.ne.b32 n, 0, 0;\n"
        " setp.eq.b32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n"
        VQK_SS("n", 0) VQK_SS("t", 2) VQK_SS("t", 4) VQK_SS("t", 6) "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id)
        : "memory");
}
// A (the weights) from tensor memory, 8 columns a step; acc: add to what is
// there
#define VQK_TS(e, col, off)                                                       \
  " add.u32 x, %1, " #col ";\n add.s64 y, %2, " off ";\n"                          \
  " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, " e ";\n"
template <int D>
__device__ __forceinline__ void mma_outputs(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                            uint32_t acc) {
  if constexpr (D == 128)
    asm volatile(
        "{\n .reg .pred n, t, q;\n .reg .b32 x;\n .reg .b64 y;\n setp.ne.b32 n, %4, 0;\n"
        " setp.eq.b32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n"
        VQK_TS("n", 0, "0") VQK_TS("t", 8, "2") VQK_TS("t", 16, "4") VQK_TS("t", 24, "6")
        VQK_TS("t", 32, "1024") VQK_TS("t", 40, "1026") VQK_TS("t", 48, "1028")
        VQK_TS("t", 56, "1030") "}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred n, t, q;\n .reg .b32 x;\n .reg .b64 y;\n setp.ne.b32 n, %4, 0;\n"
        " setp.eq.b32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n"
        VQK_TS("n", 0, "0") VQK_TS("t", 8, "2") VQK_TS("t", 16, "4") VQK_TS("t", 24, "6")
        VQK_TS("t", 32, "512") VQK_TS("t", 40, "514") VQK_TS("t", 48, "516")
        VQK_TS("t", 56, "518") "}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

#define VQK_R8(v, i)                                                              \
  "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]),     \
      "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define VQK_S8(v, i)                                                              \
  "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]),          \
      "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])

// 32 columns of this thread's lane
__device__ __forceinline__ void tm_ld32(uint32_t t, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : VQK_R8(v, 0), VQK_R8(v, 8), VQK_R8(v, 16), VQK_R8(v, 24)
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t t, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : VQK_R8(v, 0), VQK_R8(v, 8)
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tm_ld8(uint32_t t, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : VQK_R8(v, 0)
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t t, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(t),
      VQK_S8(v, 0)
      : "memory");
}
__device__ __forceinline__ void tm_ld64(uint32_t t, uint32_t (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : VQK_R8(v, 0), VQK_R8(v, 8), VQK_R8(v, 16), VQK_R8(v, 24), VQK_R8(v, 32),
        VQK_R8(v, 40), VQK_R8(v, 48), VQK_R8(v, 56)
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t t, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(t),
      VQK_S8(v, 0), VQK_S8(v, 8)
      : "memory");
}
// 2^d for a whole d <= 0 or -infinity
__device__ __forceinline__ float pow2(float d) {
  return d < -126.f ? 0.f : __int_as_float(((int)d + 127) << 23);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void tm_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---- the work line -------------------------------------------------------------

__device__ __forceinline__ int pairs_of(const Seq &s, int tpt) {
  return (s.n + 2 * tpt - 1) / (2 * tpt);
}
// key tiles that pair p of a sequence walks (one at least, so that rows
// without keys are written too)
__device__ __forceinline__ int tiles_of(const Seq &s, int p, int tpt) {
  const int limit = s.len - s.n + min(s.n, (p + 1) * 2 * tpt);
  return limit > kTile ? (limit + kTile - 1) / kTile : 1;
}

// prefix[b] = key tiles of sequences before b over all kv heads, b <= B; the
// whole CTA takes part
__device__ void tile_prefix(const PagedArgs &a, int max_new, int tpt, long long *prefix) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  for (int b = warp; b < a.B; b += nw) {
    const Seq s = sequence_of(a, b, max_new);
    const int np = pairs_of(s, tpt);
    long long sum = 0;
    for (int p = lane; p < np; p += 32) sum += tiles_of(s, p, tpt);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0) prefix[b + 1] = sum * a.H_kv;
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  __syncthreads();
  if (warp == 0) {
    long long base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      long long v = b0 + lane < a.B ? prefix[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += x;
      }
      if (b0 + lane < a.B) prefix[b0 + lane + 1] = base + v;
      base += __shfl_sync(kFull, v, 31);
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int ctas_used(long long units, int ctas) {
  const long long c = (units + kMinTiles - 1) / kMinTiles;
  return (int)(c < ctas ? c : ctas);
}
// the line's pieces differ by one tile at most
struct Cut {
  long long each;
  int more;
  __device__ Cut(long long units, int ctas) : each(units / ctas), more((int)(units % ctas)) {}
  __device__ long long first(int c) const { return each * c + (c < more ? c : more); }
};

// A place on the line: key tile k of pair `pair` of kv head h of sequence b,
// and how many tiles of the CTA's piece are left from here.  Kept small: every
// role holds one across its inner loop.
struct Walk {
  int left, b, h, pair, k;
  Seq s;
  __device__ int tiles(int tpt) const { return tiles_of(s, pair, tpt); }
  // tiles of this pair in the piece
  __device__ int steps(int tpt) const { return min(tiles(tpt) - k, left); }
  // both query tiles have rows
  __device__ bool two(int tpt) const { return pair * 2 * tpt + tpt < s.n; }
  // to tile u of the line, with n tiles left
  __device__ void seek(const PagedArgs &a, const long long *prefix, long long u, int n,
                       int max_new, int tpt) {
    left = n;
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= u) lo = mid; else hi = mid;
    }
    b = lo;
    s = sequence_of(a, b, max_new);
    const long long per = (prefix[b + 1] - prefix[b]) / a.H_kv;
    long long v = u - prefix[b];
    h = (int)(v / per);
    v -= h * per;
    pair = 0;
    for (int t = tiles_of(s, 0, tpt); v >= t; t = tiles_of(s, pair, tpt)) {
      v -= t;
      ++pair;
    }
    k = (int)v;
  }
  // to the next pair; false at the end of the piece
  __device__ bool advance(const PagedArgs &a, const long long *prefix, int max_new, int tpt) {
    left -= steps(tpt);
    if (left <= 0) return false;
    k = 0;
    if (++pair >= pairs_of(s, tpt)) {
      pair = 0;
      if (++h == a.H_kv) {
        h = 0;
        do { ++b; } while (prefix[b + 1] == prefix[b]);
        s = sequence_of(a, b, max_new);
      }
    }
    return true;
  }
};

// A pair whose keys were cut: left by the CTA that has its first tiles, read
// by the merge.
struct alignas(16) CutPair {
  int first;   // row of the token tensors of its first token
  int n;       // tokens from there on in the sequence (0: no cut pair)
  int h;       // kv head
  int last;    // CTA with its last tiles
};

// ---- shared memory --------------------------------------------------------------

template <int D, int NG>
struct Smem {
  static constexpr int KB = D / 64;
  static constexpr int OP = KB * 16384;            // one 128 x D fp16 operand
  static constexpr int BLK = 16 * D + 128 * NG, HALF = BLK / 2;   // keys, values
  static constexpr int Q = 0, K = 2 * OP, V = 4 * OP, RAW = 6 * OP;
  static constexpr int BAR = RAW + kRaw * 4 * BLK;
  static constexpr int PREFIX = BAR + 384;
  static constexpr int ALLOC = PREFIX + 8 * (kNear + 1) + 8 + 1024;   // room to align the base
};

// byte of 16-byte chunk `c` of row `r` in a tile of 128-byte swizzled rows
__device__ __forceinline__ int sw(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

struct Bars {
  uint64_t raw_full[2][kRaw], raw_empty[2][kRaw];   // keys, values
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
  uint64_t x_full, drain;
  uint32_t good[2][kRaw];   // which of a stage's 4 blocks arrived
  uint32_t tmem;
  int dead;
  CutPair cut;
};

template <typename T, int D, int NG>
__global__ void __launch_bounds__(kThreads, 1)
k_paged_chunk(PagedArgs a, PagedAttend t, float *part, float *swap, CutPair *cuts,
              long long *prefixes) {
  using SM = Smem<D, NG>;
  constexpr int I = D / 32, G = D / NG, BLK = SM::BLK;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  Bars &B = *reinterpret_cast<Bars *>(sm + SM::BAR);
  static_assert(sizeof(Bars) <= 384, "barriers fit");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int GQ = a.H_q / a.H_kv, tpt = kTile / GQ;
  if (tid == 0) {
    for (int i = 0; i < 2 * kRaw; ++i) {
      bar_init(&B.raw_full[0][0] + i, 1);
      bar_init(&B.raw_empty[0][0] + i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&B.k_full[i], 4);
      bar_init(&B.v_full[i], 4);
      bar_init(&B.k_empty[i], 1);
      bar_init(&B.v_empty[i], 1);
      bar_init(&B.q_full[i], 4);
      bar_init(&B.s_full[i], 1);
      bar_init(&B.p_full[i], 4);
      bar_init(&B.o_full[i], 1);
    }
    bar_init(&B.x_full, 4);
    bar_init(&B.drain, 1);
    B.dead = 0;
    B.cut.n = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
        smem_addr(&B.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  long long *prefix = a.B <= kNear
                          ? reinterpret_cast<long long *>(sm + SM::PREFIX)
                          : prefixes + (long long)blockIdx.x * (a.B + 1);
  tile_prefix(a, t.max_new, tpt, prefix);
  fence_after();
  const uint32_t tmem = B.tmem;
  volatile int *dead = &B.dead;
  const long long units = prefix[a.B];
  const int ctas = units > 0 ? ctas_used(units, gridDim.x) : 0;
  Walk walk;
  bool have = (int)blockIdx.x < ctas;
  if (have) {
    const Cut cut(units, ctas);
    const long long u = cut.first(blockIdx.x);
    walk.seek(a, prefix, u, (int)(cut.first(blockIdx.x + 1) - u), t.max_new, tpt);
  }
  auto advance = [&]() { return walk.advance(a, prefix, t.max_new, tpt); };

  // of the launch's 640 x 96 registers: 256 x 144 + 384 x 64 = 61440
  if (warp < 8) {
    // ---- softmax ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t ts = tl + 128 * wg, to = tl + 256 + 128 * wg;
    uint32_t ph_s = 0, ph_o = 0, ph_x = 0;
    float sl2 = 0.f;
    bool far_q = false;
    // query row of this thread, of the slot's query tile
    auto token = [&]() {
      return walk.pair * 2 * tpt + (walk.two(tpt) ? wg * tpt : 0) + row / GQ;
    };
    // this thread's query row into shared memory
    auto load_q = [&]() {
      const int tok = token();
      const bool valid = row < tpt * GQ && tok < walk.s.n;
      const T *q = static_cast<const T *>(t.q) + (int64_t)(walk.s.first + tok) * t.q_token +
                   (int64_t)(walk.h * GQ + row % GQ) * t.q_head;
      uint4 r[D / 8];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) r[c] = make_uint4(0u, 0u, 0u, 0u);
      if (valid) {
#pragma unroll
        for (int c = 0; c < D / 8; ++c) r[c] = reinterpret_cast<const uint4 *>(q)[c];
      }
      sl2 = t.scale;
      float up = 1.f;
      if constexpr (!std::is_same<T, __half>::value) {
        // a bf16 row as fp16: scaled by a power of two to a maximum near 2^14
        uint32_t m = 0u;               // largest magnitude, as bits
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t w[4] = {r[c].x, r[c].y, r[c].z, r[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m = max(m, max((w[e] << 16) & 0x7fffffffu, w[e] & 0x7fff0000u));
        }
        const RowScale rs = row_scale(m, t.scale);
        up = rs.up;
        sl2 = rs.back;
      }
      unsigned char *dst = sm + SM::Q + wg * SM::OP;
      __half2 size[2] = {bits_h2(0u), bits_h2(0u)};    // sum |q| / 256
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        uint32_t w[4] = {r[c].x, r[c].y, r[c].z, r[c].w};
        if constexpr (!std::is_same<T, __half>::value) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = h2_bits(__floats2half2_rn(__uint_as_float(w[i] << 16) * up,
                                             __uint_as_float(w[i] & 0xffff0000u) * up));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          size[i & 1] = __hfma2(__habs2(bits_h2(w[i])), bits_h2(0x1c001c00u), size[i & 1]);
        *reinterpret_cast<uint4 *>(dst + (c >> 3) * 16384 + sw(row, c & 7)) =
            make_uint4(__byte_perm(w[0], w[2], 0x5410), __byte_perm(w[0], w[2], 0x7632),
                       __byte_perm(w[1], w[3], 0x5410), __byte_perm(w[1], w[3], 0x7632));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(&B.q_full[wg]);
      // whether keys of fp16's size could take a row's scores beyond kFar (5 %
      // and 1 / 64 cover the roundings of the sum; NaN counts as yes)
      const float2 s2 = __half22float2(__hadd2(size[0], size[1]));
      far_q = __any_sync(kFull, !(65504.f * sl2 * (269.f * (s2.x + s2.y) + 0.015625f) <= kFar));
    };
    // key tiles before this pair, for the stages that they lie in
    uint32_t ring = 0;
    auto next = [&]() {
      ring += walk.steps(tpt);
      have = advance();
    };
    // past the pairs that this slot has no part in
    auto settle = [&]() {
      while (have && wg == 1 && !walk.two(tpt) && walk.steps(tpt) < 2) next();
    };
    // The stages go back to the rebuilding warps from here: a commit of the
    // tensor cores holds the next products up by more than 100 cycles, and
    // the scores' own already says that the products before them are done.
    // Slot 1 is the later user of a tile that both slots use.
    const bool gives = (warp & 3) == 0 && lane == 0;
    bool ok = true;
    settle();
    if (have) load_q();
    while (have && ok) {
      const int tok = token();
      const bool valid = row < tpt * GQ && tok < walk.s.n;
      // warps without a row leave the weights as they are: their rows of the
      // output are not read.  Rows without a query see everything.
      const bool idle = !__any_sync(kFull, valid);
      const bool two = walk.two(tpt);
      const int steps = walk.steps(tpt);
      const float raw = sl2;
      float m = -INFINITY, l = 0.f;
      // columns up to vis are seen
      int vis = (valid ? walk.s.len - walk.s.n + tok : 0x3fffffff) -
                (walk.k + (two ? 0 : wg)) * kTile;
      const int ahead = two ? kTile : 2 * kTile;
      // In one fma with the maximum a weight's exponent is off by the
      // maximum's own rounding, whole bits from 2^24 on: rows that may go
      // that far get their scores scaled, and rounded, beforehand, in a loop
      // of their own (a branch within the loop made all rows 3 to 5 % slower).
      auto tiles = [&](auto scaled_before) {
        constexpr bool before = decltype(scaled_before)::value;
        const float scale = before ? 1.f : raw;
        for (int j = two ? 0 : wg; j < steps; j += two ? 1 : 2, vis -= ahead) {
          ok = bar_wait(&B.s_full[wg], ph_s, dead);
          ph_s ^= 1u;
          if (!__all_sync(kFull, ok)) { ok = false; break; }
          fence_after();
          if (gives && (!two || wg == 1)) {
            bar_arrive(&B.k_empty[(ring + j) & 1]);
            // the values of this slot's tile before
            if (j >= (two ? 1 : 2)) bar_arrive(&B.v_empty[(ring + j - (two ? 1 : 2)) & 1]);
          }
          if (idle) {
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&B.p_full[wg]);
            continue;
          }
          if constexpr (before) {
#pragma unroll 1
            for (int c = 0; c < kTile; c += 16) {
              uint32_t v[16];
              tm_ld16(ts + c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * raw);
              tm_st16(ts + c, v);
            }
            tm_wait_st();
          }
          const bool all = __all_sync(kFull, vis >= kTile - 1);
          float mo = m;       // the maximum that the tile's weights stand on
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < kTile; c += 64) {
            uint32_t v[64];
            tm_ld64(ts + c, v);
            if (!all) {
#pragma unroll
              for (int j = 0; j < 64; ++j)
                if (c + j > vis) v[j] = __float_as_uint(-INFINITY);
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 64; j += 2)
              mx[j / 2 & 3] = max3(mx[j / 2 & 3], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
            const float top = scale * fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
            if (__any_sync(kFull, top + (kTop - mo) > kMost)) {
              const float mn = top + (kTop - mo) > kMost
                                   ? fmaxf(mo, stand_in(ceilf(top), kTop)) : mo;
              const float f = mn > mo ? pow2(mo - mn) : 1.f;
              l *= f;
              if (c > 0) {
                // the weights of this tile so far
                sum[0].x *= f; sum[0].y *= f; sum[1].x *= f; sum[1].y *= f;
                tm_wait_st();
#pragma unroll 1
                for (int d = 0; d < c / 2; d += 8) {
                  uint32_t p[8];
                  tm_ld8(ts + d, p);
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    // in fp32: the factor itself may be too small for fp16
                    const float2 y = __half22float2(bits_h2(p[j]));
                    p[j] = h2_bits(__floats2half2_rn(y.x * f, y.y * f));
                  }
                  tm_st8(ts + d, p);
                }
              }
              mo = mn;
            }
            const float base = mo == -INFINITY ? 0.f : kTop - mo;
#pragma unroll
            for (int d = 0; d < 64; d += 32) {
              uint32_t p[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[d + 2 * j]),
                                                        __uint_as_float(v[d + 2 * j + 1])),
                                            make_float2(scale, scale), make_float2(base, base));
                const float2 y = make_float2(ex2(x.x), ex2(x.y));
                sum[j & 1] = __fadd2_rn(sum[j & 1], y);
                p[j] = h2_bits(__floats2half2_rn(y.x, y.y));
              }
              // the weights of 32 columns take 16, all behind what is read
              tm_st16(ts + (c + d) / 2, p);
            }
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          // O goes to the new maximum
          if (j >= (two ? 1 : 2) && __any_sync(kFull, mo > m)) {
            const float f = mo > m ? pow2(m - mo) : 1.f;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t v[16];
              tm_ld16(to + c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
              tm_st16(to + c, v);
            }
          }
          m = mo;
          tm_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&B.p_full[wg]);
        }
      };
      if (far_q) tiles(std::true_type{});
      else tiles(std::false_type{});
      if (!ok) break;
      // slot 1 of a single query tile hands its sums to slot 0
      const bool halves = !two && steps > 1;
      const bool give = halves && wg == 1;
      const bool whole = walk.k == 0 && steps == walk.tiles(tpt);
      float *xr = swap + (blockIdx.x * kTile + row) * (D + 4);
      float *pr = give ? xr
                       : part + ((2 * blockIdx.x + (walk.k > 0 ? 0 : 1)) * 2 * kTile +
                                 (two ? wg * kTile : 0) + row) * (D + 4);
      T *orow = static_cast<T *>(t.out) +
                ((int64_t)(walk.s.first + tok) * a.H_q + walk.h * GQ + row % GQ) * D;
      // the stage of this slot's last tile
      const uint32_t vlast = (ring + (two ? steps - 1 : steps - 1 - ((steps - 1 - wg) & 1))) & 1;
      // the next queries: this slot's last scores have been read
      next();
      settle();
      if (have) load_q();
      ok = bar_wait(&B.o_full[wg], ph_o, dead);
      ph_o ^= 1u;
      if (!__all_sync(kFull, ok)) { ok = false; break; }
      fence_after();
      if (gives && (!two || wg == 1)) bar_arrive(&B.v_empty[vlast]);
      float f0 = 1.f, f1 = 0.f;
      if (halves && wg == 0) {
        ok = bar_wait(&B.x_full, ph_x, dead);
        ph_x ^= 1u;
        if (!__all_sync(kFull, ok)) { ok = false; break; }
        if (valid) {
          const float2 ml = *reinterpret_cast<const float2 *>(xr + D);
          const float M = fmaxf(m, ml.x);
          // a part without a seen token weighs nothing (NaN sums stay)
          f0 = m == -INFINITY ? (l != l ? l : 0.f) : ex2(m - M);
          f1 = ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.f) : ex2(ml.x - M);
          l = l * f0 + ml.y * f1;
          m = M;
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (!idle) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          __syncwarp();
          tm_ld32(to + c, v);
          if (halves && wg == 0 && valid) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 x = *reinterpret_cast<const float4 *>(xr + c + j);
              v[j] = __float_as_uint(__uint_as_float(v[j]) * f0 + x.x * f1);
              v[j + 1] = __float_as_uint(__uint_as_float(v[j + 1]) * f0 + x.y * f1);
              v[j + 2] = __float_as_uint(__uint_as_float(v[j + 2]) * f0 + x.z * f1);
              v[j + 3] = __float_as_uint(__uint_as_float(v[j + 3]) * f0 + x.w * f1);
            }
          }
          if (valid && whole && !give) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(v[j + e]) * inv;
              store8<T>(orow + c + j, y);
            }
          } else if (valid) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4 *>(pr + c + j) =
                  make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          }
        }
        if (valid && (give || !whole)) *reinterpret_cast<float2 *>(pr + D) = make_float2(m, l);
      }
      __syncwarp();
      if (give && lane == 0) bar_arrive(&B.x_full);
      fence_before();
    }
  } else if (warp < 16) {
    // ---- k_hat (warps 8-11) and v_hat (12-15) ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int kv = (warp - 8) >> 2, w = warp & 3, n8 = lane >> 2, t4 = lane & 3;
    uint64_t *full = kv ? B.v_full : B.k_full, *empty = kv ? B.v_empty : B.k_empty;
    uint32_t raw = 0, ph_raw = 0, st = 0, ph_e = 1;    // stages start empty
    bool ok = true;
    // values: where this lane's four stores of an octet go, and the shifts to
    // the nibbles that they hold (the lanes of a store differ in the channel's
    // low bits)
    uint32_t to[4], shift[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = (q + t4) & 3;
      to[q] = sw(32 * t4 + 4 * n8 + r, 2 * w);
      shift[q] = 4 * r;
    }
    const __half2 k1024 = bits_h2(0x64006400u), k16 = bits_h2(0x2c002c00u),
                  k64 = bits_h2(0xd400d400u);
    for (; ok && have; have = advance()) {
      const int steps = walk.steps(tpt);
      // the sequence's tokens from this tile on
      int left = walk.s.len - walk.k * kTile;
      for (int j = 0; ok && j < steps; ++j, left -= kTile) {
        ok = bar_wait(&empty[st], ph_e, dead);
        unsigned char *dst = sm + (kv ? SM::V : SM::K) + st * SM::OP;
        for (int hf = 0; hf < 2; ++hf) {
          ok = ok && bar_wait(&B.raw_full[kv][raw], ph_raw, dead);
          if (!__all_sync(kFull, ok)) { ok = false; break; }
          // warp w takes block w of the stage
          const unsigned char *blk = sm + SM::RAW + ((kv * kRaw + raw) * 4 + w) * SM::HALF;
          const bool good = (B.good[kv][raw] >> w) & 1u;
          const int r0 = 64 * hf + 16 * w;             // its first key in the tile
          if (!kv) {
            // the 8 lanes of a 16-byte store hold rows r and r + 4, whose
            // swizzled chunks meet 8 different bank groups
            const int nr = (n8 >> 1) | ((n8 & 1) << 2);
            uint32_t kw[2][I];
            uint2 km[2][NG];
#pragma unroll
            for (int oct = 0; oct < 2; ++oct) {
              const int tk = 8 * oct + nr;
              load_words<I>(blk + tk * (D / 2) + t4 * (4 * I), kw[oct]);
              load_meta<NG>(blk + off_km(D) + (tk >> 1) * (8 * NG), km[oct]);
            }
            const unsigned sel = !good ? 0x4444u : (nr & 1) ? 0x3232u : 0x1010u;
            unsigned char *row = dst + (r0 + nr) * 128;
            // chunk t4 of the row's lower half; the upper half is chunk t4 + 4
            const int lower = (t4 ^ nr) << 4, upper = lower ^ 64;
#pragma unroll
            for (int oct = 0; oct < 2; ++oct) {
              __half2 s, z;
#pragma unroll
              for (int i = 0; i < I; ++i) {
                if ((32 * i) % G == 0) {
                  s = bits_h2(__byte_perm(km[oct][32 * i / G].x, 0u, sel));
                  z = bits_h2(__byte_perm(km[oct][32 * i / G].y, 0u, sel));
                }
                uint32_t x = kw[oct][i], o[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const __half2 c0 = __hsub2(field<0x000f000fu>(x), k1024);
                  const __half2 c1 = __hfma2(field<0x00f000f0u>(x), k16, k64);
                  o[2 * j] = h2_bits(__hfma2(c0, s, z));
                  o[2 * j + 1] = h2_bits(__hfma2(c1, s, z));
                  x >>= 8;
                }
                *reinterpret_cast<uint4 *>(row + oct * 1024 + (i >> 1) * 16384 +
                                           ((i & 1) ? upper : lower)) =
                    make_uint4(o[0], o[1], o[2], o[3]);
              }
            }
          } else {
            // lane (n8, t4) reads the words of token pair t4, then the four
            // lanes of n8 exchange them, so that lane j has the four pairs (8
            // tokens) of the 32-channel span j
#pragma unroll
            for (int oct = 0; oct < 2; ++oct) {
              uint32_t x[4] = {0u, 0u, 0u, 0u};
              const unsigned char *vp = blk + (32 * oct + lane) * (4 * I);
              if constexpr (I == 4) {
                const uint4 y = *reinterpret_cast<const uint4 *>(vp);
                x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
              } else {
                const uint2 y = *reinterpret_cast<const uint2 *>(vp);
                x[0] = y.x; x[1] = y.y;
              }
              // 4 x 4 transposition over the lanes t4 in two exchanges
              {
                const bool o1 = t4 & 1, o2 = t4 & 2;
                uint32_t s0 = o1 ? x[0] : x[1], s1 = o1 ? x[2] : x[3];
                s0 = __shfl_xor_sync(kFull, s0, 1);
                s1 = __shfl_xor_sync(kFull, s1, 1);
                if (o1) { x[0] = s0; x[2] = s1; } else { x[1] = s0; x[3] = s1; }
                s0 = o2 ? x[0] : x[2];
                s1 = o2 ? x[1] : x[3];
                s0 = __shfl_xor_sync(kFull, s0, 2);
                s1 = __shfl_xor_sync(kFull, s1, 2);
                if (o2) { x[0] = s0; x[1] = s1; } else { x[2] = s0; x[3] = s1; }
              }
              const int span = t4;
              if (I == 4 || span < I) {
                const uint2 *vm = reinterpret_cast<const uint2 *>(blk + 8 * D) + 4 * oct * NG +
                                  32 * span / G;
                uint2 m[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) m[p] = vm[p * NG];
                if (!good || left < r0 + 16) {
                  // tokens behind the sequence hold anything: their values
                  // become 0
#pragma unroll
                  for (int p = 0; p < 4; ++p) {
                    const int e = left - (r0 + 8 * oct + 2 * p);
                    const unsigned keep = !good || e <= 0 ? 0u : (e == 1 ? 0x0000ffffu : kFull);
                    m[p].x &= keep;
                    m[p].y &= keep;
                  }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  uint32_t o[4];
#pragma unroll
                  for (int p = 0; p < 4; ++p) {
                    const __half2 cc = __hsub2(field<0x000f000fu>(x[p] >> shift[q]), k1024);
                    o[p] = h2_bits(__hfma2(cc, bits_h2(m[p].x), bits_h2(m[p].y)));
                  }
                  *reinterpret_cast<uint4 *>(dst + hf * (D * 128) + (to[q] ^ (oct << 4))) =
                      make_uint4(o[0], o[1], o[2], o[3]);
                }
              }
            }
          }
          __syncwarp();
          if (lane == 0) bar_arrive(&B.raw_empty[kv][raw]);
          raw = raw + 1 == kRaw ? 0 : raw + 1;
          ph_raw ^= raw == 0;
        }
        if (!ok) break;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(&full[st]);
        st ^= 1u;
        ph_e ^= st == 0;
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  }
  if (warp == 16) {
    // ---- the products ----
    {
      const uint32_t id_s = idesc(kTile, kTile), id_o = idesc(kTile, D);
      const uint32_t sb = smem_addr(sm);
      uint32_t ks = 0, ph_k = 0, vs = 0, ph_v = 0, ph_q = 0, ph_p = 0;   // a bit a slot
      bool ok = true;
      const uint64_t dq = desc128(sb + SM::Q), dk = desc128(sb + SM::K),
                     dv = desc128(sb + SM::V);
      auto scores = [&](int i, uint32_t stage) {
        mma_scores<D>(tmem + 128 * i, dq + i * (SM::OP >> 4), dk + stage * (SM::OP >> 4), id_s);
        mma_commit(&B.s_full[i]);
      };
      auto outputs = [&](int i, uint32_t stage, bool more) {
        mma_outputs<D>(tmem + 256 + 128 * i, tmem + 128 * i, dv + stage * (SM::OP >> 4), id_o,
                       more);
      };
      // waits for the keys of the next tile, and goes on from them
      auto keys = [&]() {
        const bool r = __all_sync(kFull, bar_wait(&B.k_full[ks], ph_k, dead));
        fence_after();
        return r;
      };
      auto keys_done = [&]() {
        ks ^= 1u;
        ph_k ^= ks == 0;
      };
      for (; ok && have; have = advance()) {
        const int nt = walk.steps(tpt);
        const bool two = walk.two(tpt);
        const int slots = two || nt > 1 ? 2 : 1;
        // first scores of both slots: one key tile for two query tiles, or a
        // key tile each for one
        for (int i = 0; ok && i < slots; ++i) {
          ok = __all_sync(kFull, bar_wait(&B.q_full[i], (ph_q >> i) & 1u, dead));
          ph_q ^= 1u << i;
          if (ok && (i == 0 || !two)) ok = keys();
          if (!ok) break;
          fence_after();
          scores(i, ks);
          if (!two || i + 1 == slots) keys_done();
        }
        for (int j = 0; ok && j < nt; ++j) {
          ok = __all_sync(kFull, bar_wait(&B.v_full[vs], ph_v, dead));
          const bool last = two ? j + 1 == nt : j + 2 >= nt;
          for (int i = two ? 0 : j & 1, n = two ? 2 : i + 1; ok && i < n; ++i) {
            ok = __all_sync(kFull, bar_wait(&B.p_full[i], (ph_p >> i) & 1u, dead));
            ph_p ^= 1u << i;
            if (!ok) break;
            fence_after();
            outputs(i, vs, two ? j > 0 : j > 1);
            if (last) {
              mma_commit(&B.o_full[i]);
            } else {
              if (i == 0 || !two) ok = keys();
              if (!ok) break;
              scores(i, ks);
              if (!two || i == 1) keys_done();
            }
          }
          if (!ok) break;
          vs ^= 1u;
          ph_v ^= vs == 0;
        }
      }
      // products in flight end before the tensor memory is given up
      mma_commit(&B.drain);
      int never = 0;
      bar_wait(&B.drain, 0, &never);
    }
  } else if (warp == 17 || warp == 18) {
    // ---- copies: keys (17) and values (18) ----
    const int kv = warp - 17, bpp = a.page_log2 - 4;
    uint32_t raw = 0, ph_e = 1;
    uint32_t used = 0;             // stages with copies not known to have landed
    bool ok = true;
    for (; ok && have; have = advance()) {
      if (kv && lane == 0 && walk.k == 0 && walk.steps(tpt) < walk.tiles(tpt)) {
        // the pair goes on in the next CTAs' pieces
        const Cut cut(units, ctas);
        int last = blockIdx.x;
        for (long long rest = walk.tiles(tpt) - walk.steps(tpt); rest > 0; ++last)
          rest -= cut.each + (last + 1 < cut.more ? 1 : 0);
        const int tok0 = walk.pair * 2 * tpt;
        B.cut = CutPair{walk.s.first + tok0, walk.s.n - tok0, walk.h, last};
      }
      const int nblk = (walk.s.len + kBlk - 1) / kBlk, end = 2 * (walk.k + walk.steps(tpt));
      // lane j looks up block 4 k4 + j of the next 8 stages at once, so that
      // a table's latency is met once in 512 tokens
      const uint8_t *src = nullptr;
      unsigned there = 0u;
      for (int k4 = 2 * walk.k, i = 0; ok && k4 < end; ++k4, i = (i + 1) & 7) {
        if (i == 0) {
          const int blk = 4 * k4 + lane;
          bool good = blk < nblk && blk < 4 * end;
          if (good) {
            const int p = a.table[(int64_t)walk.b * a.table_stride + (blk >> bpp)];
            if ((unsigned)p >= (unsigned)a.n_pages) {
              atomicOr(a.status, kBadPage);
              good = false;
            }
            src = a.pool + ((((int64_t)p * a.H_kv + walk.h) << bpp) + (blk & ((1 << bpp) - 1))) *
                               BLK + kv * SM::HALF;
          }
          there = __ballot_sync(kFull, good);
        }
        ok = bar_wait(&B.raw_empty[kv][raw], ph_e, dead);
        if (!__all_sync(kFull, ok)) { ok = false; break; }
        const unsigned mask = (there >> (4 * i)) & 15u;
        if (lane == 0) {
          B.good[kv][raw] = mask;
          mbar_expect_tx(&B.raw_full[kv][raw], __popc(mask) * SM::HALF);
        }
        __syncwarp();
        if (lane >> 2 == i && (there >> lane & 1u))
          bulk_g2s(sm + SM::RAW + ((kv * kRaw + raw) * 4 + (lane & 3)) * SM::HALF, src, SM::HALF,
                   &B.raw_full[kv][raw]);
        used |= 1u << raw;
        raw = raw + 1 == kRaw ? 0 : raw + 1;
        ph_e ^= raw == 0;
      }
    }
    // copies in flight land before the shared memory is given up: the phase
    // of a stage's last copies is the one before its next turn's
    if (lane == 0) {
      for (int i = 0; i < kRaw; ++i) {
        int never = 0;
        const uint32_t turn = (uint32_t)i < raw ? ph_e ^ 1u : ph_e;   // parity of its last full
        if ((used >> i) & 1u) bar_wait(&B.raw_full[kv][i], turn, &never);
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (tid == 0) {
    if (B.dead) atomicOr(a.status, kGaveUp);
    cuts[blockIdx.x] = B.cut;
  }
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// Merge of a pair whose keys were cut: CTA (slice, c) merges 16 rows of the
// pair that CTA c of the attention began and did not end.  One warp per row,
// lanes over channels.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kSliceRows)
k_paged_chunk_merge(PagedArgs a, PagedAttend t, const float *part, const CutPair *cuts) {
  constexpr int CPL = D / 32, ROW = D + 4;
  const int c = blockIdx.y, lane = threadIdx.x & 31,
            r = blockIdx.x * kSliceRows + (threadIdx.x >> 5);
  const int GQ = a.H_q / a.H_kv, tpt = kTile / GQ;
  const int row = r & 127, tok = (r >> 7) * tpt + row / GQ;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 q = *reinterpret_cast<const int4 *>(&cuts[c]);
  const CutPair cut{q.x, q.y, q.z, q.w};
  if (row >= tpt * GQ || tok >= cut.n) return;
  auto at = [&](int i) {
    return part + ((int64_t)(i == c ? 2 * c + 1 : 2 * i) * 2 * kTile + r) * ROW;
  };
  // the first two parts are there for every cut pair: on their way before the
  // maximum is known
  float v[2][CPL], m2[2], l2[2];
  auto load = [&](int i, float (&x)[CPL], float &pm, float &pl) {
    const float *p = at(i);
    const float2 ml = *reinterpret_cast<const float2 *>(p + D);
    pm = ml.x;
    pl = ml.y;
    if constexpr (CPL == 4) {
      const float4 y = *reinterpret_cast<const float4 *>(p + 4 * lane);
      x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
    } else {
      const float2 y = *reinterpret_cast<const float2 *>(p + 2 * lane);
      x[0] = y.x; x[1] = y.y;
    }
  };
  load(c, v[0], m2[0], l2[0]);
  load(c + 1, v[1], m2[1], l2[1]);
  float M = fmaxf(m2[0], m2[1]);
  if (cut.last > c + 1) {
    for (int i = c + 2 + lane; i <= cut.last; i += 32) M = fmaxf(M, at(i)[D]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  }
  float L = 0.f, acc[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
  auto add = [&](const float (&x)[CPL], float pm, float pl) {
    // a part without a seen token weighs nothing (NaN sums stay)
    const float f = pm == -INFINITY ? (pl != pl ? pl : 0.f) : ex2(pm - M);
    L = fmaf(f, pl, L);
#pragma unroll
    for (int e = 0; e < CPL; ++e) acc[e] = fmaf(f, x[e], acc[e]);
  };
  add(v[0], m2[0], l2[0]);
  add(v[1], m2[1], l2[1]);
#pragma unroll 4
  for (int i = c + 2; i <= cut.last; ++i) {
    load(i, v[0], m2[0], l2[0]);
    add(v[0], m2[0], l2[0]);
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  T *o = static_cast<T *>(t.out) +
         ((int64_t)(cut.first + tok) * a.H_q + cut.h * GQ + row % GQ) * D + CPL * lane;
#pragma unroll
  for (int e = 0; e < CPL; e += 2) {
    if constexpr (std::is_same<T, __half>::value)
      *reinterpret_cast<__half2 *>(o + e) = __floats2half2_rn(acc[e] * inv, acc[e + 1] * inv);
    else
      *reinterpret_cast<__nv_bfloat162 *>(o + e) =
          __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
  }
}

// two partials (pairs cut at either end of a CTA's piece) of 256 rows a CTA,
// and 128 rows for what slot 1 hands to slot 0
size_t part_floats(int D, int sm_count) { return (size_t)2 * sm_count * 2 * kTile * (D + 4); }
size_t swap_floats(int D, int sm_count) { return (size_t)sm_count * kTile * (D + 4); }

template <typename T, int D, int NG>
cudaError_t launch_d(const PagedArgs &a, const PagedAttend &t, int sm_count, cudaStream_t st) {
  using SM = Smem<D, NG>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_paged_chunk<T, D, NG>, SM::ALLOC, done);
  if (e != cudaSuccess) return e;
  float *part = t.ws, *swap = part + part_floats(D, sm_count);
  CutPair *cuts = reinterpret_cast<CutPair *>(swap + swap_floats(D, sm_count));
  long long *prefixes = reinterpret_cast<long long *>(cuts + sm_count);
  e = launch_pdl(k_paged_chunk<T, D, NG>, dim3(sm_count), dim3(kThreads), SM::ALLOC, st, a, t,
                 part, swap, cuts, prefixes);
  count_launch();
  if (e != cudaSuccess) return e;
  // rows of a pair that can hold queries: one tile's, or both tiles'
  const int GQ = a.H_q / a.H_kv;
  const int slices = t.max_new <= kTile / GQ ? (t.max_new * GQ + kSliceRows - 1) / kSliceRows
                                             : 2 * kTile / kSliceRows;
  e = launch_pdl(k_paged_chunk_merge<T, D>, dim3(slices, sm_count), dim3(32 * kSliceRows), 0,
                 st, a, t, (const float *)part, (const CutPair *)cuts);
  count_launch();
  return e;
}

template <typename T>
cudaError_t launch_t(const PagedArgs &a, const PagedAttend &t, int D, int sm_count,
                     cudaStream_t st) {
  const int ng = D / a.g;
  if (D == 64)
    return ng == 1 ? launch_d<T, 64, 1>(a, t, sm_count, st)
                   : launch_d<T, 64, 2>(a, t, sm_count, st);
  return ng == 1   ? launch_d<T, 128, 1>(a, t, sm_count, st)
         : ng == 2 ? launch_d<T, 128, 2>(a, t, sm_count, st)
                   : launch_d<T, 128, 4>(a, t, sm_count, st);
}

}  // namespace chunk

size_t paged_chunk_ws(int B, int, int D, int sm_count) {
  return (chunk::part_floats(D, sm_count) + chunk::swap_floats(D, sm_count)) * sizeof(float) +
         sm_count * sizeof(chunk::CutPair) +
         (size_t)sm_count * (B + 1) * sizeof(long long);
}

cudaError_t launch_paged_chunk(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                               int sm_count, cudaStream_t st) {
  return dtype == VQ_F16 ? chunk::launch_t<__half>(a, t, D, sm_count, st)
                         : chunk::launch_t<__nv_bfloat16>(a, t, D, sm_count, st);
}

}  // namespace vqk
