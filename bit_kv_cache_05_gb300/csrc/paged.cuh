// The paged 4-bit cache: layout, what a call says about its batch, and the
// launchers of its operators.
//
// Pool: [n_pages][H_kv][page / 16][block], a block holding 16 tokens of one kv
// head in one contiguous run of 16 D + 128 D / g bytes (2560 at D = 128,
// g = 32), so that one bulk copy brings everything an attention step needs:
//   key codes    16 rows of D / 2 bytes; word (D / 32) t + i of a row (t < 4)
//                holds channels 32 i + 8 t ... + 7, lowest nibble first
//   key meta     per token pair (2 p, 2 p + 1) and group: s, s', z, z' (fp16)
//   value codes  word ((8 h + n) 4 + t) (D / 32) + i: channels 32 i + 4 n ... + 3
//                of token 8 h + 2 t in the low half, of the next in the high half
//   value meta   as key meta
// In these orders lane (n = lane / 4, t = lane % 4) of a warp finds its
// operands of mma.m16n8k16 in consecutive words: for the scores the codes of
// token n (B fragments, one 16-byte load per 8 tokens at D = 128), for the
// output the channel quads 4 n of its two token pairs.  Two neighbouring
// 16-bit halves of a word shifted by 4 r always form one fp16 pair.
//
// A stored value stands for fp16(code * s + z), rounded once: what the
// attention kernels multiply and vq_kivi_paged_dequantize returns.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "bulk_pipe.cuh"
#include "rope.cuh"
#include "vq_kivi.h"

namespace vqk {

constexpr int kMaxSeqs = 1024;   // sequences of one paged call
constexpr int kBlk = 16;         // tokens of a block
constexpr int kMaxTree = 64;     // nodes of a tree of drafts: bits of a mask
constexpr int kMaxLen = 0x7fff0000;   // tokens of a sequence: a place and what a
                                      // kernel takes at once fit in 31 bits

// status bits (device word)
constexpr unsigned kBadPage = 1u;     // a block table entry outside the pool
constexpr unsigned kBadLength = 2u;   // lens / cu_new outside their ranges
constexpr unsigned kGaveUp = 4u;      // a bounded wait ran out
constexpr unsigned kBadPath = 8u;     // a path of kept tokens outside its tree

__host__ __device__ constexpr int paged_meta_bytes(int D, int g) { return 64 * (D / g); }
__host__ __device__ constexpr int paged_block_bytes(int D, int g) {
  return 2 * (8 * D + paged_meta_bytes(D, g));
}

// bytes into a block: key codes, key meta, value codes, value meta
__host__ __device__ constexpr int off_km(int D) { return 8 * D; }
__host__ __device__ constexpr int off_vc(int D, int g) { return 8 * D + paged_meta_bytes(D, g); }
__host__ __device__ constexpr int off_vm(int D, int g) {
  return 16 * D + paged_meta_bytes(D, g);
}

struct PagedArgs {
  uint8_t *pool;
  unsigned *status;
  const int32_t *table;      // [B][max_pages]
  const int32_t *lens;       // [B] tokens of each sequence, the new ones among them
  const int32_t *cu;         // [B + 1] offsets of the new tokens, nullptr: one each
  int64_t table_stride;
  int64_t tokens;            // new tokens the token tensors have room for
  int n_pages, page_log2, max_pages, B;
  int H_q, H_kv, g;
  int max_len;               // tokens that a table has room for, kMaxLen at most
};

// What a call says of sequence b: tokens, new tokens, row of the first new one.
struct Seq {
  int len, n, first;
};

// One whose lengths lie outside their ranges counts as empty (and sets the
// status bit).  max_new: no sequence has more new tokens.
__device__ __forceinline__ Seq sequence_of(const PagedArgs &a, int b, int max_new) {
  Seq s{a.lens[b], 1, b};
  if (a.cu) {
    s.first = a.cu[b];
    s.n = a.cu[b + 1] - s.first;
  }
  if (s.len < 0 || s.len > a.max_len || s.n < 0 || s.n > max_new ||
      s.first < 0 || (int64_t)s.first + s.n > a.tokens) {
    atomicOr(a.status, kBadLength);
    s.len = s.n = 0;
  }
  return s;
}

// sequence of new token i and its place in the sequence (-1: not in the
// cache): the new tokens of a sequence are its last ones
struct Place {
  int b, pos;
};

// As sequence_of, ranges are checked.  Sequences that no token leads to are
// looked at as well, so that every operator reports the same of a batch: by
// warps beyond those of the tokens, a lane a sequence (`look`, else -1), which
// get no place.  (Looking in a branch of its own made the append of four
// ragged chunks 71 us instead of 69.)
__device__ __forceinline__ Place find_place(const PagedArgs &a, int64_t i, int64_t look) {
  int lo = (int)i, end = (int)i + 1;
  bool in = true;
  if (look >= 0 && (!a.cu || look >= a.B)) return Place{-1, -1};
  if (a.cu) {
    int hi = a.B;
    lo = 0;
    if (look >= 0) {
      lo = (int)look;
      hi = lo + 1;
    } else if (i < a.cu[0] || i >= a.cu[a.B]) {
      return Place{-1, -1};
    }
    while (hi - lo > 1) {   // cu[lo] <= i < cu[hi]
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= i) lo = mid; else hi = mid;
    }
    end = a.cu[hi];
    in = a.cu[lo] >= 0 && end >= a.cu[lo] && end <= a.tokens;
  }
  const int len = a.lens[lo];
  if (!in || len < 0 || len > a.max_len) {
    atomicOr(a.status, kBadLength);
    return Place{lo, -1};
  }
  const int pos = look >= 0 ? -1 : len - (end - (int)i);
  return Place{lo, pos < 0 ? -1 : pos};
}

// Which of the new tokens row `tok` of a sequence's tree sees: bits of new
// tokens that the sequence does not have are left out.
__device__ __forceinline__ unsigned long long tree_mask(const unsigned long long *tree,
                                                        const Seq &s, int tok) {
  const unsigned long long all = s.n >= kMaxTree ? ~0ull : (1ull << s.n) - 1ull;
  return tree[s.first + tok] & all;
}

// The columns that a row sees of 64 whose first lies `at` behind the last token
// before the new ones: a column before them is seen.
__device__ __forceinline__ unsigned long long tree_columns(unsigned long long mask, int at) {
  if (at >= 64) return 0ull;
  if (at >= 0) return mask >> at;
  if (at > -64) return (mask << -at) | ((1ull << -at) - 1ull);
  return ~0ull;
}

// A row of a tree: its mask and where the new tokens begin.  own: the place of
// the row's own token (negative: padding, or no row), which sees nothing.
struct TreeRow {
  unsigned long long mask;
  int base;
  __device__ __forceinline__ bool sees(int token) const {
    const int j = token - base;
    return j < 0 || (j < 64 && ((mask >> j) & 1ull));
  }
};
__device__ __forceinline__ TreeRow tree_row(const unsigned long long *tree, const Seq &s, int tok,
                                            int own) {
  if (own < 0) return TreeRow{0ull, -0x3fffffff};
  return TreeRow{tree_mask(tree, s, tok), s.len - s.n};
}

// the block of kv head h that holds position pos of sequence b, nullptr (and
// the status bit) when its page is not one of the pool
__device__ __forceinline__ uint8_t *find_block(const PagedArgs &a, int b, int pos, int h,
                                               int block_bytes) {
  const int p = a.table[(int64_t)b * a.table_stride + (pos >> a.page_log2)];
  if ((unsigned)p >= (unsigned)a.n_pages) {
    atomicOr(a.status, kBadPage);
    return nullptr;
  }
  const int in = (pos & ((1 << a.page_log2) - 1)) >> 4;
  return a.pool + ((((int64_t)p * a.H_kv + h) << (a.page_log2 - 4)) + in) * block_bytes;
}

// A bf16 query row enters the products as fp16, times the power of two that
// brings its largest magnitude (`top`, the bits of an fp32) near 2^14; `back`
// is the scores' factor for it.  Both are normal numbers for every top,
// infinity and NaN among them, and every scale: a factor of 0 or infinity would
// make masked scores (-infinity), or scores of 0, NaN.
struct RowScale {
  float up, back;
};

__device__ __forceinline__ RowScale row_scale(uint32_t top, float scale) {
  int f = top ? 14 - ((int)(top >> 23) - 127) : 0;     // -114 ... 141
  f = f > 126 ? 126 : f;
  const float back = scale * __uint_as_float((uint32_t)(127 - f) << 23);
  return RowScale{__uint_as_float((uint32_t)(127 + f) << 23),
                  fminf(fmaxf(back, 1.17549435e-38f), 3.40282347e+38f)};
}

// Far maxima.  A weight is 2^(score - maximum + top), a few bits above 1 for
// the largest.  From 2^24 on fp32 has no room for those bits beside the
// maximum, so that they are left out there (2^(score - maximum), which is
// what a maximum larger by `top` gives); kFar leaves the nearer ones exact.
constexpr float kFar = 8388608.f;
__device__ __forceinline__ bool is_far(float m) {
  return fabsf(m) > kFar && m != -INFINITY;
}
__device__ __forceinline__ float stand_in(float m, float top) {
  return is_far(m) ? m + top : m;
}

// Waits for a barrier's phase; false after about half a second, or soon after
// *dead (when given) is set.  Reading the clock between the tries is also the
// pause that a waiting warp leaves the others: tries with none, with
// nanosleep (20 to 300) or with a long suspend hint made the chunk attention
// 10 to 20 % slower (2 x 512 tokens at 33280: 514 us, the others 590 to 690).
__device__ __forceinline__ bool bounded_wait(uint64_t *bar, uint32_t parity,
                                             volatile int *dead = nullptr) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (dead && *dead) return false;
    if (global_ns() - t0 > 500000000ull) return false;
  }
  return true;
}

// Dynamic shared memory of a kernel beyond 48 KB, allowed once per device
template <typename F>
inline cudaError_t allow_smem(F *fn, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// The operators wait for the stream's previous kernel before they read
// anything.  Those whose outputs a caller sees do not release their
// dependents early: the contiguous cache's append loads its input rows before
// its own programmatic wait, and those rows may come from norm_rope or from
// the read-back.  Only the attention kernels release their merges early.
cudaError_t launch_norm_rope(int dtype, const HeadRows &q, const HeadRows &k,
                             const RopeArgs &r, int D, int64_t tokens, float eps,
                             int sm_count, cudaStream_t st);
cudaError_t launch_paged_append(int dtype, const PagedArgs &a, const HeadRows &q,
                                const HeadRows &k, const HeadRows &v, const RopeArgs &r,
                                bool rotate_by_place, int D, float eps, int sm_count,
                                cudaStream_t st);
cudaError_t launch_paged_dequantize(const PagedArgs &a, __half *K, __half *V, int D,
                                    int sm_count, cudaStream_t st);

struct PagedAttend {
  const void *q;
  void *out;
  int64_t q_token, q_head;   // element strides; out is [tokens][H_q][D]
  float scale;
  int max_new;               // no sequence has more new tokens
  float *ws;                 // workspace
  const unsigned long long *tree = nullptr;   // mask of each new token
};

// accumulated weights: element (sequence, kv head, token) at at[b seq + h head + t]
struct PagedWeights {
  float *at;
  int64_t seq, head, capacity;   // capacity: places of a row
};

// few rows: up to 16 (new token, query head) pairs per kv head
size_t paged_decode_ws(int B, int H_kv, int D, int rows, int sm_count);
cudaError_t launch_paged_decode(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                                int sm_count, cudaStream_t st);
cudaError_t launch_paged_decode_tree(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                                     int sm_count, cudaStream_t st);
// capacity: tokens that a sequence's table has room for
size_t paged_weigh_ws(int B, int H_kv, int D, int rows, int64_t capacity, int sm_count);
cudaError_t launch_paged_weigh(int dtype, const PagedArgs &a, const PagedAttend &t,
                               const PagedWeights &w, int D, int sm_count, cudaStream_t st);
// any number of new tokens
size_t paged_chunk_ws(int B, int H_kv, int D, int sm_count);
cudaError_t launch_paged_chunk(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                               int sm_count, cudaStream_t st);
cudaError_t launch_paged_chunk_tree_small(int dtype, const PagedArgs &a, const PagedAttend &t,
                                          int D, int sm_count, cudaStream_t st);
cudaError_t launch_paged_chunk_tree(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                                    int sm_count, cudaStream_t st);


// tokens that stay move together: new tokens along a path (launch_paged_keep),
// or those that weigh most, per kv head (launch_paged_evict)
cudaError_t launch_paged_keep(const PagedArgs &a, const int32_t *path, const int32_t *counts,
                              int32_t *lens_out, int D, cudaStream_t st);
struct PagedEvict {
  PagedWeights in, out;
  int32_t *lens_out;
  int budget, recent, first;
  int2 *pairs;               // workspace: (place to fill, token that fills it)
};
size_t paged_evict_ws(int B, int H_kv, int budget, int recent);
cudaError_t launch_paged_evict(const PagedArgs &a, const PagedEvict &e, int D, int sm_count,
                               cudaStream_t st);

// verification of drafted tokens (drafts.cu)
struct Drafts {
  const void *target, *draft;          // rows of V probabilities, of one type
  int64_t target_row, draft_row;       // element strides
  const void *tokens;
  const int32_t *parents, *cu;
  const float *uniforms;
  int32_t *path, *counts;
  void *after;
  int64_t rows;                        // rows of the token arrays
  int B, V, tokens64;
};
cudaError_t launch_verify(int dtype, const Drafts &d, int sm_count, cudaStream_t st);

}  // namespace vqk
