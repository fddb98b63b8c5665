// Tokens of the paged 4-bit cache that stay and move together, as codes: the
// kept path of a tree of drafts (vq_kivi_paged_keep), and the tokens of the
// largest accumulated weights (vq_kivi_paged_evict).
#include "cluster.cuh"
#include "paged.cuh"
#include "vqk_internal.cuh"

namespace vqk {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBatch = 8;         // tokens that a warp reads before it writes them

// ---- one token's codes -----------------------------------------------------------
//
// A token is D / 2 + 4 D / g values of 16 bits in its block: key codes side by
// side, value codes every second one (the other is its pair's other token),
// (scale, min) likewise.  A lane takes every 32nd of them; value i of token tl
// lies at a + (tl >> 3) x + (tl / 2 mod 4) y + (tl & 1) z.
template <int D, int NG>
struct TokenLanes {
  static constexpr int I = D / 32, N = D / 2 + 4 * NG, PER = (N + 31) / 32;
  int a[PER], x[PER], y[PER], z[PER];
  __device__ __forceinline__ explicit TokenLanes(int lane) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      int e = lane + 32 * i;
      a[i] = -1;
      x[i] = y[i] = z[i] = 0;
      if (e >= N) continue;
      const bool value = e >= N / 2;
      if (value) e -= N / 2;
      const int half = value ? 4 * D + 32 * NG : 0;
      if (e >= D / 4) {                                 // (scale, min) of a group
        e -= D / 4;
        a[i] = half + 4 * D + (e % NG) * 4 + 2 * (e / NG);
        x[i] = 16 * NG;
        y[i] = 4 * NG;
        z[i] = 1;
      } else if (value) {
        a[i] = half + 2 * ((e / I) * 4 * I + e % I);
        x[i] = 64 * I;
        y[i] = 2 * I;
        z[i] = 1;
      } else {
        a[i] = e;
        x[i] = 2 * D;
        y[i] = D / 2;
        z[i] = D / 4;
      }
    }
  }
  __device__ __forceinline__ int at(int i, int tl) const {
    return a[i] + (tl >> 3) * x[i] + ((tl >> 1) & 3) * y[i] + (tl & 1) * z[i];
  }
  __device__ __forceinline__ void load(const uint8_t *blk, int tl, uint16_t (&v)[PER]) const {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (a[i] >= 0) v[i] = reinterpret_cast<const uint16_t *>(blk)[at(i, tl)];
  }
  __device__ __forceinline__ void store(uint8_t *blk, int tl, const uint16_t (&v)[PER]) const {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (a[i] >= 0) reinterpret_cast<uint16_t *>(blk)[at(i, tl)] = v[i];
  }
};

// The block of position pos in kv head 0, as a number; -1 (and the status bit)
// where its page is not one of the pool.
__device__ __forceinline__ int64_t block_of(const PagedArgs &a, int b, int pos) {
  const int p = a.table[(int64_t)b * a.table_stride + (pos >> a.page_log2)];
  if ((unsigned)p >= (unsigned)a.n_pages) {
    atomicOr(a.status, kBadPage);
    return -1;
  }
  return (((int64_t)p * a.H_kv) << (a.page_log2 - 4)) + ((pos & ((1 << a.page_log2) - 1)) >> 4);
}

// Up to kBatch tokens of a warp: lane j0 + j has the blocks and places of token
// j's source and destination (source block -1: no token, or none to move).  All
// are read before `between` is called and any is written.
template <int D, int NG, typename F>
__device__ __forceinline__ void move_batch(const PagedArgs &a, const TokenLanes<D, NG> &lanes,
                                           int h, int j0, int n, int64_t from, int from_tl,
                                           int64_t to, int to_tl, F between) {
  constexpr int BLK = paged_block_bytes(D, D / NG);
  const int64_t head = (int64_t)h << (a.page_log2 - 4);
  uint16_t v[kBatch][TokenLanes<D, NG>::PER];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    if (j >= n) break;
    const int64_t s = __shfl_sync(kFull, from, j0 + j);
    const int tl = __shfl_sync(kFull, from_tl, j0 + j);
    if (s >= 0) lanes.load(a.pool + (s + head) * BLK, tl, v[j]);
  }
  between();
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    if (j >= n) break;
    const int64_t s = __shfl_sync(kFull, from, j0 + j), d = __shfl_sync(kFull, to, j0 + j);
    const int tl = __shfl_sync(kFull, to_tl, j0 + j);
    if (s >= 0) lanes.store(a.pool + (d + head) * BLK, tl, v[j]);
  }
}

// ---- the kept path of a tree -----------------------------------------------------

// One CTA a sequence, so that its length can be written where it was read; a
// warp a kv head.  The path rises, so that a token moves to its own place or an
// earlier one, and what a warp writes was read by it before: kBatch tokens at a
// time, the earlier ones first.
template <int D, int NG>
__global__ void __launch_bounds__(1024)
k_paged_keep(PagedArgs a, const int32_t *path, const int32_t *counts, int32_t *lens_out) {
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int raw = a.lens[b];
  const Seq s = sequence_of(a, b, kMaxTree);
  const int count = counts[b];
  const int base = s.len - s.n, lead = base < 0 ? -base : 0;   // new tokens before the cache
  const int start = base + lead;
  const bool in = count >= 0 && count <= s.n - lead;
  int node[2] = {0, 0};
  bool rises = true;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    if (in && j < count) {
      node[i] = path[s.first + j];
      const int before = j > 0 ? path[s.first + j - 1] : lead - 1;
      rises = rises && node[i] > before && node[i] < s.n;
    }
  }
  const bool good = __all_sync(kFull, in && rises);
  if (!good && threadIdx.x == 0) atomicOr(a.status, kBadPath);
  __syncthreads();                      // every warp has read the length
  if (threadIdx.x == 0) lens_out[b] = s.n == 0 || !good ? raw : start + count;
  if (s.n == 0 || !good) return;
  // blocks of this lane's two tokens
  int64_t from[2] = {-1, -1}, to[2] = {-1, -1};
  int from_tl[2] = {0, 0}, to_tl[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    if (j >= count || base + node[i] == start + j) continue;
    from[i] = block_of(a, b, base + node[i]);
    to[i] = block_of(a, b, start + j);
    if (to[i] < 0) from[i] = -1;
    from_tl[i] = (base + node[i]) & 15;
    to_tl[i] = (start + j) & 15;
  }
  const TokenLanes<D, NG> lanes(lane);
  for (int h = warp; h < a.H_kv; h += blockDim.x >> 5)
    for (int j0 = 0; j0 < count; j0 += kBatch) {
      const int i = j0 >> 5;
      move_batch<D, NG>(a, lanes, h, j0 & 31, min(kBatch, count - j0), i ? from[1] : from[0],
                        i ? from_tl[1] : from_tl[0], i ? to[1] : to[0], i ? to_tl[1] : to_tl[0],
                        [] { __syncwarp(); });
      __syncwarp();
    }
}

// ---- eviction ----------------------------------------------------------------------

// Weights in an order of whole numbers: NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct EvictSmem {
  uint32_t hist[2][256];
  uint32_t counts[2];       // this CTA's weights above the threshold, and at it
  uint32_t warp[32], own[32];
  uint32_t digit[3];        // the digit found, how many of its weights stay, how many it has
  uint32_t kept;            // tokens before K that stay (the CTA that has place K)
};

// One cluster a (sequence, kv head).  K = budget - recent places in front hold
// the first tokens and the heaviest of the others, the newest tokens follow in
// their order.
//   1  the threshold: the weight of rank K - first, found 8 bits at a time from
//      counts per digit
//   2  the tokens before K that go are places to fill, the tokens behind K that
//      stay fill them: both lists in rising order, written by ranks from counts
//   3  the places are filled; the newest tokens move down
// Nothing else moves: sources of 3 lie at K or behind, places before K, so no
// token is overwritten before it is read.
template <int D, int NG, int THREADS, bool ONE>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
k_paged_evict(PagedArgs a, PagedEvict e) {
  __shared__ EvictSmem sm;
  constexpr int nw = THREADS / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned rank = ONE ? 0u : cluster_rank(), ctas = ONE ? 1u : cluster_ctas();
  const int row = blockIdx.x / ctas, b = row / a.H_kv, h = row - b * a.H_kv;
  auto all_sync = [] {                // of all threads of the row
    if constexpr (ONE) __syncthreads();
    else cluster_sync();
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int len = a.lens[b];
  const bool ok = len >= 0 && len <= a.max_len;
  const float *in = e.in.at + b * e.in.seq + h * e.in.head;
  float *out = e.out.at + b * e.out.seq + h * e.out.head;
  const bool same = e.in.at == e.out.at;
  if (h == 0 && rank == 0 && tid == 0) {
    if (!ok) atomicOr(a.status, kBadLength);
    e.lens_out[b] = ok && len > e.budget ? e.budget : len;
  }
  const int64_t step = (int64_t)ctas * THREADS, me = (int64_t)rank * THREADS + tid;
  if (!ok || len <= e.budget) {
    // as it was, and zero behind; a length outside its range says nothing of
    // where that is
    const int64_t n = ok ? len : e.in.capacity;
    for (int64_t p = (same ? n : 0) + me; p < e.out.capacity; p += step)
      out[p] = p < n ? in[p] : 0.f;
    return;
  }
  const int K = e.budget - e.recent, lo = e.first, hi = len - e.recent;
  const int per = (hi - lo + (int)ctas - 1) / (int)ctas;
  const int p0 = min(lo + (int)rank * per, hi), p1 = min(p0 + per, hi);
  // this CTA's weights in an order of whole numbers, several on their way
  auto each = [&](auto f) {
    constexpr int U = 8;
    for (int q = p0; q < p1; q += U * THREADS) {
      float w[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int p = q + i * THREADS + tid;
        w[i] = p < p1 ? in[p] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int p = q + i * THREADS + tid;
        if (p < p1) f(p, order_of(w[i]));
      }
    }
  };

  // ---- 1: the threshold ----
  uint32_t found = 0u, mask = 0u;
  int need = K - lo;                  // how many of the weights at the threshold stay
  uint32_t above_here = 0u, equal_here = 0u;
  if (need > 0) {
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      uint32_t *hist = sm.hist[(shift >> 3) & 1];
      for (int i = tid; i < 256; i += THREADS) hist[i] = 0u;
      __syncthreads();
      each([&](int, uint32_t u) {
        if (((u ^ found) & mask) == 0u) atomicAdd(&hist[(u >> shift) & 255u], 1u);
      });
      all_sync();
      // thread t: digit 255 - t, over the cluster and of this CTA, and how many
      // lie above it
      uint32_t here = 0u, inc = 0u, own = 0u, own_inc = 0u;
      if (tid < 256) {
        own = hist[255 - tid];
        here = own;
        if (!ONE) {
          here = 0u;
#pragma unroll
          for (unsigned r = 0; r < 8; ++r)
            if (r < ctas) here += peer_load(&hist[255 - tid], r);
        }
        inc = here;
        own_inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(kFull, inc, o), w = __shfl_up_sync(kFull, own_inc, o);
          if (lane >= o) {
            inc += v;
            own_inc += w;
          }
        }
        if (lane == 31) {
          sm.warp[warp] = inc;
          sm.own[warp] = own_inc;
        }
      }
      __syncthreads();
      if (tid < 256) {
        uint32_t above = inc - here, mine = own_inc - own;
        for (int w = 0; w < warp; ++w) {
          above += sm.warp[w];
          mine += sm.own[w];
        }
        if (above < (uint32_t)need && (uint32_t)need <= above + here) {
          sm.digit[0] = 255 - tid;
          sm.digit[1] = need - above;
          sm.digit[2] = here;
          sm.counts[0] = mine;
          sm.counts[1] = own;
        }
      }
      __syncthreads();
      found |= sm.digit[0] << shift;
      need = (int)sm.digit[1];
      mask |= 255u << shift;
      above_here += sm.counts[0];
      equal_here = sm.counts[1];
      if (sm.digit[2] == (uint32_t)need) break;    // all of them stay: no need to tell them apart
    }
  } else {
    found = mask = kFull;             // none stays
  }
  // the lower bits may be left open
  auto is_above = [&](uint32_t u) { return (u & mask) > found; };
  auto is_at = [&](uint32_t u) { return (u & mask) == found; };

  // ---- 2: places to fill and tokens that fill them ----
  int above = 0, equal = 0;           // before this CTA's weights
  if (!ONE) {
    __syncthreads();                  // the last pass's counts have been read
    if (tid == 0) {
      sm.counts[0] = above_here;
      sm.counts[1] = equal_here;
    }
    all_sync();
#pragma unroll
    for (unsigned r = 0; r < 8; ++r)
      if (r < rank) {
        above += (int)peer_load(&sm.counts[0], r);
        equal += (int)peer_load(&sm.counts[1], r);
      }
  }
  // pairs: the n-th place to fill, and the n-th token that stays
  int2 *pairs = e.pairs + (int64_t)row * K;
  constexpr int V = 4;                // neighbouring weights of a thread
  for (int q0 = p0; q0 < p1; q0 += V * THREADS) {
    const int q = q0 + V * tid;
    float w[V];
    uint32_t gt = 0u, eq = 0u;        // a bit each
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = q + i < p1 ? in[q + i] : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t u = order_of(w[i]);
      gt |= (q + i < p1 && is_above(u) ? 1u : 0u) << i;
      eq |= (q + i < p1 && is_at(u) ? 1u : 0u) << i;
    }
    const uint32_t own = __popc(gt) | (__popc(eq) << 16);
    uint32_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();                  // the last tile's counts have been read
    if (lane == 31) sm.warp[warp] = inc;
    __syncthreads();
    uint32_t ahead = 0u, total = 0u;
#pragma unroll
    for (int k = 0; k < nw; ++k) {
      if (k < warp) ahead += sm.warp[k];
      total += sm.warp[k];
    }
    ahead += inc - own;
    const int g = above + (int)(ahead & 0xffffu), x = equal + (int)(ahead >> 16);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = q + i;
      if (p >= p1) break;
      const uint32_t below = (1u << i) - 1u;
      // of the weights at the threshold the first ones stay
      const int n_eq = x + __popc(eq & below), kept = g + __popc(gt & below) + min(n_eq, need);
      const bool stays = ((gt >> i) & 1u) || (((eq >> i) & 1u) && n_eq < need);
      if (p == K) sm.kept = (uint32_t)kept;
      if (p < K) {
        if (!stays) pairs[p - lo - kept].x = p;
        else if (!same) out[p] = w[i];
      } else if (stays) {
        pairs[kept].y = p;
      }
    }
    above += (int)(total & 0xffffu);
    equal += (int)(total >> 16);
  }
  if (!same) {
    for (int64_t p = me; p < lo; p += step) out[p] = in[p];
    for (int64_t p = e.budget + me; p < e.out.capacity; p += step) out[p] = 0.f;
  }
  all_sync();

  // ---- 3: the places are filled ----
  // (K lies among the weights: more than K - first of them compete)
  const unsigned at_k = (unsigned)((K - lo) / per);
  const int kept_k = (int)(ONE ? sm.kept : peer_load(&sm.kept, at_k)), holes = K - lo - kept_k;
  const TokenLanes<D, NG> lanes(lane);
  const int gw = (int)rank * nw + warp;
  // a lane looks up a pair, then the warp moves kBatch of them at a time
  for (int i0 = 0; i0 < holes; i0 += (int)ctas * nw * 32) {
    // the warps share what is left evenly
    const int left = holes - i0, share = min(32, (left + (int)ctas * nw - 1) / ((int)ctas * nw)),
              first = i0 + gw * share, n = min(share, holes - first);
    int64_t from = -1, to = -1;
    int src = 0, dst = 0;
    if (lane < n) {
      dst = pairs[first + lane].x;
      src = pairs[kept_k + first + lane].y;
      from = block_of(a, b, src);
      to = block_of(a, b, dst);
      if (to < 0) from = -1;
      out[dst] = in[src];
    }
    for (int j = 0; j < n; j += kBatch)
      move_batch<D, NG>(a, lanes, h, j, min(kBatch, n - j), from, src & 15, to, dst & 15, [] {});
  }
  // the newest tokens move down by hi - K places, the front ones first: all CTAs
  // have read a round (and, in the first, what fills places) before any writes
  const int round = (int)ctas * nw * kBatch;
  for (int r0 = 0; r0 < e.recent; r0 += round) {
    const int left = e.recent - r0,
              share = min(kBatch, (left + (int)ctas * nw - 1) / ((int)ctas * nw)),
              i0 = r0 + gw * share, n = max(0, min(share, e.recent - i0));
    int64_t from = -1, to = -1;
    int src = 0, dst = 0;
    float w = 0.f;
    if (lane < n) {
      src = hi + i0 + lane;
      dst = K + i0 + lane;
      from = block_of(a, b, src);
      to = block_of(a, b, dst);
      if (to < 0) from = -1;
      w = in[src];
    }
    move_batch<D, NG>(a, lanes, h, 0, n, from, src & 15, to, dst & 15, all_sync);
    if (lane < n) out[dst] = w;
  }
  if (same || !ONE) all_sync();       // (no CTA ends while others read its counts)
  if (same)
    for (int64_t p = e.budget + me; p < e.out.capacity; p += step) out[p] = 0.f;
}

template <int D, int NG>
cudaError_t keep_d(const PagedArgs &a, const int32_t *path, const int32_t *counts,
                   int32_t *lens_out, cudaStream_t st) {
  const int warps = a.H_kv < 32 ? a.H_kv : 32;
  cudaError_t e = launch_pdl(k_paged_keep<D, NG>, dim3(a.B), dim3(32 * warps), 0, st, a, path,
                             counts, lens_out);
  count_launch();
  return e;
}

template <int D, int NG, int THREADS, bool ONE>
cudaError_t evict_t(const PagedArgs &a, const PagedEvict &v, int cluster, cudaStream_t st) {
  const dim3 grid(a.B * a.H_kv * cluster), block(THREADS);
  cudaError_t e = ONE ? launch_pdl(k_paged_evict<D, NG, THREADS, ONE>, grid, block, 0, st, a, v)
                      : launch_cluster(k_paged_evict<D, NG, THREADS, ONE>, grid, block, cluster,
                                       0, st, a, v);
  count_launch();
  return e;
}

// Short rows, longer ones of which few tokens go, and any when there are many
// take one CTA of few threads: no barriers of a cluster, and four on an SM.
// Others are shared by as many CTAs as there is room for.  One CTA of 256 threads
// against clusters of up to 8 of 512 (one of 512 from 256 rows on), with the
// read-back, us (8 kv heads of D = 128; tables as long as the sequences):
//             1025 > 1024  1025 > 512  2049 > 2048  2049 > 1024  4097 > 4096  4097 > 2048
//   8 rows     9.0 / 13.0  16.1 / 16.7  11.1 / 14.0  24.6 / 17.7  14.6 / 15.7  42.5 / 19.0
//   64 rows   18.4 / 22.0  21.1 / 20.8  25.8 / 31.6  36.2 / 30.5  44.0 / 46.6  65.9 / 44.4
//   256 rows  41.2 / 42.4  38.5 / 38.5  71.9 / 72.4  66.1 / 64.3   125 / 125    120 / 117
//   608       84.6 / 91.7  73.3 / 76.8   149 / 154    135 / 136    276 / 281    254 / 253
//   1216       156 / 171    136 / 145    283 / 296    253 / 255    540 / 551    483 / 479
//   2432       300 / 327    255 / 277    553 / 578    478 / 486
// (at 8193 > 8192, 8 rows: 26.5 / 21.4)
// The rule goes by the tables' room, as the host does not know the lengths.  Tables
// of 131072 places take the cluster below 8 rows an SM, which their weights want in
// any case: all places behind the budget are cleared.
//             513 > 512    1025 > 1024  1025 > 512   2049 > 2048  4097 > 2048
//   8 rows    16.8 / 13.5  17.4 / 14.0  23.5 / 16.2  18.9 / 14.8  50.5 / 19.7
//   64 rows   23.1 / 24.6  26.2 / 28.3  30.6 / 27.9  35.8 / 36.7  74.4 / 48.2
//   256 rows  47.3 / 48.1  61.9 / 62.2  60.7 / 60.1  90.2 / 89.7   144 / 138
template <int D, int NG>
cudaError_t evict_d(const PagedArgs &a, const PagedEvict &v, int sm_count, cudaStream_t st) {
  const int64_t rows = (int64_t)a.B * a.H_kv;
  const int64_t room = (int64_t)a.max_pages << a.page_log2;
  const bool few_go = room - v.budget <= 128 && room <= 6144;
  if (room <= 1536 || few_go || rows >= 8 * sm_count)
    return evict_t<D, NG, 256, true>(a, v, 1, st);
  int c = 1;
  while (c < 8 && room > 1024 * c && rows * c <= sm_count) c *= 2;
  return c == 1 ? evict_t<D, NG, 512, true>(a, v, 1, st)
                : evict_t<D, NG, 512, false>(a, v, c, st);
}

}  // namespace

cudaError_t launch_paged_keep(const PagedArgs &a, const int32_t *path, const int32_t *counts,
                              int32_t *lens_out, int D, cudaStream_t st) {
  const int ng = D / a.g;
  if (D == 64)
    return ng == 1 ? keep_d<64, 1>(a, path, counts, lens_out, st)
                   : keep_d<64, 2>(a, path, counts, lens_out, st);
  return ng == 1   ? keep_d<128, 1>(a, path, counts, lens_out, st)
         : ng == 2 ? keep_d<128, 2>(a, path, counts, lens_out, st)
                   : keep_d<128, 4>(a, path, counts, lens_out, st);
}

size_t paged_evict_ws(int B, int H_kv, int budget, int recent) {
  return (size_t)B * H_kv * (budget - recent) * sizeof(int2);
}

cudaError_t launch_paged_evict(const PagedArgs &a, const PagedEvict &e, int D, int sm_count,
                               cudaStream_t st) {
  const int ng = D / a.g;
  if (D == 64)
    return ng == 1 ? evict_d<64, 1>(a, e, sm_count, st) : evict_d<64, 2>(a, e, sm_count, st);
  return ng == 1   ? evict_d<128, 1>(a, e, sm_count, st)
         : ng == 2 ? evict_d<128, 2>(a, e, sm_count, st)
                   : evict_d<128, 4>(a, e, sm_count, st);
}

}  // namespace vqk
