// Verification of drafted tokens (vq_kivi_verify_drafts): a walk down each
// sequence's tree, and a token drawn where the walk ends.
//
// With p the target's row of the node that the walk is at and q the draft's, a
// rejected child leaves the residual max(p - q, 0), normed.  Rejections after
// the first have the same q, so that the residual of k of them is
//   w = max(p - c q, 0) / S,   S = sum w,   c' = c + S   (c = 0 and S = 1 first)
// and nothing of a row is kept between two children: a row is read once per
// rejection.  Without q the drafted tokens stand for themselves: a rejected one
// is taken out of p, S falls by what it had.
//
// Sums are whole numbers of 2^-44 (each value rounded once; 2^63 of them in a
// row of 2^19 values of 1), so no order of summation changes a decision or
// a token; products are taken in 64 bits.
//
// Bound: two rows of V values a sequence from HBM, or with few sequences the
// chain of loads (offsets, tokens, probabilities, row) and barriers.  A cluster
// takes a sequence; each CTA walks (all of them the same way) and sums its
// slice of the row, each warp a piece of it, 16 bytes a lane.
#include "cluster.cuh"
#include "paged.cuh"
#include "rope.cuh"
#include "vqk_internal.cuh"

namespace vqk {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr double kUnit = 17592186044416.0;           // 2^44

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// What is left of a value: max(p - c q, 0), rounded once, at most 1; a NaN
// counts as nothing.
__device__ __forceinline__ float left_of(float p, float q, float c) {
  float w;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(w) : "f"(-c), "f"(q), "f"(p));
  return w;
}

// Whole numbers of 2^-44 in two halves of 22 bits, each the low bits of an fp32
// next to 2^23: whole = floor(w 2^22), then the rest, rounded to the nearest.
// (With conversions to 64-bit integers 64 sequences with rows of 131072 took 54
// us instead of 30.)  The halves of up to 1023 values add up in 32 bits.
struct Halves {
  uint32_t hi = 0u, lo = 0u;
  __device__ __forceinline__ void add(float w) {
    const float t = __fmaf_rd(w, 4194304.f, 8388608.f);
    const float rest = __fmaf_rn(w, 4194304.f, 8388608.f - t);
    hi += __float_as_uint(t) - 0x4b000000u;
    lo += __float_as_uint(__fmaf_rn(rest, 4194304.f, 8388608.f)) - 0x4b000000u;
  }
  __device__ __forceinline__ unsigned long long units() const {
    return ((unsigned long long)hi << 22) + lo;
  }
};
__device__ __forceinline__ unsigned long long units_of(float w) {
  Halves h;
  h.add(__saturatef(w));
  return h.units();
}
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// N neighbouring values of a row from v on, 16 bytes of it: at once where they
// are all in the row and lie on a 16-byte boundary (`wide`), else one by one;
// 0 outside.
template <typename T>
struct Values {
  static constexpr int N = 16 / sizeof(T);
  float x[N];
  __device__ __forceinline__ void load(const T *row, int v, int V, bool wide) {
    if (wide && v >= 0 && v + N <= V) {
      const uint4 u = *reinterpret_cast<const uint4 *>(row + v);
      const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = as_float(e[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = v + i >= 0 && v + i < V ? as_float(row[v + i]) : 0.f;
    }
  }
};

struct VerifySmem {
  uint64_t totals[2][8];            // of the cluster's CTAs, of the last two sums
  uint64_t warp[kWarps];            // of this CTA's warps, of the last sum
  int64_t token[kMaxTree];
  double uq[kMaxTree];              // uniform times q, or the uniform
  float p[kMaxTree], q[kMaxTree];
  int parent[kMaxTree];
  int good[kMaxTree];               // accepted if it is the first that is tried
  int gone[kMaxTree];               // without q: the rejected tokens
  uint64_t run[kWarps];             // of the last search: sums of runs of steps
  float last;                       // the uniform of the last draw
  int bad;
};

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kThreads)
k_verify(Drafts d) {
  __shared__ VerifySmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned rank = cluster_rank(), ctas = cluster_ctas();
  const int b = blockIdx.x / ctas;
  const T *target = static_cast<const T *>(d.target), *draft = static_cast<const T *>(d.draft);
  cluster_began();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int start = d.cu[b], n = d.cu[b + 1] - start;
  const bool lead = rank == 0 && tid == 0;
  auto put = [&](int64_t after, int count) {
    d.counts[b] = count;
    if (d.tokens64) static_cast<int64_t *>(d.after)[b] = after;
    else static_cast<int32_t *>(d.after)[b] = (int)after;
  };
  if (n <= 0 || n > kMaxTree || start < 0 || (int64_t)start + n > d.rows) {
    // (more nodes than a tree has: their rows are there)
    if (rank == 0 && start >= 0 && (int64_t)start + n <= d.rows)
      for (int i = tid; i < n; i += kThreads) d.path[start + i] = -1;
    if (lead) put(-1, n == 0 ? 0 : -1);
    cluster_runs();
    return;
  }
  // nodes: their tokens, and what their parents' rows say of them
  if (tid == 0) sm.bad = 0;
  __syncthreads();
  if (tid < kMaxTree) {
    sm.parent[tid] = -1;
    if (tid < n) {
      const int64_t x = d.tokens64 ? static_cast<const int64_t *>(d.tokens)[start + tid]
                                   : static_cast<const int32_t *>(d.tokens)[start + tid];
      const int parent = d.parents ? d.parents[start + tid] : tid - 1;
      const float u = d.uniforms[start + tid];
      if (tid == 0) sm.last = u;
      if (tid > 0) {
        if (parent < 0 || parent >= tid || x < 0 || x >= d.V) {
          sm.bad = 1;
        } else {
          sm.parent[tid] = parent;
          sm.token[tid] = x;
          const float p = as_float(target[(int64_t)(start + parent) * d.target_row + x]);
          double uq = u;
          if (DRAFT) {
            const float q = as_float(draft[(int64_t)(start + parent) * d.draft_row + x]);
            sm.q[tid] = q;
            uq *= (double)q;        // exact
          }
          sm.p[tid] = p;
          sm.uq[tid] = uq;
          sm.good[tid] = uq < (double)p;
        }
      }
    }
  }
  __syncthreads();
  cluster_runs();                   // row_sum writes to the other CTAs
  if (sm.bad) {
    for (int i = tid; rank == 0 && i < n; i += kThreads) d.path[start + i] = -1;
    if (lead) put(-1, -1);
    return;
  }
  // A warp's piece of a row: `each` values from v0 on, counted from the
  // 16-byte boundary at or before the row.
  constexpr int N = Values<T>::N, STEP = 32 * N;
  const int pieces = (int)ctas * kWarps,
            each = (d.V + N - 1 + pieces * STEP - 1) / (pieces * STEP) * STEP,
            first = ((int)rank * kWarps + warp) * each;
  auto before = [&](const T *pr) {
    return (int)(reinterpret_cast<uintptr_t>(pr) % 16 / sizeof(T));
  };
  int gone = 0;                     // rejected tokens of the node, without q
  unsigned sums = 0;                // taken so far
  // the sum of what is left of node `node`'s row; kept per CTA and per warp
  auto row_sum = [&](int node, float c) {
    const T *pr = target + (int64_t)(start + node) * d.target_row;
    const T *qr = DRAFT ? draft + (int64_t)(start + node) * d.draft_row : nullptr;
    const int v0 = first - before(pr), v1 = min(d.V, v0 + each);
    const bool with_q = DRAFT && c != 0.f, wide = with_q && before(pr) == before(qr);
    unsigned long long sum = 0ull;
    if (with_q) {
      for (int o = v0; o < v1; o += 16 * STEP) {
        Halves h;
#pragma unroll 4
        for (int v = o + lane * N; v < min(v1, o + 16 * STEP); v += STEP) {
          Values<T> p, q;
          p.load(pr, v, d.V, true);
          q.load(qr, v, d.V, wide);
#pragma unroll
          for (int i = 0; i < N; ++i) h.add(left_of(p.x[i], q.x[i], c));
        }
        sum += h.units();
      }
    } else {
      for (int o = v0; o < v1; o += 16 * STEP) {
        Halves h;
#pragma unroll 4
        for (int v = o + lane * N; v < min(v1, o + 16 * STEP); v += STEP) {
          Values<T> p;
          p.load(pr, v, d.V, true);
#pragma unroll
          for (int i = 0; i < N; ++i) h.add(__saturatef(p.x[i]));
        }
        sum += h.units();
      }
    }
    if (!DRAFT)
      for (int i = lane; i < gone; i += 32) {
        const int x = sm.gone[i];
        if (x >= v0 && x < v1) sum -= units_of(as_float(pr[x]));
      }
    sum = warp_sum(sum);
    __syncthreads();                // the last sum's warps have been read
    if (lane == 0) sm.warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      const unsigned long long all = warp_sum(lane < kWarps ? sm.warp[lane] : 0ull);
      if (lane < (int)ctas) peer_store(&sm.totals[sums & 1][rank], lane, all);
    }
    cluster_sync();
    unsigned long long total = 0ull;
    for (unsigned r = 0; r < ctas; ++r) total += sm.totals[sums & 1][r];
    ++sums;
    return total;
  };

  // the walk, by every warp alike
  int at = 0, count = 1;
  float c = 0.f;
  double mass = 1.0;
  unsigned long long total = 0ull;  // of the node, once it has been summed
  bool summed = false;
  if (rank == 0)
    for (int i = tid; i < n; i += kThreads)
      if (i > 0) d.path[start + i] = -1;
  __syncthreads();
  if (lead) d.path[start] = 0;
  for (bool down = true; down;) {
    down = false;
    unsigned long long kids = (unsigned long long)__ballot_sync(kFull, sm.parent[lane] == at) |
                              (unsigned long long)__ballot_sync(kFull, sm.parent[lane + 32] == at)
                                  << 32;
    bool first_child = true;
    while (kids) {
      const int i = __ffsll((long long)kids) - 1;
      kids &= kids - 1;
      const int x = (int)sm.token[i];
      float w = sm.p[i];
      bool good, taken = false;     // taken: rejected before, as another node
      if (first_child) {
        good = sm.good[i];          // (64-bit products are slow: done for all nodes at once)
      } else if (DRAFT) {
        w = __fmaf_rn(-c, sm.q[i], w);
        good = mass > 0.0 && sm.uq[i] * mass < (double)w;
      } else {
        for (int j = lane; j < gone; j += 32) taken = taken || sm.gone[j] == x;
        taken = __any_sync(kFull, taken);
        if (taken) w = 0.f;
        good = mass > 0.0 && sm.uq[i] * mass < (double)w;
      }
      first_child = false;
      if (good) {
        if (lead) d.path[start + count] = i;
        ++count;
        at = i;
        c = 0.f;
        mass = 1.0;
        gone = 0;
        summed = false;
        down = true;
        break;
      }
      if (DRAFT) {
        if (mass > 0.0) {
          c = (float)((double)c + mass);
          total = row_sum(at, c);
          mass = (double)total / kUnit;
          summed = true;
        }
      } else if (!taken) {
        mass = fmax(mass - (double)units_of(w) / kUnit, 0.0);
        __syncthreads();            // every warp has looked for x
        if (tid == 0) sm.gone[gone] = x;
        ++gone;
        __syncthreads();
      }
    }
  }
  if (!summed) total = row_sum(at, c);
  if (total == 0ull && (c != 0.f || gone > 0)) {
    // nothing left after rounding: from the target's row itself
    c = 0.f;
    gone = 0;
    total = row_sum(at, 0.f);
  }
  // r of [0, total): the token is the first whose running sum passes it
  const float u = sm.last;
  const unsigned long long U = u > 0.f ? (unsigned long long)(fminf(u, 0.99999994f) * 2147483648.f)
                                       : 0ull;
  unsigned long long r = (__umul64hi(total, U) << 33) | ((total * U) >> 31);
  if (total == 0ull) {
    if (lead) put(-1, count);
  } else {
    for (unsigned k = 0; k < rank; ++k) {
      const unsigned long long x = sm.totals[(sums - 1) & 1][k];
      r = r < x ? ~0ull : r - x;    // in an earlier CTA's slice: in no warp's here
      if (r == ~0ull) break;
    }
    if (r < sm.totals[(sums - 1) & 1][rank]) {      // the same for all of the CTA
      int owner = 0;                // the warp whose piece it is in
      while (owner < kWarps - 1 && r >= sm.warp[owner]) r -= sm.warp[owner++];
      // All warps look at that piece, a run of its steps each: the sums of the
      // runs first, then the steps of one run.
      const T *pr = target + (int64_t)(start + at) * d.target_row;
      const T *qr = DRAFT ? draft + (int64_t)(start + at) * d.draft_row : nullptr;
      const int piece = ((int)rank * kWarps + owner) * each - before(pr),
                run = (each / STEP + kWarps - 1) / kWarps * STEP,
                v0 = piece + warp * run, v1 = min(min(d.V, piece + each), v0 + run);
      const bool with_q = DRAFT && c != 0.f, wide = with_q && before(pr) == before(qr);
      // this lane's values of the step from `base` on, in whole numbers
      unsigned long long x[N];
      auto step_of = [&](int base) {
        const int v = base + lane * N;
        Values<T> p, q;
        p.load(pr, v, d.V, true);
        if (with_q) q.load(qr, v, d.V, wide);
        unsigned long long own = 0ull;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          x[i] = units_of(with_q ? left_of(p.x[i], q.x[i], c) : p.x[i]);
          if (!DRAFT)
            for (int k = 0; k < gone; ++k)
              if (sm.gone[k] == v + i) x[i] = 0ull;
          own += x[i];
        }
        return own;
      };
      unsigned long long sum = 0ull;
      for (int base = v0; base < v1; base += STEP) sum += step_of(base);
      sum = warp_sum(sum);
      if (lane == 0) sm.run[warp] = sum;
      __syncthreads();
      int mine = 0;
      while (mine < kWarps - 1 && r >= sm.run[mine]) r -= sm.run[mine++];
      if (mine == warp)
        for (int base = v0; base < v1; base += STEP) {
          const unsigned long long own = step_of(base);
          unsigned long long inc = own;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += y;
          }
          const unsigned hit = __ballot_sync(kFull, inc > r);
          if (hit) {
            if (lane == __ffs(hit) - 1) {
              inc -= own;
              int i = 0;
              for (; i < N - 1 && inc + x[i] <= r; ++i) inc += x[i];
              put(base + lane * N + i, count);
            }
            break;
          }
          r -= __shfl_sync(kFull, inc, 31);
        }
    }
  }
  cluster_sync();                   // no CTA ends while others write to its totals
}

// CTAs of a cluster: as many as keep the SMs busy.  64 sequences of V = 131072,
// 4 CTAs of 512 threads each: 21.6 us; 2: 30.0, 8: 28.5; 4 of 1024: 31.1; 8 of 256
// the same 21.6, but 16 trees of V = 100003 then take 23.5 us, with 512 21.0.
int verify_cluster(int B, int sm_count) {
  int c = 1;
  while (c < 8 && B * c * 2 <= 2 * sm_count) c *= 2;
  return c;
}

template <typename T>
cudaError_t launch_t(const Drafts &d, int sm_count, cudaStream_t st) {
  const int c = verify_cluster(d.B, sm_count);
  cudaError_t e = d.draft ? launch_cluster(k_verify<T, true>, dim3(d.B * c), dim3(kThreads), c, 0,
                                           st, d)
                          : launch_cluster(k_verify<T, false>, dim3(d.B * c), dim3(kThreads), c,
                                           0, st, d);
  count_launch();
  return e;
}

}  // namespace

cudaError_t launch_verify(int dtype, const Drafts &d, int sm_count, cudaStream_t st) {
  return dtype == VQ_F32   ? launch_t<float>(d, sm_count, st)
         : dtype == VQ_F16 ? launch_t<__half>(d, sm_count, st)
                           : launch_t<__nv_bfloat16>(d, sm_count, st);
}

}  // namespace vqk
