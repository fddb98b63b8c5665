// The split-KV attention of the paged cache with the weights of the stored
// tokens (paged_decode.cuh).
#include "paged_decode.cuh"

namespace vqk {
namespace {

// weights[token] += sum over the rows of 2^(score + top - maximum) / sum, from
// what the attention and its merge left.  A token is one thread's, so that no
// two threads add to one place and the order of a sum is fixed.
//
// The scores are kept (4 bytes a row and token, written and read) rather than
// computed a second time: with 4 rows that is 32 bytes against the 80 of the
// key's codes at D = 128, g = 32, and no product.
// Bound: latency (offsets, lengths, then scores and weights at once), so that
// a warp takes four steps at a time, eight lanes a step, and 16 bytes a load
// (16 sequences of 8192, 8 kv heads, 4 rows: 16.5 us with a step a warp).
constexpr int kWeighWarps = 4;
constexpr int kWeighSteps = 4;
__global__ void __launch_bounds__(32 * kWeighWarps)
k_paged_weigh(PagedArgs a, PagedAttend t, const int *prefixes, const float *scores,
              const float2 *stats, PagedWeights w) {
  extern __shared__ int prefix[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = threadIdx.x; i <= a.B; i += blockDim.x) prefix[i] = prefixes[i];
  __syncthreads();
  const int lane = threadIdx.x & 31, H = a.H_kv, R = t.max_new * (a.H_q / H);
  const int units = prefix[a.B];
  for (int u = (blockIdx.x * kWeighWarps + (threadIdx.x >> 5)) * kWeighSteps + (lane >> 3);
       u < units; u += gridDim.x * kWeighWarps * kWeighSteps) {
    int b = 0, hi = a.B;
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (prefix[mid] <= u) b = mid; else hi = mid;
    }
    const int nb = (prefix[b + 1] - prefix[b]) / H, h = (u - prefix[b]) / nb,
              tok = (u - prefix[b] - h * nb) * kStep + 4 * (lane & 7);
    const Seq L = sequence_of(a, b, t.max_new);
    const int rows = L.n * (a.H_q / H);
    const float4 *x = reinterpret_cast<const float4 *>(scores + (int64_t)u * (R * kStep)) +
                      (lane & 7);
    const float2 *st = stats + (int64_t)(b * H + h) * R;
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
      const float2 f = st[r];
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

}  // namespace

size_t paged_weigh_ws(int B, int H_kv, int D, int rows, int64_t capacity, int sm_count) {
  return scores_at(B, H_kv, D, rows, sm_count) +
         (size_t)B * H_kv * ((capacity + kStep - 1) / kStep) * kStep * rows * sizeof(float);
}

cudaError_t launch_paged_weigh(int dtype, const PagedArgs &a, const PagedAttend &t,
                               const PagedWeights &w, int D, int sm_count, cudaStream_t st) {
  cudaError_t e = launch_form<kWeigh>(dtype, a, t, D, sm_count, st);
  const int64_t steps = (int64_t)a.B * a.H_kv *
                        ((((int64_t)a.max_pages << a.page_log2) + kStep - 1) / kStep);
  if (e != cudaSuccess || steps == 0) return e;
  const int rows = t.max_new * (a.H_q / a.H_kv);
  const char *ws = reinterpret_cast<const char *>(t.ws);
  const int64_t each = kWeighWarps * kWeighSteps, need = (steps + each - 1) / each,
                all = 16 * (int64_t)sm_count;
  e = launch_pdl(
      k_paged_weigh, dim3((unsigned)(need < all ? need : all)), dim3(32 * kWeighWarps),
      sizeof(int) * (a.B + 1), st, a, t,
      reinterpret_cast<const int *>(ws + prefix_at(a.B, a.H_kv, D, rows, sm_count)),
      reinterpret_cast<const float *>(ws + scores_at(a.B, a.H_kv, D, rows, sm_count)),
      reinterpret_cast<const float2 *>(ws + stats_at(a.B, a.H_kv, D, rows, sm_count)), w);
  count_launch();
  return e;
}

}  // namespace vqk
