// Causal attention of any number of new tokens over the paged 4-bit cache
// (vq_kivi_paged_attend): one warp per (new token, query head), lanes over
// channels, one key at a time, an online softmax in fp32.
#include "paged.cuh"
#include "vqk_internal.cuh"

namespace vqk {
namespace {

constexpr int kThreads = 128;
constexpr unsigned kFull = 0xffffffffu;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
k_paged_chunk(PagedArgs a, PagedAttend t) {
  constexpr int CPL = D / 32, I = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t i = w / a.H_q;
  const int hq = (int)(w % a.H_q), h = hq / (a.H_q / a.H_kv);
  if (i >= a.tokens) return;
  const Place at = find_place(a, i);
  if (at.b < 0) return;
  float q[CPL], o[CPL], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < CPL; ++e) {
    q[e] = (float)static_cast<const T *>(t.q)[i * t.q_token + hq * t.q_head + 32 * e + lane];
    o[e] = 0.f;
  }
  const uint8_t *blk = nullptr;
  for (int p = 0; p <= at.pos; ++p) {
    const int tl = p & 15;
    if (tl == 0) blk = find_block(a, at.b, p, h, paged_block_bytes(D, a.g));
    if (!blk) continue;
    float kv[2][CPL];
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
      const int c = 32 * e + lane;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int off = v ? off_vc(D, a.g) + 2 * (tl & 1) + (c % 4) / 2 +
                                4 * (((8 * (tl >> 3) + c % 32 / 4) * 4 + (tl & 7) / 2) * I + c / 32)
                          : tl * (D / 2) + 4 * (c % 32 / 8 * I + c / 32) + c % 8 / 2;
        const int code = (blk[off] >> (4 * (c & 1))) & 15;
        const __half *mt = reinterpret_cast<const __half *>(
                               blk + (v ? off_vm(D, a.g) : off_km(D))) +
                           ((tl >> 1) * (D / a.g) + c / a.g) * 4 + (tl & 1);
        kv[v][e] = __half2float(__hfma(__int2half_rn(code), mt[0], mt[2]));
      }
    }
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < CPL; ++e) x = fmaf(q[e], kv[0][e], x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(kFull, x, d);
    x *= t.scale;
    const float mn = fmaxf(m, x);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float y = exp2f(x - (mn == -INFINITY ? 0.f : mn));
    m = mn;
    l = l * f + y;
#pragma unroll
    for (int e = 0; e < CPL; ++e) o[e] = o[e] * f + y * kv[1][e];
  }
#pragma unroll
  for (int e = 0; e < CPL; ++e) {
    const float y = l == 0.f ? 0.f : o[e] / l;
    static_cast<T *>(t.out)[(i * a.H_q + hq) * D + 32 * e + lane] = (T)y;
  }
}

template <typename T>
cudaError_t launch_t(const PagedArgs &a, const PagedAttend &t, int D, cudaStream_t st) {
  const int64_t warps = a.tokens * a.H_q, wpc = kThreads / 32;
  const dim3 grid((unsigned)((warps + wpc - 1) / wpc));
  cudaError_t e = D == 64 ? launch_pdl(k_paged_chunk<T, 64>, grid, dim3(kThreads), 0, st, a, t)
                          : launch_pdl(k_paged_chunk<T, 128>, grid, dim3(kThreads), 0, st, a, t);
  count_launch();
  return e;
}

}  // namespace

size_t paged_chunk_ws(int, int, int, int) { return 0; }

cudaError_t launch_paged_chunk(int dtype, const PagedArgs &a, const PagedAttend &t, int D, int,
                               cudaStream_t st) {
  return dtype == VQ_F16 ? launch_t<__half>(a, t, D, st) : launch_t<__nv_bfloat16>(a, t, D, st);
}

}  // namespace vqk
