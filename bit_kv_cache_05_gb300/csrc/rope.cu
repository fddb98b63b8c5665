// Norm and rotation of query and key heads in one pass (vq_kivi_norm_rope).
//
//   y = R(position) (x * rsqrt(mean x^2 + eps) * weight)     per token and head
//
// in fp32, rounded once to the rows' type.  A row is read once and written
// once; the norm, the angles (see rope.cuh) and the rotation happen in the
// lanes that hold it, so HBM bounds the kernel for prompts and the launch for
// single tokens.  A warp serves one token: 32 / LPR rows at a time, the
// angles worked out once per warp.  With few tokens a token's rows are dealt
// out to several warps (`parts`), so that a decode step spreads over the SMs.
#include <type_traits>

#include "paged.cuh"
#include "rope.cuh"
#include "vqk_internal.cuh"

namespace vqk {
namespace {

constexpr int kThreads = 128;

template <typename T, int LPR>
__global__ void __launch_bounds__(kThreads)
k_norm_rope(HeadRows q, HeadRows k, RopeArgs r, int D, int64_t tokens, float eps, int parts) {
  constexpr int RPW = 32 / LPR, NV = sizeof(T) == 4 ? 2 : 1;
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = w / parts;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (t >= tokens) return;
  const int gq = (q.heads + RPW - 1) / RPW, gk = (k.heads + RPW - 1) / RPW;
  const bool active = 16 * l < D;
  int p0, p1;
  chunk_places(r, l, p0, p1);

  auto fetch = [&](int gi, uint4 (&a)[NV], uint4 (&b)[NV]) {
    const bool isk = gi >= gq;
    const HeadRows &h = isk ? k : q;
    const int row = (isk ? gi - gq : gi) * RPW + sub;
    if (gi < gq + gk && active && row < h.heads) {
      const T *x = static_cast<const T *>(h.x) + t * h.x_token + row * h.x_head;
      load8<T>(x + p0, a);
      load8<T>(x + p1, b);
    }
  };
  uint4 na[NV] = {}, nb[NV] = {};
  int gi = (int)(w % parts);
  fetch(gi, na, nb);

  float c[8], s[8];
  rope_angles<LPR>(r, [&](int ax) -> long long {
    const int64_t i = (int64_t)ax * r.pos_stride + t;
    return r.pos64 ? static_cast<const long long *>(r.pos)[i]
                   : (long long)static_cast<const int *>(r.pos)[i];
  }, lane, c, s);

  float w0[8], w1[8];
  const void *held = nullptr;
  for (; gi < gq + gk; gi += parts) {
    const bool isk = gi >= gq;
    const HeadRows &h = isk ? k : q;
    const int row = (isk ? gi - gq : gi) * RPW + sub;
    float x0[8], x1[8];
    unpack8<T>(na, x0);
    unpack8<T>(nb, x1);
    fetch(gi + parts, na, nb);
    if (h.weight) {
      if (held != h.weight) {
        held = h.weight;
        uint4 a[NV] = {}, b[NV] = {};
        if (active) {
          load8<T>(static_cast<const T *>(h.weight) + p0, a);
          load8<T>(static_cast<const T *>(h.weight) + p1, b);
        }
        unpack8<T>(a, w0);
        unpack8<T>(b, w1);
      }
      norm_row<T, LPR>(x0, x1, w0, w1, D, eps);
    }
    if (8 * l < r.half) rotate_row(r.interleaved, c, s, x0, x1);
    if (active && row < h.heads) {
      T *y = static_cast<T *>(h.out) + t * h.out_token + row * h.out_head;
      store8<T>(y + p0, x0);
      store8<T>(y + p1, x1);
    }
  }
}

template <typename T, int LPR>
cudaError_t launch(const HeadRows &q, const HeadRows &k, const RopeArgs &r, int D,
                   int64_t tokens, float eps, int sm_count, cudaStream_t st) {
  constexpr int RPW = 32 / LPR;
  const int groups = (q.heads + RPW - 1) / RPW + (k.heads + RPW - 1) / RPW;
  // warps for about 16 per SM, at most one row group each
  int64_t parts = (int64_t)sm_count * 16 / (tokens > 0 ? tokens : 1);
  parts = parts < 1 ? 1 : (parts > groups ? groups : parts);
  const int64_t warps = tokens * parts, wpc = kThreads / 32;
  cudaError_t e = launch_pdl(k_norm_rope<T, LPR>, dim3((unsigned)((warps + wpc - 1) / wpc)),
                             dim3(kThreads), 0, st, q, k, r, D, tokens, eps, (int)parts);
  count_launch();
  return e;
}

template <typename T>
cudaError_t launch_t(const HeadRows &q, const HeadRows &k, const RopeArgs &r, int D,
                     int64_t tokens, float eps, int sm_count, cudaStream_t st) {
  if (D <= 64) return launch<T, 4>(q, k, r, D, tokens, eps, sm_count, st);
  if (D <= 128) return launch<T, 8>(q, k, r, D, tokens, eps, sm_count, st);
  return launch<T, 16>(q, k, r, D, tokens, eps, sm_count, st);
}

}  // namespace

cudaError_t launch_norm_rope(int dtype, const HeadRows &q, const HeadRows &k,
                             const RopeArgs &r, int D, int64_t tokens, float eps,
                             int sm_count, cudaStream_t st) {
  switch (dtype) {
    case VQ_F16: return launch_t<__half>(q, k, r, D, tokens, eps, sm_count, st);
    case VQ_BF16: return launch_t<__nv_bfloat16>(q, k, r, D, tokens, eps, sm_count, st);
    default: return launch_t<float>(q, k, r, D, tokens, eps, sm_count, st);
  }
}

}  // namespace vqk
