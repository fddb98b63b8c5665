// The split-KV attention of the paged cache with the weights of the stored
// tokens (paged_decode.cuh).
#include "paged_decode.cuh"

namespace vqk {

size_t paged_weigh_ws(int B, int H_kv, int D, int rows, int64_t capacity, int sm_count) {
  return scores_at(B, H_kv, D, rows, sm_count) +
         (size_t)B * H_kv * ((capacity + kStep - 1) / kStep) * kStep * rows * sizeof(float);
}

cudaError_t launch_paged_weigh(int dtype, const PagedArgs &a, const PagedAttend &t,
                               const PagedWeights &w, int D, int sm_count, cudaStream_t st) {
  return launch_form<kWeigh>(dtype, a, t, &w, D, sm_count, st);
}

}  // namespace vqk
