// The split-KV attention of the paged cache, causal (paged_decode.cuh).
#include "paged_decode.cuh"

namespace vqk {

size_t paged_decode_ws(int B, int H_kv, int D, int rows, int sm_count) {
  return scores_at(B, H_kv, D, rows, sm_count);
}

cudaError_t launch_paged_decode(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                                int sm_count, cudaStream_t st) {
  return launch_form<kCausal>(dtype, a, t, nullptr, D, sm_count, st);
}

}  // namespace vqk
