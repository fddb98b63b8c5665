// The split-KV attention of the paged cache over trees of drafts
// (paged_decode.cuh).
#include "paged_decode.cuh"

namespace vqk {

cudaError_t launch_paged_decode_tree(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                                     int sm_count, cudaStream_t st) {
  return launch_form<kTree>(dtype, a, t, nullptr, D, sm_count, st);
}

}  // namespace vqk
