// The tensor-memory attention of the paged cache over trees of drafts of at most
// 64 rows of a kv head (paged_chunk.cuh).
#include "paged_chunk.cuh"

namespace vqk {

cudaError_t launch_paged_chunk_tree_small(int dtype, const PagedArgs &a, const PagedAttend &t,
                                          int D, int sm_count, cudaStream_t st) {
  return chunk::launch_form<true, true>(dtype, a, t, D, sm_count, st);
}

}  // namespace vqk
