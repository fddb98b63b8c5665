// The tensor-memory attention of the paged cache over trees of drafts
// (paged_chunk.cuh).
#include "paged_chunk.cuh"

namespace vqk {

cudaError_t launch_paged_chunk_tree(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                                    int sm_count, cudaStream_t st) {
  return t.max_new * (a.H_q / a.H_kv) <= chunk::kSmallRows
             ? launch_paged_chunk_tree_small(dtype, a, t, D, sm_count, st)
             : chunk::launch_form<true, false>(dtype, a, t, D, sm_count, st);
}

}  // namespace vqk
