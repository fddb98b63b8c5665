// The tensor-memory attention of the paged cache over trees of drafts
// (paged_chunk.cuh).
#include "paged_chunk.cuh"

namespace vqk {

// Up to 64 rows the form for few rows is the faster one at both head sizes.
// Replayed graphs, 8 kv heads, that form against the other, us:
//                            20 rows        32 rows        64 rows
//   16 x 4096-8192, D = 128  77.9 / 93.8    81.8 / 96.8    80.4 / 101
//   1 x 32768, D = 128       38.2 / 45.3    41.5 / 48.5    44.4 / 51.0
//   16 x 4096-8192, D = 64   61.3 / 77.9    65.1 / 82.8    62.4 / 78.9
//   1 x 32768, D = 64        29.9 / 35.4    30.8 / 35.7    33.1 / 37.6
cudaError_t launch_paged_chunk_tree(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                                    int sm_count, cudaStream_t st) {
  return t.max_new * (a.H_q / a.H_kv) <= chunk::kSmallRows
             ? launch_paged_chunk_tree_small(dtype, a, t, D, sm_count, st)
             : chunk::launch_form<true, false>(dtype, a, t, D, sm_count, st);
}

}  // namespace vqk
