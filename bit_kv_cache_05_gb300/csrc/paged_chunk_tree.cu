// The tensor-memory attention of the paged cache over trees of drafts
// (paged_chunk.cuh).
#include "paged_chunk.cuh"

namespace vqk {

// Up to 64 rows the form for few rows is the faster one at both head sizes.
// Replayed graphs, 8 kv heads, that form against the other, us:
//                            20 rows        32 rows        64 rows
//   16 x 4096-8192, D = 128  73.1 / 93.8    76.8 / 96.8    77.8 / 101
//   1 x 32768, D = 128       37.6 / 45.3    40.7 / 48.5    44.2 / 51.0
//   16 x 4096-8192, D = 64   62.4 / 77.9    64.9 / 82.8    61.8 / 78.9
//   1 x 32768, D = 64        30.2 / 35.4    31.1 / 35.7    32.8 / 37.6
cudaError_t launch_paged_chunk_tree(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                                    int sm_count, cudaStream_t st) {
  return t.max_new * (a.H_q / a.H_kv) <= chunk::kSmallRows
             ? launch_paged_chunk_tree_small(dtype, a, t, D, sm_count, st)
             : chunk::launch_form<true, false>(dtype, a, t, D, sm_count, st);
}

}  // namespace vqk
