// The tensor-memory attention of the paged cache, causal (paged_chunk.cuh).
#include "paged_chunk.cuh"

namespace vqk {

size_t paged_chunk_ws(int B, int, int D, int sm_count) {
  return (chunk::part_floats(D, sm_count) + chunk::swap_floats(D, sm_count)) * sizeof(float) +
         sm_count * sizeof(chunk::CutPair) +
         (size_t)sm_count * (B + 1) * sizeof(long long);
}

cudaError_t launch_paged_chunk(int dtype, const PagedArgs &a, const PagedAttend &t, int D,
                               int sm_count, cudaStream_t st) {
  return chunk::launch_form<false, false>(dtype, a, t, D, sm_count, st);
}

}  // namespace vqk
