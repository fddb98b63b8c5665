// Bookkeeping of a warp's ring of shared-memory stages: which blocks have
// copies under way to a stage, and the parity of the barrier phase that ends
// them.  Plain C++, so that it can be checked on the host.
#pragma once

#ifdef __CUDACC__
#define VQK_HD __host__ __device__ __forceinline__
#else
#define VQK_HD inline
#endif

namespace vqk {

struct StageRing {
  unsigned under_way = 0u;   // two bits a stage, one a block
  unsigned phases = 0u;      // a bit a stage

  VQK_HD unsigned blocks(int s) const { return (under_way >> (2 * s)) & 3u; }
  VQK_HD unsigned parity(int s) const { return (phases >> s) & 1u; }
  // copies of `which` blocks go to stage s, which is empty
  VQK_HD void issued(int s, unsigned which) { under_way |= which << (2 * s); }
  // a wait for stage s has ended with its copies landed (not by giving up: a
  // warp that gives up still waits for what it left under way)
  VQK_HD void landed(int s) {
    under_way &= ~(3u << (2 * s));
    phases ^= 1u << s;
  }
};

}  // namespace vqk
