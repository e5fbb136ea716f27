// Rings of tiles in shared memory: which phase of a slot's barrier a copy completes.
#pragma once
#if defined(__CUDACC__)
#define KFAC_HD __host__ __device__ __forceinline__
#else
#define KFAC_HD inline
#endif

namespace kfac {

// Of `issued` tiles that took `stages` slots in turn, how many took slot s.
KFAC_HD int ring_uses(int issued, int s, int stages) {
  return issued > s ? (issued - 1 - s) / stages + 1 : 0;
}
// The parity of the phase that a slot's last use completes (uses > 0).  A wait for it ends
// when that copy has landed, and not before: no later phase will begin.
KFAC_HD unsigned ring_last_parity(int uses) { return (unsigned)(uses - 1) & 1u; }

}  // namespace kfac
