// Steps that warps take together with bounded waits between them, apart from what is waited for.
#pragma once

#ifdef __CUDACC__
#define EMP_STEPS __device__ __forceinline__
#else
#define EMP_STEPS inline
#endif

namespace emp {

// Stages first, first + step, ... below n: wait(k) for the stage, read(k), a barrier among the warps that share it, write(k).
// Every warp comes to the barrier of every stage: one whose wait ran out would otherwise leave the others, whose waits
// did not, in a barrier without a limit.  From the first wait that runs out on a warp neither waits, reads nor writes.
// False if one did.
template <typename Wait, typename Read, typename Barrier, typename Write>
EMP_STEPS bool in_place_stages(int first, int step, int n, Wait wait, Read read, Barrier barrier, Write write) {
  bool ok = true;
  for (int k = first; k < n; k += step) {
    ok = ok && wait(k);
    if (ok) read(k);
    barrier();
    if (ok) write(k);
  }
  return ok;
}

}  // namespace emp
