// steps_done.h -- which waits for a step's products a data warp of the packed state kernel still has to
// make.  Two barriers, one for even and one for odd steps, tell that step n's products are done, each by
// the parity of its phase.  Step n + 2 completes the next phase of step n's barrier, and may do so as
// soon as every data warp has arrived for it: a warp that waits for step n only then finds a parity that
// does not come back before step n + 4, which needs this warp.  So a warp waits for a step once, before it
// arrives for the step two behind it, and afterwards knows.  Products are done in the order of their steps.
#pragma once

#if defined(__CUDACC__)
#define RETNET_ON_BOTH __host__ __device__ __forceinline__
#else
#define RETNET_ON_BOTH inline
#endif

namespace retnet {

struct StepsDone {
  int known = 0;  // the products of steps 0 .. known - 1 are done
  RETNET_ON_BOTH bool must_wait(int n) const { return n >= known; }
  RETNET_ON_BOTH void waited(int n) { known = n + 1; }
};

}  // namespace retnet
