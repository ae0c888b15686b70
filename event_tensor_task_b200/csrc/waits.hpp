// waits.hpp — a warp's wait with a limit, kept free of CUDA so that a host
// model of the lanes can run it.
#pragma once

#ifdef __CUDACC__
#define MK_WAIT_FN __device__ __forceinline__
#else
#define MK_WAIT_FN inline
#endif

namespace mk {

// All lanes of a warp come here and leave together with one answer: true once
// every lane has seen what it waits for, false once a lane has waited longer
// than `limit`.  A poll may answer differently from lane to lane, so no lane
// acts on its own: each turn of the loop is decided by a vote of all.
template <class Warp>
MK_WAIT_FN bool wait_together(Warp& w, unsigned long long limit) {
  if (w.all(w.there())) return true;
  const unsigned long long t0 = w.now();
  for (;;) {
    if (w.all(w.there())) return true;
    if (w.any(w.now() - t0 > limit)) return false;
  }
}

}  // namespace mk
