// The end of a cluster after a wait that ran out (without one the MMA issuers have waited for every copy).  A stage's full barrier may count bytes that several CTAs ask for, while only its
// own CTA announces them (one arrival that expects all the bytes of a fill).  The CTAs may have asked for different numbers
// of fills: an announced fill lacks the bytes of a CTA that stopped earlier, and a CTA that went
// further has copies under way that nobody announced.  Before a CTA exits, every copy into shared memory of the cluster has
// to have landed, so the CTAs tell each other how many fills they asked for, and what each barrier's count lacks is
// made up for, after which its phase ends with the last copy that is under way.  A fill is asked for only when the same
// stage's last one has been consumed everywhere, so only the last STAGES fills are in question, and counts differ by no more.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define XT_HD __host__ __device__ __forceinline__
#else
#define XT_HD inline
#endif

namespace xt {
namespace gemm {

struct DrainStep {
  uint32_t complete;  // bytes to count as landed: announced for CTAs that never asked for them
  uint32_t expect;    // bytes to announce: asked for by other CTAs, not announced by this one
  bool wait;          // copies of this fill may be under way
};

// What CTA `self` does for fill number `fill` (from 0) on its own barrier: issued[c] fills were asked for by CTA c, each
// bringing bytes[c] to this barrier (bytes[self] > 0).
template <int CL>
XT_HD DrainStep drain_step(int fill, const int (&issued)[CL], int self, const uint32_t (&bytes)[CL]) {
  uint32_t want = 0, have = 0;
  bool announced = false;
#ifdef __CUDACC__
#pragma unroll
#endif
  for (int c = 0; c < CL; ++c) {
    want += bytes[c];
    if (issued[c] > fill) {
      have += bytes[c];
      announced = announced || c == self;
    }
  }
  return {announced ? want - have : 0u, announced ? 0u : have, have > 0};
}

}  // namespace gemm
}  // namespace xt
