// pkv_join.h -- how the CTAs of a cluster join what each has summed.  Plain C++, so that the
// rule can be run on the host too.
#pragma once

#ifdef __CUDACC__
#define PKV_JOIN __device__ __forceinline__
#else
#define PKV_JOIN inline
#endif

namespace pkv {

// The parts part(0) .. part(share - 1) added in rank order.  False where any rank gave up on a
// wait: its part, and so the total, lacks some of its terms.
template <typename Part, typename GaveUp>
PKV_JOIN bool join_ranks(int share, Part part, GaveUp gave_up, float& total) {
  bool whole = true;
  total = 0.f;
  for (int k = 0; k < share; ++k) {
    whole = whole && !gave_up(k);
    total += part(k);
  }
  return whole;
}

}  // namespace pkv
