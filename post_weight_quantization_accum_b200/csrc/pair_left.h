// What the two producers of a CTA pair left under way: plain C++, so that it
// can be checked on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define GPTQ_HD __host__ __device__
#else
#define GPTQ_HD
#endif

namespace gptq {

// Two producers fill a ring of `stages`, use u in stage u % stages, each with
// half of a use's bytes; both count them on the even one's barrier of the stage,
// which the even one arms for the two halves.  They have stopped after `even`
// and `odd` uses.  Where both went to the end the counts are equal; after a wait
// that ran out they may differ, by no more than the ring holds.
//   uses [first, most)  the last of each stage, may still be under way
//   uses [both, most)   issued by one of them alone (all in [first, most)): the
//                       barrier lacks the odd one's half (even > odd) or was
//                       never armed (odd > even)
struct PairLeft {
  uint32_t first, both, most;
};
inline GPTQ_HD PairLeft pair_left(uint32_t even, uint32_t odd, uint32_t stages) {
  const uint32_t most = even > odd ? even : odd;
  return {most > stages ? most - stages : 0u, even > odd ? odd : even, most};
}

}  // namespace gptq
