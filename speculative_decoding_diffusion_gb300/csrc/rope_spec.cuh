// rope_spec.cuh -- rotary positions of simsd_rope_spec: the plan made on the
// host (frequencies in fp64, scaled for long contexts) and the (cos, sin) of
// a pair on the device.
#pragma once

#include "internal.h"
#include "rope.cuh"

namespace simsd {

// What the kernels take: the scaled frequencies of the first `half` pairs.
struct RopePlan {
  RopeTable tab;
  float mul;          // factor on cos and sin
  int half;           // rotated pairs, rotary_dim / 2
  int interleaved;    // pairs (2i, 2i+1) instead of (i, i + half)
};

// SIMSD_OK, or SIMSD_ERR_SHAPE for numbers outside the header's ranges.  The
// last plan is kept and copied while calls repeat the same numbers.
simsd_status make_rope_plan(const simsd_rope_spec &s, int hd, RopePlan *p);

// The same plan (a kernel parameter) read through global memory: a warp whose
// lanes index a parameter differently reads it one lane after another.
__device__ __forceinline__ const RopePlan &plan_by_lane(const RopePlan &p) {
  const RopePlan *q = &p;
  asm("" : "+l"(q));
  return *q;
}

// (cos, sin) times the plan's factor of pair d < half at position pos
// (negative positions turn the other way).
__device__ __forceinline__ float2 rope_plan_cs(const RopePlan &p, int d, int pos) {
  const float2 cs = rope_cs(p.tab, d, pos < 0 ? -pos : pos);
  return make_float2(cs.x * p.mul, (pos < 0 ? -cs.y : cs.y) * p.mul);
}

}  // namespace simsd
