// rope_spec.cuh -- rotary positions of simsd_rope_spec: the plan made on the
// host (turns per position in fp64, scaled for long contexts) and the (cos,
// sin) of a pair on the device.
//
// The angle is kept in turns, t = pos * w / (2 pi): the integer part drops
// out exactly, and sincospif of twice the rest needs no reduction of its own.
// With w / (2 pi) = hi + lo in two floats and the product's rounding error
// recovered by an fma, the angle is off by ~2e-7 rad for |pos| < 2^24;
// farther positions take fp64 (in a function of its own, so that no path
// that does not need it issues fp64 instructions: if-converted they took a
// fifth of the append's time).
#pragma once

#include "internal.h"
#include "vec.cuh"

namespace simsd {

// What the kernels take: the first `half` pairs' turns per position.
struct RopePlan {
  double turns[64];
  float hi[64], lo[64];
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

// The part of a turn left at a far position.
static __device__ __noinline__ float far_turn(double turns, int pos) {
  const double t = (double)pos * turns;
  return (float)(t - rint(t));
}

// (cos, sin) of pair d < half at position pos (negative positions turn the
// other way); hi, lo: the plan's for d.
__device__ __forceinline__ float2 rope_angle(const RopePlan &p, float hi, float lo, int d, int pos) {
  float rest;
  if (pos < (1 << 24) && pos > -(1 << 24)) {
    const float x = (float)pos;                      // exact
    const float t = x * hi;
    const float t_lo = fmaf(x, lo, fmaf(x, hi, -t));
    rest = (t - rintf(t)) + t_lo;
  } else {
    rest = far_turn(p.turns[d], pos);
  }
  float s, c;
  sincospif(2.f * rest, &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ float2 rope_plan_angle(const RopePlan &p, int d, int pos) {
  return rope_angle(p, p.hi[d], p.lo[d], d, pos);
}

// Place of pair d in a shared-memory row of angles that lanes read eight
// pairs at a time: 16-byte units exchanged so that eight lanes, 64 bytes
// apart, meet different banks.
__device__ __forceinline__ int angle_at(int d) { return ((((d >> 1) ^ ((d >> 4) & 3)) << 1) | (d & 1)); }

// Pairs d0 .. d0 + 7 (d0 a multiple of 8) of such a row.
__device__ __forceinline__ void load_angles8(const float2 *row, int d0, float2 *w) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float4 x = *reinterpret_cast<const float4 *>(row + angle_at(d0 + i));
    w[i] = make_float2(x.x, x.y);
    w[i + 1] = make_float2(x.z, x.w);
  }
}

// The same times the plan's factor.
__device__ __forceinline__ float2 rope_plan_cs(const RopePlan &p, int d, int pos) {
  const float2 cs = rope_plan_angle(p, d, pos);
  return make_float2(cs.x * p.mul, cs.y * p.mul);
}

// Elements e0 .. e0 + 7 (e0 a multiple of 8) of a head's row, rotated by the
// angles cs (placed by angle_at, identity pairs past the rotated part).
template <typename T>
__device__ __forceinline__ void rotate8(const RopePlan &p, const float2 *cs, const T *row, int e0, float *x) {
  load_vec<T, 8>(row + e0, x);
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 z = *reinterpret_cast<const float4 *>(cs + angle_at((e0 + i) >> 1));
      const float a0 = x[i], b0 = x[i + 1], a1 = x[i + 2], b1 = x[i + 3];
      x[i] = a0 * z.x - b0 * z.y;
      x[i + 1] = b0 * z.x + a0 * z.y;
      x[i + 2] = a1 * z.z - b1 * z.w;
      x[i + 3] = b1 * z.z + a1 * z.w;
    }
  } else if (p.half % 8 == 0) {
    if (e0 >= 2 * p.half) return;
    const bool low = e0 < p.half;
    float y[8];
    float2 z[8];
    load_vec<T, 8>(row + (low ? e0 + p.half : e0 - p.half), y);
    load_angles8(cs, low ? e0 : e0 - p.half, z);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * z[i].x + (low ? -y[i] : y[i]) * z[i].y;
  } else {                                   // partners off the chunk grid
#pragma unroll 1
    for (int i = 0; i < 8 && e0 + i < 2 * p.half; ++i) {
      const int d = e0 + i;
      const bool low = d < p.half;
      const float u = Elem<T>::load(row + d), y = Elem<T>::load(row + (low ? d + p.half : d - p.half));
      const float2 z = cs[angle_at(low ? d : d - p.half)];
      const float v = u * z.x + (low ? -y : y) * z.y;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = k == i ? v : x[k];   // no indexed registers
    }
  }
}

// Sixteen elements of a row, rotated: its chunks (of eight) c0, in x[0..7], and
// c1, in x[8..15], which i = 0.. (a sixteenth of the row) selects.  Where
// partners lie on the chunk grid the two are each other's, so a pair and its
// angle are read once.
template <typename T>
__device__ __forceinline__ void rotate16(const RopePlan &p, const float2 *cs, const T *row, int i, int &c0, int &c1,
                                         float *x) {
  if (!p.interleaved && p.half % 8 == 0 && i < p.half / 8) {
    c0 = i;
    c1 = i + p.half / 8;
    float2 z[8];
    load_vec<T, 8>(row + c0 * 8, x);
    load_vec<T, 8>(row + c1 * 8, x + 8);
    load_angles8(cs, c0 * 8, z);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = x[e], v = x[e + 8];
      x[e] = u * z[e].x - v * z[e].y;
      x[e + 8] = v * z[e].x + u * z[e].y;
    }
  } else {
    c0 = 2 * i;
    c1 = 2 * i + 1;
    rotate8(p, cs, row, c0 * 8, x);
    rotate8(p, cs, row, c1 * 8, x + 8);
  }
}

}  // namespace simsd
