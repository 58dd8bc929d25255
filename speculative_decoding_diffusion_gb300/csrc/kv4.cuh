// kv4.cuh -- the 4-bit cache's format: a page and head's record, e2m1 codes and
// their scales (bits 14..7 of an f16), and the rows of a call that writes or
// reads them.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace simsd {

constexpr int kScaleGroup = 16;            // elements of a scale
constexpr float kScale4Max = 10240.f;      // 6 times it still lies inside f16
constexpr uint32_t kScale4Nan = 0xfcu;     // a group that got a NaN or an infinity

// Byte offsets inside the record of 18 hd bytes.
template <int HD>
struct Record {
  static constexpr int kV = 8 * HD, kKs = 16 * HD, kVs = 17 * HD, kBytes = 18 * HD;
  // the first of a pair's 16 value bytes of elements 16 g ..
  static __host__ __device__ constexpr int v_at(int pair, int g) { return kV + (g >> 1) * 256 + pair * 32 + (g & 1) * 16; }
  static __host__ __device__ constexpr int vs_at(int pair, int g) { return kVs + pair * (HD / 8) + 2 * g; }
};

// A scale byte as f16 bits.
__device__ __forceinline__ float scale4_value(uint32_t byte) { return __half2float(__ushort_as_half((unsigned short)(byte << 7))); }

// Two scale bytes (low 16 bits) as an f16 pair; byte `b` of the two twice.
__device__ __forceinline__ uint32_t scale4_pair(uint32_t two) { return (two & 0xffu) << 7 | (two & 0xff00u) << 15; }
__device__ __forceinline__ uint32_t scale4_twice(uint32_t two, int b) { return ((two >> (8 * b)) & 0xffu) * ((1u << 7) | (1u << 23)); }

// The scale byte of a group whose largest magnitude is amax (NaN if it holds
// one): nearest to amax / 6, ties to the even byte.  The correctly rounded
// quotient lies on the same side of every middle between two scales as the
// exact one, and on it only where that does: m * 6 is exact for such a middle
// m (five bits), and amax differs from it by a step of its own or more.
__device__ __forceinline__ uint32_t scale4_of(float amax) {
  if (!(amax < INFINITY)) return kScale4Nan;
  const float q = fminf(__fdiv_rn(amax, 6.f), kScale4Max);
  const uint32_t u = __float_as_uint(q);
  const uint32_t normal = ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
  return q < 6.103515625e-5f ? (uint32_t)__float2int_rn(q * 131072.f) : normal;   // below 2^-14: steps of 2^-17
}

// Elements to codes: x / s for a scale s, correctly rounded, so that a middle
// between two codes is met exactly where x / s lies on it.  With r the
// correctly rounded 1 / s, a product and one correction by the remainder give
// that quotient (P. Markstein, Computation of elementary functions on the IBM
// RISC System/6000, 1990).
struct Scaler {
  float s, r;
};
__device__ __forceinline__ Scaler scaler_of(uint32_t byte) {
  Scaler c;
  c.s = scale4_value(byte);
  c.r = byte == 0u ? 0.f : __frcp_rn(c.s);         // no scale: codes of zero
  return c;
}
__device__ __forceinline__ float over(float x, const Scaler &c) {
  const float q = x * c.r;
  return fmaf(fmaf(-q, c.s, x), c.r, q);
}

// Two elements to a byte (nearest, ties to even, saturating), lo in the low bits.
__device__ __forceinline__ uint32_t pack_e2m1x2(float lo, float hi) {
  uint32_t w;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
      "cvt.u32.u8 %0, b;\n\t}" : "=r"(w) : "f"(lo), "f"(hi));
  return w;
}

// Eight codes as four f16 pairs, lower bits first (exact).
__device__ __forceinline__ uint4 unpack_e2m1x8(uint32_t codes) {
  uint4 h;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h.x), "=r"(h.y), "=r"(h.z), "=r"(h.w)
      : "r"(codes));
  return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// ------------------------------------------------- rows of an append or a read
constexpr int kTileRows = 16;              // rows that a CTA takes

struct Rows4 {
  const int32_t *block_table, *start, *cu_n, *take;   // take: or null
  uint32_t *status;
  int batch, max_pages, num_pages, total_n;
};

// Where a row lies: page id (-1: no row, or nothing to be done), position,
// whether it is its sequence's first row and whether the next row is the
// sequence's next token.
struct Row4 {
  int page, pos;
  bool first, more;
  // A pair of tokens that shares value bytes (positions 2 i, 2 i + 1) belongs
  // to its first row in the call.
  __device__ bool leads() const { return page >= 0 && ((pos & 1) == 0 || first); }
  __device__ bool has(int odd) const { return (pos & 1) == odd || (odd == 1 && more); }
};

// Whether a sequence's numbers are out of range; its tokens to *n.
__device__ __forceinline__ bool bad_sequence4(const Rows4 &a, int c0, int c1, int start, int b, int *n) {
  *n = 0;
  if (c0 < 0 || c1 < c0 || c1 > a.total_n || start < 0) return true;
  *n = a.take != nullptr ? __ldg(a.take + b) : c1 - c0;
  return *n < 0 || *n > c1 - c0 || (int64_t)start + *n > (int64_t)a.max_pages * kPage;
}

// The row's place, found by a whole warp together: 32 bounds of cu_n are looked
// at in each step (batch up to 32: one, up to 1024: two).  Where cu_n falls
// somewhere a row may find none.
__device__ __forceinline__ Row4 find_row4(const Rows4 &a, int row, int lane) {
  Row4 w = {-1, 0, false, false};
  if (row >= a.total_n) return w;
  int lo = 0, hi = a.batch;                // the last b in [lo, hi) with cu_n[b] <= row
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool in = at < hi && __ldg(a.cu_n + at) <= row;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    const int k = m == 0u ? 0 : 31 - __clz(m);
    lo += k * step;
    hi = min(hi, lo + step);
  }
  const int b = lo;
  const int c0 = __ldg(a.cu_n + b), c1 = __ldg(a.cu_n + b + 1), start = __ldg(a.start + b);
  int n;
  if (bad_sequence4(a, c0, c1, start, b, &n) || row < c0 || row - c0 >= n) return w;
  const int i = row - c0;
  w.pos = start + i;
  w.first = i == 0;
  w.more = i + 1 < n;
  const int page = __ldg(a.block_table + (int64_t)b * a.max_pages + w.pos / kPage);
  if (page >= 0 && page < a.num_pages) w.page = page;
  else if (lane == 0) raise_status(a.status, kStatusBadInput);
  return w;
}

// Every sequence's numbers, once in the grid.
__device__ __forceinline__ void check_rows4(const Rows4 &a) {
  for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.batch; b += gridDim.x * blockDim.x) {
    const int c0 = __ldg(a.cu_n + b), c1 = __ldg(a.cu_n + b + 1), start = __ldg(a.start + b);
    int n;
    if (bad_sequence4(a, c0, c1, start, b, &n)) raise_status(a.status, kStatusBadInput);
  }
}

}  // namespace simsd
