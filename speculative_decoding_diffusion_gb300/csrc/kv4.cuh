// kv4.cuh -- the 4-bit cache's format: a page and head's record, e2m1 codes and
// their scales (bits 14..7 of an f16), and the rows of a call that writes or
// reads them.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "kvq.cuh"
#include "vec.cuh"

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

// x / s, correctly rounded, from 1 / s in two parts: hi the rounded reciprocal,
// lo its remainder, x / s = x hi + x lo to 2^-47, rounded once.
struct Reciprocal {
  float hi, lo;
};
__device__ __forceinline__ Reciprocal reciprocal_of(float s) {
  Reciprocal r;
  r.hi = __frcp_rn(s);
  r.lo = fmaf(-r.hi, s, 1.f) * r.hi;
  return r;
}
__device__ __forceinline__ float2 over(float2 x, const Reciprocal &r) {
  return fma_f32x2(x, make_float2(r.hi, r.hi), mul_f32x2(x, make_float2(r.lo, r.lo)));
}

// The scale byte of a group whose largest magnitude is amax (NaN if it holds
// one): nearest to amax / 6, ties to the even byte.  The correctly rounded
// quotient lies on the same side of every middle between two scales as the
// exact one, and on it only where that does: m * 6 is exact for such a middle
// m (five bits), and amax differs from it by a step of its own or more.  The
// same holds for codes below: a middle between two codes times a scale has
// seven bits.
__device__ __forceinline__ uint32_t scale4_of(float amax) {
  // 1 / 6 in two parts
  const float q = fminf(fmaf(amax, 0x1.555556p-3f, amax * -0x1.555556p-28f), kScale4Max);
  const uint32_t u = __float_as_uint(q);
  const uint32_t normal = ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
  const uint32_t low = (uint32_t)__float2int_rn(q * 131072.f);   // below 2^-14: steps of 2^-17
  return !(amax < INFINITY) ? kScale4Nan : q < 6.103515625e-5f ? low : normal;
}

// The factor from elements to codes; no scale: codes of zero.
__device__ __forceinline__ Reciprocal scaler_of(uint32_t byte) {
  const Reciprocal r = reciprocal_of(scale4_value(byte == 0u ? 0x78u : byte));
  return byte == 0u ? Reciprocal{0.f, 0.f} : r;
}

// Eight elements to codes (nearest, ties to even, saturating), the first one in
// the low bits.
__device__ __forceinline__ uint32_t pack_e2m1x8(float2 a, float2 b, float2 c, float2 d) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
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

// ------------------------------------------ new tokens' values in the attention
// A new token's values are held as f16 relative to 2^ve, at most 65280 of it, and
// its weight p = 2^(t + ve - M) multiplies them, M a reference over t + ve.  Its
// share of the sum of weights, 2^(t - M), must not be taken from p: beside a token
// of much larger values p is 0 where the share is not.  So the sum has an
// exponential of its own, 2^(t - M + kShareLift), whose lift is taken back once a
// block: t - M is at most kNewLift + 64 (ve >= -64) and, for the row's largest t, at
// least kNewLift - 112.  M starts kNewLift below a row's largest t + ve, as far as
// f16 weights go, so that the prompt's weights, relative to the same M, fall below
// fp32's range only from 2^(112 - kNewLift - 126) = 2^-29 of the row's largest on.
constexpr float kNewLift = 15.f, kShareLift = 32.f;
constexpr float kShareUnlift = 1.f / 4294967296.f;       // 2^-kShareLift
// 2^x, its subnormal results too (the square of the root's; for merges, whose
// references lie as far apart): two instructions more than the approximation's, exp2f
// takes 256 x 256..8192 keys from 539 to 541 us.
__device__ __forceinline__ float ex2_low(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(0.5f * x));
  return y * y;
}
__device__ __forceinline__ int value_exponent(float amax) { return scale_exponent(amax, -57, 119) - 7; }

// ------------------------------------------------- rows of an append or a read
constexpr int kTileRows = 16;              // most rows that a CTA takes

struct Rows4 {
  const int32_t *block_table, *start, *cu_n, *take;   // take: or null
  uint32_t *status;
  int batch, max_pages, num_pages, total_n;
  int tile;                                // rows of a CTA: 16, or fewer where that leaves SMs without any
};

// 16 rows a CTA, halved while there would be fewer CTAs than SMs.
inline int tile_rows4(int total_n) {
  int t = kTileRows;
  while (t > 1 && (total_n + t - 1) / t < device_sm_count()) t /= 2;
  return t;
}

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

// Whether a sequence's numbers are out of range; *n: its take, replaced by its
// tokens where there is no such array.
__device__ __forceinline__ bool bad_sequence4(const Rows4 &a, int c0, int c1, int start, int *n) {
  if (c0 < 0 || c1 < c0 || c1 > a.total_n || start < 0) return true;
  if (a.take == nullptr) *n = c1 - c0;
  return *n < 0 || *n > c1 - c0 || (int64_t)start + *n > (int64_t)a.max_pages * kPage;
}

// The places of rows row0 + warp and row0 + warp + kWarps, found by the whole warp
// for both at once: 32 bounds of cu_n are looked at in each step (batch up to
// 32: one, up to 1024: two).  Where cu_n falls somewhere a row may find none.
template <int kWarps>
__device__ __forceinline__ void find_rows4(const Rows4 &a, int row0, int warp, int lane, Row4 *out) {
  constexpr int N = kTileRows / kWarps;
  int lo[N], hi[N];                        // the last b in [lo, hi) with cu_n[b] <= row
#pragma unroll
  for (int i = 0; i < N; ++i) {
    lo[i] = 0;
    hi[i] = a.batch;
  }
  for (int span = a.batch; span > 1; span = (span + 31) / 32) {
    const int step = (span + 31) / 32;
    uint32_t m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = lo[i] + lane * step;
      m[i] = __ballot_sync(0xffffffffu, at < hi[i] && __ldg(a.cu_n + at) <= row0 + warp + i * kWarps);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      lo[i] += (m[i] == 0u ? 0 : 31 - __clz(m[i])) * step;
      hi[i] = min(hi[i], lo[i] + step);
    }
  }
  int c0[N], c1[N], start[N], n[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    c0[i] = __ldg(a.cu_n + lo[i]);
    c1[i] = __ldg(a.cu_n + lo[i] + 1);
    start[i] = __ldg(a.start + lo[i]);
    n[i] = a.take != nullptr ? __ldg(a.take + lo[i]) : -1;
  }
  int page[N];
  bool any[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = row0 + warp + i * kWarps;
    any[i] = row < a.total_n && !bad_sequence4(a, c0[i], c1[i], start[i], &n[i]) && row >= c0[i] && row - c0[i] < n[i];
    page[i] = any[i] ? __ldg(a.block_table + (int64_t)lo[i] * a.max_pages + (start[i] + row - c0[i]) / kPage) : -1;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = warp + i * kWarps, k = row0 + r - c0[i];
    Row4 w = {-1, 0, false, false};
    if (any[i]) {
      w.pos = start[i] + k;
      w.first = k == 0;
      w.more = k + 1 < n[i];
      if (page[i] >= 0 && page[i] < a.num_pages) w.page = page[i];
      else if (lane == 0 && r < a.tile) raise_status(a.status, kStatusBadInput);
    }
    if (lane == 0) out[r] = w;
  }
}

// Every sequence's numbers, once in the grid.
__device__ __forceinline__ void check_rows4(const Rows4 &a) {
  for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.batch; b += gridDim.x * blockDim.x) {
    const int c0 = __ldg(a.cu_n + b), c1 = __ldg(a.cu_n + b + 1), start = __ldg(a.start + b);
    int n = a.take != nullptr ? __ldg(a.take + b) : 0;
    if (bad_sequence4(a, c0, c1, start, &n)) raise_status(a.status, kStatusBadInput);
  }
}

}  // namespace simsd
