// vec.cuh -- N consecutive values of a row as fp32: 16-byte vector accesses
// for N = 4 (fp32) and N = 8 (bf16; fp32 takes two), single elements for 1.
#pragma once

#include "common.cuh"

namespace simsd {

template <typename T, int N>
__device__ __forceinline__ void load_vec(const T *p, float *f) {
  if constexpr (N == 1) {
    f[0] = Elem<T>::load(p);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 v = reinterpret_cast<const float4 *>(p)[i];
      f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
    }
  } else {
    static_assert(N == 8, "one 16-byte vector of bf16");
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <typename T, int N>
__device__ __forceinline__ void store_vec(T *p, const float *f) {
  if constexpr (N == 1) {
    Elem<T>::store(p, f[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<float4 *>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else {
    static_assert(N == 8, "one 16-byte vector of bf16");
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                               pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
}

// N elements as they lie in memory, held so until they are used (bf16: half
// the registers of their fp32 values).
template <typename T, int N>
struct __align__(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Raw {
  T x[N];
};

// max(m, |a|, |b|), NaN if any is.
__device__ __forceinline__ float absmax_nan(float m, float a, float b) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(a), "f"(b));
  return d;
}

}  // namespace simsd
