// logprobs.cu -- simsd_token_logprobs: log probabilities of given tokens, their
// ranks, the entropy and the likeliest tokens of each row of logits.
//
// With c = log2(e) / T, a reference M and t_v = c (l_v - M): S = sum 2^t_v and
// W = sum t_v 2^t_v give log2 p_v = t_v - log2 S and the entropy ln 2 (log2 S -
// W / S).  The references are the parts' own maxima, exact in the logits' type,
// so l_v - M loses nothing that the exponential would show.
//
// First pass, every logit read once: a warp per part of 2048 entries, all of it
// requested at once and held in registers; it leaves M, S, W, how many entries
// are ahead of the row's token, and the maximum of each segment of 256.  The
// second pass, a CTA per row, merges the parts; the k-th largest maximum over
// any disjoint sets of segments is a bound that k entries reach, so only the
// segments whose maximum reaches it are read again (some 22 of 594 for k = 20
// and 151,936 entries) and only the entries that do are sorted.  A key of 64
// bits, the value's ordered bits over the inverted index, makes the order total.
//
// 1536 rows of 151,936 take the first pass 87 us in bf16, 5.4 TB/s (0.80 of the copy
// rate; DRAM 68%, issue slots 67%, ALU 50%: reads and arithmetic share it), in CTAs of
// 128 threads, eight an SM (ten: 2% less on many rows, 10% more on few; 256 threads,
// four: 103 us).  Both passes: 99.5 us, in fp32 152 (0.92), with nine tenths of the
// entries at -1e9 and T = 0.3 101; four rows 6.2 us, two launches and their round trips.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "vec.cuh"

namespace simsd {
namespace {

constexpr int kPart = 2048, kSeg = 256, kSegs = kPart / kSeg;
constexpr int kLane = kPart / 32;          // entries of a lane
constexpr int kPassThreads = 128;
constexpr int kMaxTop = 32;
constexpr float kMinTemperature = 1e-30f, kMaxTemperature = 1e30f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSegList = 64, kCand = 1024;  // segments and entries that reach the bound, kept aside

struct Part {
  float m, s, w;
  int ahead;
};

struct LogprobArgs {
  const void *logits;
  const int32_t *tokens;
  float *logprob, *entropy, *top_logprobs;
  int32_t *rank, *top_ids;
  Part *parts;                             // [rows][n_parts]
  float *seg_max;                          // [rows][n_parts][kSegs]
  uint32_t *status;
  int64_t stride;
  int rows, vocab, top_k, n_parts;
  float c, inv_c, inv_half_t;              // log2(e) / T and its inverse; 2 / T
};

// Entries (of T) in 16 bytes.
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

// How many entries before the row's first one its 16-byte block begins.
template <typename T>
__device__ __forceinline__ int lead_of(const T *row) {
  return (int)(((uintptr_t)row & 15u) / sizeof(T));
}

__device__ __forceinline__ uint4 load16(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// The 16 bytes that begin at entry e (an aligned address), -inf for entries
// outside 0..vocab-1.
template <typename T>
__device__ __forceinline__ uint4 load_entries(const T *row, int e, int vocab) {
  constexpr int V = kVec<T>;
  if (e >= 0 && e + V <= vocab) return load16(row + e);
  float x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = e + i >= 0 && e + i < vocab ? Elem<T>::load(row + e + i) : -INFINITY;
  if constexpr (V == 8)
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  else
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ float2 bf16_pair(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger of the two, NaN if x is.
__device__ __forceinline__ float at_least(float x, float low) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(low));
  return y;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
  return x;
}

// What a lane does with 16 bytes of entries, by type.  bf16: maxima, the lower
// bound and the counts are taken two entries at a time, as they lie.
template <typename T> struct Lane;

template <> struct Lane<float> {
  static __device__ __forceinline__ float max_of(const uint4 &v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  // the smallest value above x
  static __device__ __forceinline__ float above(float x) { return nextafterf(x, INFINITY); }
  // a value of the type that is at most x, and below y
  static __device__ __forceinline__ float below(float x, float y) { return fminf(x, nextafterf(y, -INFINITY)); }
  using Bound = float;
  static __device__ __forceinline__ Bound bound(float x) { return x; }
  static __device__ __forceinline__ float2 pair(const uint4 &v, int i, Bound least) {
    return i == 0 ? make_float2(at_least(__uint_as_float(v.x), least), at_least(__uint_as_float(v.y), least))
                  : make_float2(at_least(__uint_as_float(v.z), least), at_least(__uint_as_float(v.w), least));
  }
  // a running count of the entries of at least `least`
  struct Count {
    float least;
    int n = 0;
    __device__ explicit Count(float l) : least(l) {}
    __device__ void add(const uint4 &v) {
      n += (__uint_as_float(v.x) >= least) + (__uint_as_float(v.y) >= least) + (__uint_as_float(v.z) >= least) +
           (__uint_as_float(v.w) >= least);
    }
    __device__ int total() const { return n; }
  };
  static __device__ __forceinline__ float entry(const uint4 &v, int j) { return __uint_as_float(word_of(v, j)); }
};

template <> struct Lane<__nv_bfloat16> {
  static __device__ __forceinline__ __nv_bfloat162 two(uint32_t u) { return *reinterpret_cast<__nv_bfloat162 *>(&u); }
  static __device__ __forceinline__ uint32_t bits(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t *>(&x); }
  static __device__ __forceinline__ float max_of(const uint4 &v) {
    const float2 m = bf16_pair(bits(__hmax2(__hmax2(two(v.x), two(v.y)), __hmax2(two(v.z), two(v.w)))));
    return fmaxf(m.x, m.y);
  }
  static __device__ __forceinline__ float above(float x) {       // (x is a bf16 value)
    const uint32_t u = __float_as_uint(x + 0.f);
    return x == INFINITY ? x : u == 0u ? __uint_as_float(0x00010000u)
           : __uint_as_float((int32_t)u < 0 ? u - 0x10000u : u + 0x10000u);
  }
  static __device__ __forceinline__ float below(float x, float y) {
    const uint32_t u = __float_as_uint(x);                       // towards -inf: a negative magnitude up, a positive one down
    const float down = __uint_as_float(((int32_t)u < 0 ? u + 0xffffu : u) & 0xffff0000u);
    const uint32_t w = __float_as_uint(y + 0.f);                 // (a bf16 value)
    const float next = w == 0u ? __uint_as_float(0x80010000u) : __uint_as_float((int32_t)w < 0 ? w + 0x10000u : w - 0x10000u);
    return fminf(down, next);
  }
  using Bound = __nv_bfloat162;
  static __device__ __forceinline__ Bound bound(float x) { return __float2bfloat162_rn(x); }   // (exact)
  static __device__ __forceinline__ float2 pair(const uint4 &v, int i, Bound least) {
    return bf16_pair(bits(__hmax2_nan(two(word_of(v, i)), least)));
  }
  struct Count {                           // (exact: at most 32 in each half)
    __nv_bfloat162 least, n;
    __device__ explicit Count(float l) : least(__float2bfloat162_rn(l)), n(__float2bfloat162_rn(0.f)) {}
    __device__ void add(const uint4 &v) {
      n = __hadd2(n, __hadd2(__hadd2(__hge2(two(v.x), least), __hge2(two(v.y), least)),
                             __hadd2(__hge2(two(v.z), least), __hge2(two(v.w), least))));
    }
    __device__ int total() const {
      const float2 x = bf16_pair(bits(n));
      return (int)(x.x + x.y);
    }
  };
  static __device__ __forceinline__ float entry(const uint4 &v, int j) {
    const float2 x = bf16_pair(word_of(v, j >> 1));
    return (j & 1) ? x.y : x.x;
  }
};

template <typename T>
__global__ void __launch_bounds__(kPassThreads, sizeof(T) == 2 ? 8 : 4)
logprob_pass_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int V = kVec<T>, N = kLane / V;              // vectors of a lane
  using L = Lane<T>;
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * (kPassThreads / 32) + (threadIdx.x >> 5);
  grid_dep_wait();
  grid_dep_launch();
  const int r = (int)(item / (uint32_t)a.n_parts), part = (int)(item - (uint32_t)r * (uint32_t)a.n_parts);
  if (r >= a.rows) return;
  const int tok = a.tokens != nullptr ? __ldg(a.tokens + r) : -2;
  if (tok == -1) return;
  const T *row = (const T *)a.logits + r * a.stride;
  const int lead = lead_of(row), e0 = part * kPart - lead;
  if (e0 >= a.vocab) return;                             // (the second pass counts parts as this line does)
  uint4 v[N];
  if (e0 >= 0 && e0 + kPart <= a.vocab) {
    const T *p = row + e0 + lane * V;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = load16(p + i * 32 * V);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = load_entries<T>(row, e0 + (i * 32 + lane) * V, a.vocab);
  }
  const bool given = a.rank != nullptr && tok >= 0 && tok < a.vocab;
  const float mine = given ? Elem<T>::load(row + tok) : 0.f;
  float m = -INFINITY, sm = -INFINITY;
  float keep = -INFINITY;                                // lane i: maximum of segment i
  constexpr int PER = kSeg / (32 * V);                   // vectors of a segment
#pragma unroll
  for (int i = 0; i < N; ++i) {
    sm = fmaxf(sm, L::max_of(v[i]));
    if ((i + 1) % PER == 0) {
      sm = warp_max(sm);
      if (lane == i / PER) keep = sm;
      m = fmaxf(m, sm);
      sm = -INFINITY;
    }
  }
  const int64_t at = (int64_t)r * a.n_parts + part;
  if (a.top_k > 0 && lane < kSegs) a.seg_max[at * kSegs + lane] = keep;
  int ahead = 0;
  if (given) {
    // before the token an equal entry is ahead too, behind it only a larger one
    const float up = L::above(mine);
    if (tok < e0 || tok >= e0 + kPart) {                 // all behind it, or all before
      typename L::Count n(tok < e0 ? up : mine);
#pragma unroll
      for (int i = 0; i < N; ++i) n.add(v[i]);
      ahead = n.total();
      if (tok >= e0 + kPart && mine == -INFINITY && e0 < 0 && lane == 0) ahead += e0;   // (entries that do not exist)
    } else {
#pragma unroll
      for (int j = 0; j < kLane; ++j) {
        const int e = e0 + ((j / V) * 32 + lane) * V + j % V;
        const float x = L::entry(v[j / V], j % V);
        ahead += x > mine || (x == mine && e < tok && e >= 0) ? 1 : 0;
      }
    }
    ahead = __reduce_add_sync(0xffffffffu, ahead);
  }
  // t = c l - c m with one rounding: c m rounded is off by `shift`, the same for
  // every entry, so the sums are brought back by 2^shift.  Entries whose weight
  // is 0 all the same are raised to where t is finite (0 times it has to be 0).
  // Up to 2^24 shift is at most a half; beyond (a part at a mask's finite fill, a
  // temperature near 0) it would leave the exponential's range, and differences
  // come first.
  const float ref = m == -INFINITY ? 0.f : m, cm = ref * a.c;
  const float least = L::below(fmaxf(ref - 1000.f * a.inv_c, -3e38f), ref);
  float2 s2 = make_float2(0.f, 0.f), w2 = s2;
  float shift = 0.f;
  const float2 c2 = make_float2(a.c, a.c);
  if (fabsf(cm) <= 16777216.f && least > -INFINITY) {
    shift = -fmaf(ref, a.c, -cm);
    const float2 m2 = make_float2(-cm, -cm);
    const typename L::Bound low = L::bound(least);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 t = fma_f32x2(L::pair(v[i], j, low), c2, m2);
        const float2 p = make_float2(ex2(t.x), ex2(t.y));
        s2 = add_f32x2(s2, p);
        w2 = fma_f32x2(p, t, w2);
      }
  } else {
    const float2 m2 = make_float2(-ref, -ref);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        float2 t = mul_f32x2(add_f32x2(make_float2(L::entry(v[i], 2 * j), L::entry(v[i], 2 * j + 1)), m2), c2);
        t = make_float2(at_least(t.x, -1000.f), at_least(t.y, -1000.f));
        const float2 p = make_float2(ex2(t.x), ex2(t.y));
        s2 = add_f32x2(s2, p);
        w2 = fma_f32x2(p, t, w2);
      }
  }
  float s = warp_sum(s2.x + s2.y), w = warp_sum(w2.x + w2.y);
  const float back = ex2(shift);                         // c (l - m) = t + shift
  w = fmaf(shift, s, w) * back;
  s *= back;
  if (lane == 0) a.parts[at] = {m, s, w, ahead};
}

// ------------------------------------------------------------- order by keys
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);           // (-0 is 0)
  return u ^ ((int32_t)u < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order ^ ((int32_t)order < 0 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(float x, int i) { return (uint64_t)ordered(x) << 32 | (0xffffffffu - (uint32_t)i); }
__device__ __forceinline__ int index_of(uint64_t key) { return (int)(0xffffffffu - (uint32_t)key); }

template <typename K>
__device__ __forceinline__ K exchange(K key, int lane, int j, bool down) {
  const K other = __shfl_xor_sync(0xffffffffu, key, j);
  return (((lane & j) == 0) == down) == (key > other) ? key : other;
}

// The warp's keys, largest in lane 0 (a bitonic sorting network).
template <typename K>
__device__ __forceinline__ K sort32(K key, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) key = exchange(key, lane, j, (lane & k) == 0);
  return key;
}

// The 32 largest of two sorted lists.
template <typename K>
__device__ __forceinline__ K merge32(K a, K b, int lane) {
  const K r = __shfl_sync(0xffffffffu, b, 31 - lane);
  K key = a > r ? a : r;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) key = exchange(key, lane, j, true);
  return key;
}

// Warp 0's list: the 32 largest keys of all warps' lists, by way of at[].
template <int W, typename K>
__device__ __forceinline__ K merge_warps(K list, K (*at)[32], int warp, int lane) {
  at[warp][lane] = list;
  __syncthreads();
#pragma unroll
  for (int half = W / 2; half > 0; half >>= 1) {
    if (warp < half) {
      list = merge32(list, at[warp + half][lane], lane);
      at[warp][lane] = list;
    }
    __syncthreads();
  }
  return list;
}

// `list` with a key a lane added (0: none); only the first k of it count.
__device__ __forceinline__ uint64_t add32(uint64_t list, uint64_t key, int k, int lane) {
  const uint64_t last = __shfl_sync(0xffffffffu, list, k - 1);
  if (!__any_sync(0xffffffffu, key > last)) return list;
  return merge32(list, sort32(key, lane), lane);
}

template <typename T, int kFinishThreads>
__global__ void __launch_bounds__(kFinishThreads)
logprob_finish_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int W = kFinishThreads / 32;
  constexpr int AHEAD = 4;                               // maxima of a lane that are requested first of all
  __shared__ float red_s[3][W];
  __shared__ int ahead_s[W];
  __shared__ uint64_t list_s[W][32];
  __shared__ uint32_t top_s[W][32];
  __shared__ uint64_t cand_s[kCand];
  __shared__ int seg_s[kSegList], n_cand_s, n_list_s;
  const int r = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch();
  const int tok = a.tokens != nullptr ? __ldg(a.tokens + r) : -2;
  if (tok == -1) return;
  const T *row = (const T *)a.logits + r * a.stride;
  const int lead = lead_of(row), n_parts = (a.vocab + lead + kPart - 1) / kPart;
  const Part *parts = a.parts + (int64_t)r * a.n_parts;
  const int n_seg = (a.vocab + lead + kSeg - 1) / kSeg, k = a.top_k;
  const float *seg_max = a.seg_max + (int64_t)r * a.n_parts * kSegs;
  float first[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    const int j = threadIdx.x + i * kFinishThreads;
    first[i] = k > 0 && j < n_seg ? __ldcg(seg_max + j) : 0.f;
  }
  const bool given = tok >= 0 && tok < a.vocab;
  const float mine = given ? Elem<T>::load(row + tok) : 0.f;
  if (threadIdx.x == 0) n_cand_s = n_list_s = 0;
  // ------------------------------------------------------- the row's sums
  auto part = [&](int j) {
    const int4 v = __ldcg(reinterpret_cast<const int4 *>(parts + j));
    return Part{__int_as_float(v.x), __int_as_float(v.y), __int_as_float(v.z), v.w};
  };
  const bool any = threadIdx.x < n_parts;                // a thread's first part stays in registers
  const Part p0 = any ? part(threadIdx.x) : Part{-INFINITY, 0.f, 0.f, 0};
  float m = p0.m;
  for (int j = threadIdx.x + kFinishThreads; j < n_parts; j += kFinishThreads) m = fmaxf(m, part(j).m);
  m = warp_max(m);
  if (lane == 0) red_s[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < W; ++i) m = fmaxf(m, red_s[0][i]);
  float s = 0.f, w = 0.f;
  int ahead = 0;
  auto add = [&](const Part &p) {
    // a part that is -inf throughout has nothing but, maybe, a NaN in its sums
    const float d = p.m == -INFINITY ? 0.f : at_least((p.m - m) * a.c, -1000.f), f = ex2(d);
    s = fmaf(f, p.s, s);
    w = fmaf(f, fmaf(d, p.s, p.w), w);
    ahead += p.ahead;
  };
  if (any) add(p0);
  for (int j = threadIdx.x + kFinishThreads; j < n_parts; j += kFinishThreads) add(part(j));
  s = warp_sum(s);
  w = warp_sum(w);
  ahead = __reduce_add_sync(0xffffffffu, ahead);
  if (lane == 0) {
    red_s[1][warp] = s;
    red_s[2][warp] = w;
    ahead_s[warp] = ahead;
  }
  __syncthreads();
  s = w = 0.f;
  ahead = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    s += red_s[1][i];
    w += red_s[2][i];
    ahead += ahead_s[i];
  }
  const float log_s = m == -INFINITY ? __uint_as_float(0x7fc00000u) : log2f(s);   // NaN: nothing there
  // ln p of a logit (halves: the difference of two finite ones stays finite)
  auto log_p = [&](float x) { return (0.5f * x - 0.5f * m) * a.inv_half_t - log_s * kLn2; };
  if (threadIdx.x == 0) {
    if (a.tokens != nullptr && !given) raise_status(a.status, kStatusBadInput);
    if (a.logprob != nullptr)
      a.logprob[r] = given ? log_p(mine) : __uint_as_float(0x7fc00000u);
    if (a.rank != nullptr) a.rank[r] = given ? ahead : -1;
    if (a.entropy != nullptr) a.entropy[r] = (log_s - w / s) * kLn2;
  }
  if (a.top_k == 0) return;
  // ------------------------------------------------ a bound for the k-th entry
  // The k-th largest of the threads' maxima, each over the segments that are its
  // own: k entries at least reach it, and few more do.
  auto maximum = [&](int i) {                            // of this thread's segment i
    const int j = threadIdx.x + i * kFinishThreads;
    return i < AHEAD ? first[i] : __ldcg(seg_max + j);
  };
  const int mine_n = (n_seg - (int)threadIdx.x + kFinishThreads - 1) / kFinishThreads;   // this thread's segments
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (i < mine_n) top = fmaxf(top, first[i]);
  for (int i = AHEAD; i < mine_n; ++i) top = fmaxf(top, maximum(i));
  (void)merge_warps<W>(sort32(mine_n > 0 ? ordered(top) : 0u, lane), top_s, warp, lane);
  const uint32_t last = top_s[0][k - 1];                 // 0: fewer than k threads have a segment
  const float least = last == 0u ? -INFINITY : value_of(last);
  // ----------------------------------------------------- the entries that reach it
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (i < mine_n && first[i] >= least) {
      const int at = atomicAdd(&n_list_s, 1);
      if (at < kSegList) seg_s[at] = threadIdx.x + i * kFinishThreads;
    }
  for (int i = AHEAD; i < mine_n; ++i)
    if (maximum(i) >= least) {
      const int at = atomicAdd(&n_list_s, 1);
      if (at < kSegList) seg_s[at] = threadIdx.x + i * kFinishThreads;
    }
  __syncthreads();
  const int n_list = n_list_s;
  constexpr int V = kVec<T>;
  if (n_list <= kSegList)
    for (int i = warp; i < n_list; i += W)
#pragma unroll
      for (int q = 0; q < kSeg / (32 * V); ++q) {
        const int e = seg_s[i] * kSeg - lead + (q * 32 + lane) * V;
        const uint4 v = load_entries<T>(row, e, a.vocab);
        if (Lane<T>::max_of(v) >= least) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float x = Lane<T>::entry(v, j);
            if (x >= least && e + j >= 0 && e + j < a.vocab) {
              const int at = atomicAdd(&n_cand_s, 1);
              if (at < kCand) cand_s[at] = key_of(x, e + j);
            }
          }
        }
      }
  __syncthreads();
  uint64_t list = 0;
  if (n_list <= kSegList && n_cand_s <= kCand) {
    if (warp != 0) return;
    const int n_cand = n_cand_s;
    for (int j = 0; j < n_cand; j += 32) list = add32(list, j + lane < n_cand ? cand_s[j + lane] : 0ull, k, lane);
  } else {
    // many equal entries, or a vocabulary of few segments: each warp keeps the best
    // of its segments in order as it reads them
    for (int j = warp; j < n_seg; j += W) {
      if (!(__ldcg(seg_max + j) >= least)) continue;
#pragma unroll 1
      for (int q = 0; q < kSeg; q += 32) {
        const int e = j * kSeg - lead + q + lane;
        const float x = e >= 0 && e < a.vocab ? Elem<T>::load(row + e) : __uint_as_float(0x7fc00000u);
        list = add32(list, x >= least ? key_of(x, e) : 0ull, k, lane);
      }
    }
    list = merge_warps<W>(list, list_s, warp, lane);
    if (warp != 0) return;
  }
  if (lane < k) {
    a.top_ids[(int64_t)r * k + lane] = list == 0ull ? 0 : index_of(list);
    a.top_logprobs[(int64_t)r * k + lane] =
        list == 0ull ? __uint_as_float(0x7fc00000u) : log_p(value_of((uint32_t)(list >> 32)));
  }
}

int parts_of(int vocab) { return (vocab + kPart - 1) / kPart + 1; }

simsd_status check(const simsd_token_logprobs_desc *d) {
  if (d == nullptr) return SIMSD_ERR_NULL;
  if (d->dtype != SIMSD_F32 && d->dtype != SIMSD_BF16) return SIMSD_ERR_DTYPE;
  if (d->rows < 0 || d->rows > (1 << 20) || d->vocab < 1 || d->vocab > (1 << 21) || d->top_k < 0 ||
      d->top_k > kMaxTop || d->top_k > d->vocab || !(d->temperature == 0.0f || (d->temperature >= kMinTemperature && d->temperature <= kMaxTemperature)) ||
      d->row_stride < 0 || (d->row_stride != 0 && d->row_stride < d->vocab && d->rows > 1))
    return SIMSD_ERR_SHAPE;
  return SIMSD_OK;
}

size_t workspace_of(const simsd_token_logprobs_desc *d) {
  return align_up(kAlign + (size_t)d->rows * parts_of(d->vocab) * (sizeof(Part) + kSegs * sizeof(float)), kAlign);
}

template <typename T>
cudaError_t launch(const LogprobArgs &a, cudaStream_t stream) {
  constexpr int W = kPassThreads / 32;
  const int64_t items = (int64_t)a.rows * a.n_parts;
  const cudaError_t e = launch_pdl(logprob_pass_kernel<T>, dim3((unsigned)((items + W - 1) / W)), dim3(kPassThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  // few rows: more threads for each
  return a.rows < 2 * device_sm_count() ? launch_pdl(logprob_finish_kernel<T, 256>, dim3((unsigned)a.rows), dim3(256), 0, stream, a)
                                        : launch_pdl(logprob_finish_kernel<T, 128>, dim3((unsigned)a.rows), dim3(128), 0, stream, a);
}

}  // namespace
}  // namespace simsd

using namespace simsd;

extern "C" {

size_t simsd_token_logprobs_workspace_size(const simsd_token_logprobs_desc *d) {
  return check(d) == SIMSD_OK ? workspace_of(d) : 0;
}

simsd_status simsd_token_logprobs(const simsd_token_logprobs_desc *d, void *stream_ptr) {
  const simsd_status st = check(d);
  if (st != SIMSD_OK) return st;
  if (d->rows == 0) return SIMSD_OK;
  if (!d->logits || (!d->tokens && (d->logprob || d->rank)) || ((d->top_k > 0) != (d->top_ids != nullptr)) ||
      ((d->top_k > 0) != (d->top_logprobs != nullptr)))
    return SIMSD_ERR_NULL;
  if ((uintptr_t)d->logits % (d->dtype == SIMSD_BF16 ? 2 : 4) != 0) return SIMSD_ERR_ALIGN;
  if (d->workspace == nullptr || (uintptr_t)d->workspace % kAlign != 0 || d->workspace_bytes < workspace_of(d))
    return SIMSD_ERR_WORKSPACE;
  LogprobArgs a;
  char *ws = (char *)d->workspace;
  a.logits = d->logits; a.tokens = d->tokens;
  a.logprob = d->logprob; a.entropy = d->entropy; a.top_logprobs = d->top_logprobs;
  a.rank = d->rank; a.top_ids = d->top_ids;
  a.n_parts = parts_of(d->vocab);
  a.parts = (Part *)(ws + kAlign);
  a.seg_max = (float *)(ws + kAlign + (size_t)d->rows * a.n_parts * sizeof(Part));
  a.status = (uint32_t *)ws;
  a.stride = d->row_stride ? d->row_stride : d->vocab;
  a.rows = d->rows; a.vocab = d->vocab; a.top_k = d->top_k;
  const double T = d->temperature == 0.0f ? 1.0 : (double)d->temperature;
  a.c = (float)(1.4426950408889634 / T);
  a.inv_c = (float)(T / 1.4426950408889634);
  a.inv_half_t = (float)(2.0 / T);
  cudaStream_t stream = (cudaStream_t)stream_ptr;
  const cudaError_t e = d->dtype == SIMSD_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
  return e == cudaSuccess ? SIMSD_OK : SIMSD_ERR_CUDA;
}

}  // extern "C"
