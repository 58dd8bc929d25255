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
// are ahead of the row's token, and the maximum of each segment of 256.  The k
// likeliest tokens lie in the k segments with the largest maxima (equal ones: the
// first), since each of those has an entry ahead of any entry elsewhere.  So the
// second pass, a CTA per row, merges the parts, picks k segments, reads them
// again (k / 594 of a row of 151,936) and sorts the entries that reach the k-th
// maximum.  A key of 64 bits, the value's ordered bits over the inverted index,
// makes the order total.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace simsd {
namespace {

constexpr int kPart = 2048, kSeg = 256, kSegs = kPart / kSeg;
constexpr int kLane = kPart / 32;          // entries of a lane
constexpr int kPassThreads = 256, kFinishThreads = 256;
constexpr int kMaxTop = 32;
constexpr int kCand = 1024;                // entries that reach the k-th maximum, kept aside

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
  float c, inv_c;                          // log2(e) / T; ln 2
};

// Entries (of T) in 16 bytes.
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

// How many entries before the row's first one its 16-byte block begins.
template <typename T>
__device__ __forceinline__ int lead_of(const T *row) {
  return (int)(((uintptr_t)row & 15u) / sizeof(T));
}

// The vector that begins at entry e (its address is 16-byte aligned), -inf for
// entries outside 0..vocab-1.
template <typename T>
__device__ __forceinline__ void load_entries(const T *row, int e, int vocab, float *x) {
  constexpr int V = kVec<T>;
  if (e >= 0 && e + V <= vocab) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(row + e));
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (V == 8) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      } else {
        x[i] = __uint_as_float(u[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = e + i >= 0 && e + i < vocab ? Elem<T>::load(row + e + i) : -INFINITY;
  }
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

template <typename T>
__global__ void __launch_bounds__(kPassThreads)
logprob_pass_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int V = kVec<T>, N = kLane / V;              // vectors of a lane
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kPassThreads / 32) + (threadIdx.x >> 5);
  grid_dep_wait();
  grid_dep_launch();
  const int r = (int)(item / a.n_parts), part = (int)(item - (int64_t)r * a.n_parts);
  if (r >= a.rows) return;
  const int tok = a.tokens != nullptr ? __ldg(a.tokens + r) : -2;
  if (tok == -1) return;
  const T *row = (const T *)a.logits + r * a.stride;
  const int lead = lead_of(row), e0 = part * kPart - lead;
  float x[kLane];
#pragma unroll
  for (int i = 0; i < N; ++i) load_entries<T>(row, e0 + (i * 32 + lane) * V, a.vocab, x + i * V);
  const bool given = a.rank != nullptr && tok >= 0 && tok < a.vocab;
  const float mine = given ? Elem<T>::load(row + tok) : 0.f;
  float m = -INFINITY, sm = -INFINITY;
  float keep = -INFINITY;                                // lane i: maximum of segment i
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int j = 0; j < V; ++j) sm = fmaxf(sm, x[i * V + j]);
    constexpr int PER = kSeg / (32 * V);                 // vectors of a segment
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
    const float up = nextafterf(mine, INFINITY);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = e0 + (i * 32 + lane) * V;
      const float least = e + V <= tok ? mine : up;
#pragma unroll
      for (int j = 0; j < V; ++j) ahead += x[i * V + j] >= least ? 1 : 0;
      if (e <= tok && tok < e + V) {
#pragma unroll
        for (int j = 0; j < V; ++j) ahead += e + j < tok && e + j >= 0 && x[i * V + j] == mine ? 1 : 0;
      } else if (e < 0 && e + V <= tok && mine == -INFINITY) {
        ahead += e;                                      // (entries that do not exist)
      }
    }
    ahead = __reduce_add_sync(0xffffffffu, ahead);
  }
  const float ref = m == -INFINITY ? 0.f : m;
  float s0 = 0.f, s1 = 0.f, w0 = 0.f, w1 = 0.f;
#pragma unroll
  for (int i = 0; i < kLane; i += 2) {
    // (below -1000 the weight is 0, and 0 times it has to be 0)
    const float t0 = at_least((x[i] - ref) * a.c, -1000.f), t1 = at_least((x[i + 1] - ref) * a.c, -1000.f);
    const float p0 = ex2(t0), p1 = ex2(t1);
    s0 += p0;
    s1 += p1;
    w0 = fmaf(p0, t0, w0);
    w1 = fmaf(p1, t1, w1);
  }
  const float s = warp_sum(s0 + s1), w = warp_sum(w0 + w1);
  if (lane == 0) a.parts[at] = {m, s, w, ahead};
}

// ------------------------------------------------------------- order by keys
__device__ __forceinline__ uint64_t key_of(float x, int i) {
  const uint32_t u = __float_as_uint(x + 0.f);           // (-0 is 0)
  return (uint64_t)(u ^ ((int32_t)u < 0 ? 0xffffffffu : 0x80000000u)) << 32 | (0xffffffffu - (uint32_t)i);
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float(u ^ ((int32_t)u < 0 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ int index_of(uint64_t key) { return (int)(0xffffffffu - (uint32_t)key); }

__device__ __forceinline__ uint64_t exchange(uint64_t key, int lane, int j, bool down) {
  const uint64_t other = __shfl_xor_sync(0xffffffffu, key, j);
  return (((lane & j) == 0) == down) == (key > other) ? key : other;
}

// The warp's keys, largest in lane 0 (a bitonic sorting network).
__device__ __forceinline__ uint64_t sort32(uint64_t key, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) key = exchange(key, lane, j, (lane & k) == 0);
  return key;
}

// The 32 largest of two sorted lists.
__device__ __forceinline__ uint64_t merge32(uint64_t a, uint64_t b, int lane) {
  const uint64_t r = __shfl_sync(0xffffffffu, b, 31 - lane);
  uint64_t key = a > r ? a : r;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) key = exchange(key, lane, j, true);
  return key;
}

// `list` with a key a lane added (0: none); only the first k of it count.
__device__ __forceinline__ uint64_t add32(uint64_t list, uint64_t key, int k, int lane) {
  const uint64_t last = __shfl_sync(0xffffffffu, list, k - 1);
  if (!__any_sync(0xffffffffu, key > last)) return list;
  return merge32(list, sort32(key, lane), lane);
}

template <typename T>
__global__ void __launch_bounds__(kFinishThreads)
logprob_finish_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int W = kFinishThreads / 32;
  __shared__ float red_s[3][W];
  __shared__ int ahead_s[W];
  __shared__ uint64_t list_s[W][32];
  __shared__ uint64_t cand_s[kCand];
  __shared__ int n_cand_s;
  const int r = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch();
  const int tok = a.tokens != nullptr ? __ldg(a.tokens + r) : -2;
  if (tok == -1) return;
  const T *row = (const T *)a.logits + r * a.stride;
  const int lead = lead_of(row), n_parts = (a.vocab + lead + kPart - 1) / kPart;
  const Part *parts = a.parts + (int64_t)r * a.n_parts;
  const bool given = tok >= 0 && tok < a.vocab;
  const float mine = given ? Elem<T>::load(row + tok) : 0.f;
  if (threadIdx.x == 0) n_cand_s = 0;
  // ------------------------------------------------------- the row's sums
  constexpr int PER = (((1 << 21) / kPart + 1) + kFinishThreads - 1) / kFinishThreads;
  Part p[PER];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = threadIdx.x + i * kFinishThreads;
    p[i] = {-INFINITY, 0.f, 0.f, 0};
    if (j < n_parts) {
      const int4 v = __ldcg(reinterpret_cast<const int4 *>(parts + j));
      p[i] = {__int_as_float(v.x), __int_as_float(v.y), __int_as_float(v.z), v.w};
    }
    m = fmaxf(m, p[i].m);
  }
  m = warp_max(m);
  if (lane == 0) red_s[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < W; ++i) m = fmaxf(m, red_s[0][i]);
  float s = 0.f, w = 0.f;
  int ahead = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (threadIdx.x + i * kFinishThreads < n_parts) {
      // a part that is -inf throughout has nothing but, maybe, a NaN in its sums
      const float d = p[i].m == -INFINITY ? 0.f : at_least((p[i].m - m) * a.c, -1000.f), k = ex2(d);
      s = fmaf(k, p[i].s, s);
      w = fmaf(k, fmaf(d, p[i].s, p[i].w), w);
      ahead += p[i].ahead;
    }
  }
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
  if (threadIdx.x == 0) {
    if (a.tokens != nullptr && !given) raise_status(a.status, kStatusBadInput);
    if (a.logprob != nullptr)
      a.logprob[r] = given ? ((mine - m) * a.c - log_s) * a.inv_c : __uint_as_float(0x7fc00000u);
    if (a.rank != nullptr) a.rank[r] = given ? ahead : -1;
    if (a.entropy != nullptr) a.entropy[r] = (log_s - w / s) * a.inv_c;
  }
  if (a.top_k == 0) return;
  // --------------------------------------------- the k segments that matter
  const int n_seg = (a.vocab + lead + kSeg - 1) / kSeg, k = a.top_k;
  const float *seg_max = a.seg_max + (int64_t)r * a.n_parts * kSegs;
  uint64_t list = 0;
  for (int j0 = warp * 32; j0 < n_seg; j0 += kFinishThreads) {
    const int j = j0 + lane;
    list = add32(list, j < n_seg ? key_of(__ldcg(seg_max + j), j) : 0ull, k, lane);
  }
  list_s[warp][lane] = list;
  __syncthreads();
#pragma unroll 1
  for (int half = W / 2; half > 0; half >>= 1) {
    if (warp < half) {
      list = merge32(list, list_s[warp + half][lane], lane);
      list_s[warp][lane] = list;
    }
    __syncthreads();
  }
  const uint64_t last = list_s[0][k - 1];                // 0: fewer than k segments
  const float least = last == 0ull ? -INFINITY : value_of(last);
  // ---------------------------------------- their entries that reach the k-th
  auto entry = [&](int i, int j) { return index_of(list_s[0][i]) * kSeg - lead + j; };   // entry j of segment i
#pragma unroll 1
  for (int i = warp; i < k; i += W) {
    if (list_s[0][i] == 0ull) break;
    float x[kSeg / 32];
#pragma unroll
    for (int j = 0; j < kSeg / 32; ++j) {
      const int e = entry(i, j * 32 + lane);
      x[j] = e >= 0 && e < a.vocab ? Elem<T>::load(row + e) : __uint_as_float(0x7fc00000u);
    }
#pragma unroll
    for (int j = 0; j < kSeg / 32; ++j) {
      const bool in = x[j] >= least;
      const uint32_t mask = __ballot_sync(0xffffffffu, in);
      if (mask == 0u) continue;
      int at = 0;
      if (lane == 0) at = atomicAdd(&n_cand_s, __popc(mask));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(mask & ((1u << lane) - 1u));
      if (in && at < kCand) cand_s[at] = key_of(x[j], entry(i, j * 32 + lane));
    }
  }
  __syncthreads();
  if (warp != 0) return;
  const int n_cand = n_cand_s;
  list = 0;
  if (n_cand <= kCand) {
    for (int j = 0; j < n_cand; j += 32) list = add32(list, j + lane < n_cand ? cand_s[j + lane] : 0ull, k, lane);
  } else {                                               // (many equal ones: read once more, one warp in turn)
#pragma unroll 1
    for (int i = 0; i < k && list_s[0][i] != 0ull; ++i)
#pragma unroll 1
      for (int j = 0; j < kSeg; j += 32) {
        const int e = entry(i, j + lane);
        const float x = e >= 0 && e < a.vocab ? Elem<T>::load(row + e) : __uint_as_float(0x7fc00000u);
        list = add32(list, x >= least ? key_of(x, e) : 0ull, k, lane);
      }
  }
  if (lane < k) {
    a.top_ids[(int64_t)r * k + lane] = list == 0ull ? 0 : index_of(list);
    a.top_logprobs[(int64_t)r * k + lane] =
        list == 0ull ? __uint_as_float(0x7fc00000u) : ((value_of(list) - m) * a.c - log_s) * a.inv_c;
  }
}

int parts_of(int vocab) { return (vocab + kPart - 1) / kPart + 1; }

simsd_status check(const simsd_token_logprobs_desc *d) {
  if (d == nullptr) return SIMSD_ERR_NULL;
  if (d->dtype != SIMSD_F32 && d->dtype != SIMSD_BF16) return SIMSD_ERR_DTYPE;
  if (d->rows < 0 || d->rows > (1 << 20) || d->vocab < 1 || d->vocab > (1 << 21) || d->top_k < 0 ||
      d->top_k > kMaxTop || d->top_k > d->vocab || !(d->temperature >= 0.0f) || !(d->temperature < INFINITY) ||
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
  return launch_pdl(logprob_finish_kernel<T>, dim3((unsigned)a.rows), dim3(kFinishThreads), 0, stream, a);
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
  a.inv_c = 0.6931471805599453f;
  cudaStream_t stream = (cudaStream_t)stream_ptr;
  const cudaError_t e = d->dtype == SIMSD_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
  return e == cudaSuccess ? SIMSD_OK : SIMSD_ERR_CUDA;
}

}  // extern "C"
