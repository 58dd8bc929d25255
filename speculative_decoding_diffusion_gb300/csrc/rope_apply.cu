// rope_apply.cu -- simsd_rope: rotary positions of query and key rows.
//
// y = R(pos) x on the pairs of the first rotary_dim elements of every head:
//   y1 = x1 cos - x2 sin, y2 = x2 cos + x1 sin, the angle position * w_i.
// A copy with six operations per pair, so DRAM bounds it; the 64 angles of a
// row are formed once and shared by its heads through shared memory, while the
// heads' first vectors are already on their way (four pairs of 16 bytes a
// thread).  262144 rows of 32 + 8 heads of 128, bf16: 0.83 ms, 6.5 TB/s of its
// bytes, 0.95 of a plain copy's rate (0.91 ms with the angles in plain order,
// where the lanes that read them met in the same banks); 128 rows of 32 heads, fp32: 3.0 us.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "rope_spec.cuh"
#include "vec.cuh"

namespace simsd {

simsd_status make_rope_plan(const simsd_rope_spec &s, int hd, RopePlan *p) {
  const int rd = s.rotary_dim == 0 ? hd : s.rotary_dim;
  if (!(s.base > 1.0f) || !(s.base < INFINITY) || rd < 2 || rd > hd || rd % 2 != 0 ||
      (s.style != SIMSD_ROPE_HALF && s.style != SIMSD_ROPE_INTERLEAVED) ||
      s.scaling < SIMSD_ROPE_PLAIN || s.scaling > SIMSD_ROPE_BANDED ||
      !(s.attn_factor >= 0.0f) || !(s.attn_factor < INFINITY))
    return SIMSD_ERR_SHAPE;
  if (s.scaling != SIMSD_ROPE_PLAIN && (!(s.factor >= 1.0f) || !(s.factor < INFINITY)))
    return SIMSD_ERR_SHAPE;
  if (s.scaling == SIMSD_ROPE_NTK && rd < 4) return SIMSD_ERR_SHAPE;
  if ((s.scaling == SIMSD_ROPE_YARN || s.scaling == SIMSD_ROPE_BANDED) &&
      (s.original_len < 1 || !(s.slow > 0.0f) || !(s.fast > s.slow) || !(s.fast < INFINITY)))
    return SIMSD_ERR_SHAPE;

  static std::mutex mu;
  static bool have = false;
  static simsd_rope_spec last_spec;
  static int last_hd = 0;
  static RopePlan last;
  std::lock_guard<std::mutex> lock(mu);
  const simsd_rope_spec &l = last_spec;
  if (!have || last_hd != hd || l.base != s.base || l.rotary_dim != s.rotary_dim ||
      l.style != s.style || l.scaling != s.scaling || l.factor != s.factor ||
      l.original_len != s.original_len || l.fast != s.fast || l.slow != s.slow ||
      l.attn_factor != s.attn_factor) {
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    RopePlan r;
    memset(&r, 0, sizeof(r));
    double base = s.base;
    const double f = s.factor, n0 = s.original_len;
    if (s.scaling == SIMSD_ROPE_NTK) base *= pow(f, rd / (rd - 2.0));
    double lo = 0.0, hi = 1.0;
    if (s.scaling == SIMSD_ROPE_YARN) {
      lo = floor(rd * log(n0 / (kTwoPi * s.fast)) / (2.0 * log(base)));
      hi = ceil(rd * log(n0 / (kTwoPi * s.slow)) / (2.0 * log(base)));
      lo = lo < 0.0 ? 0.0 : lo;
      hi = hi > rd - 1 ? rd - 1 : hi;
    }
    for (int i = 0; i < rd / 2; ++i) {
      double w = pow(base, -2.0 * i / rd);
      if (s.scaling == SIMSD_ROPE_LINEAR) {
        w /= f;
      } else if (s.scaling == SIMSD_ROPE_YARN) {
        const double t = (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
        const double ramp = t < 0.0 ? 0.0 : t > 1.0 ? 1.0 : t;
        w = w * (1.0 - ramp) + w / f * ramp;
      } else if (s.scaling == SIMSD_ROPE_BANDED) {
        const double t = (n0 * w / kTwoPi - s.slow) / ((double)s.fast - s.slow);
        const double keep = t < 0.0 ? 0.0 : t > 1.0 ? 1.0 : t;
        w = w / f * (1.0 - keep) + w * keep;
      }
      r.turns[i] = w / kTwoPi;
      r.hi[i] = (float)r.turns[i];
      r.lo[i] = (float)(r.turns[i] - (double)r.hi[i]);
    }
    r.half = rd / 2;
    r.interleaved = s.style == SIMSD_ROPE_INTERLEAVED;
    r.mul = s.attn_factor > 0.0f ? s.attn_factor
            : s.scaling == SIMSD_ROPE_YARN ? (float)(0.1 * log(f) + 1.0) : 1.0f;
    last = r;
    last_spec = s;
    last_hd = hd;
    have = true;
  }
  *p = last;
  return SIMSD_OK;
}

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 4;       // rows of a CTA: one angle per thread at head_dim 128
constexpr int kBatch = 4;         // vector pairs a thread has in flight

struct RopeArgs {
  RopePlan plan;
  const int32_t *pos;
  const void *x0, *x1;
  void *y0, *y1;
  int64_t x0_row, x0_head, y0_row, y0_head, x1_row, x1_head, y1_row, y1_head;
  int rows, h0, heads, hd, rows_per_cta, inverse;
  uint32_t inv_heads;             // ceil(2^32 / heads): row of a (row, head) index
};

// One pair of 16-byte vectors of a head.  HALF: vectors v and v + half (the
// rotated pairs), past those two neighbouring untouched ones; interleaved:
// two neighbouring vectors, each holding its own pairs.
template <typename T, bool IL, bool VEC>
__global__ void __launch_bounds__(kThreads, 3)
rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int N = VEC ? 16 / (int)sizeof(T) : 1;   // elements of a vector
  __shared__ __align__(16) float2 cs_s[kMaxRows][64];  // placed by angle_at
  const int row0 = blockIdx.x * a.rows_per_cta;
  const int n_rows = min(a.rows_per_cta, a.rows - row0);
  const int half = a.plan.half;
  const int per_head = a.hd / (2 * N);               // a power of two, <= 64
  const int lane = threadIdx.x & (per_head - 1);
  const int group = threadIdx.x / per_head, n_groups = kThreads / per_head;
  const int total = n_rows * a.heads;
  // first elements of this thread's two vectors
  int d1, d2;
  bool turn1, turn2;                                 // holds rotated elements
  if (IL) {
    d1 = 2 * lane * N; d2 = d1 + N;
    turn1 = d1 < 2 * half; turn2 = d2 < 2 * half;
  } else if (lane * N < half) {
    d1 = lane * N; d2 = d1 + half; turn1 = turn2 = true;
  } else {
    d1 = 2 * lane * N; d2 = d1 + N; turn1 = turn2 = false;
  }
  Raw<T, N> u[kBatch], v[kBatch];
  // row and head of item i: where they lie in the input and the output
  auto place = [&](int i, int &r, const T *&src, T *&dst) {
    r = a.heads == 1 ? i : (int)__umulhi((uint32_t)i, a.inv_heads);
    int h = i - r * a.heads;
    const bool second = h >= a.h0;
    h -= second ? a.h0 : 0;
    src = (const T *)(second ? a.x1 : a.x0) + (int64_t)(row0 + r) * (second ? a.x1_row : a.x0_row) +
          h * (second ? a.x1_head : a.x0_head);
    dst = (T *)(second ? a.y1 : a.y0) + (int64_t)(row0 + r) * (second ? a.y1_row : a.y0_row) +
          h * (second ? a.y1_head : a.y0_head);
  };
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * n_groups;
      if (i < total) {
        int r;
        const T *src;
        T *dst;
        place(i, r, src, dst);
        u[k] = *reinterpret_cast<const Raw<T, N> *>(src + d1);
        v[k] = *reinterpret_cast<const Raw<T, N> *>(src + d2);
      }
    }
  };
  load(group);
  for (int e = threadIdx.x; e < n_rows * 64; e += kThreads) {
    const int r = e >> 6, d = e & 63;
    if (d < half) {
      float2 cs = rope_plan_cs(plan_by_lane(a.plan), d, __ldg(a.pos + row0 + r));
      if (a.inverse) cs.y = -cs.y;
      cs_s[r][angle_at(d)] = cs;
    }
  }
  __syncthreads();
  for (int i0 = group; i0 < total; i0 += kBatch * n_groups) {
    if (i0 != group) load(i0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * n_groups;
      if (i >= total) break;
      int r;
      const T *src;
      T *dst;
      place(i, r, src, dst);
      const float2 *cs = cs_s[r];
      float x[N], y[N];
      load_vec<T, N>(reinterpret_cast<const T *>(&u[k]), x);
      load_vec<T, N>(reinterpret_cast<const T *>(&v[k]), y);
      if (!IL) {
        if (turn1 && N == 1) {
          const float2 w = cs[angle_at(d1)];
          const float x1 = x[0], x2 = y[0];
          x[0] = x1 * w.x - x2 * w.y;
          y[0] = x2 * w.x + x1 * w.y;
        } else if (turn1) {
#pragma unroll
          for (int j = 0; j + 1 < N; j += 2) {
            const float4 w = *reinterpret_cast<const float4 *>(cs + angle_at(d1 + j));
            const float x1 = x[j], x2 = y[j], x3 = x[j + 1], x4 = y[j + 1];
            x[j] = x1 * w.x - x2 * w.y;
            y[j] = x2 * w.x + x1 * w.y;
            x[j + 1] = x3 * w.z - x4 * w.w;
            y[j + 1] = x4 * w.z + x3 * w.w;
          }
        }
      } else if (N == 1) {                           // the pair itself
        if (turn1) {
          const float2 w = cs[angle_at(d1 >> 1)];
          const float x1 = x[0], x2 = y[0];
          x[0] = x1 * w.x - x2 * w.y;
          y[0] = x2 * w.x + x1 * w.y;
        }
      } else {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float *z = s ? y : x;
          if (!(s ? turn2 : turn1)) continue;
#pragma unroll
          for (int j = 0; j + 3 < N; j += 4) {
            const float4 w = *reinterpret_cast<const float4 *>(cs + angle_at(((s ? d2 : d1) + j) >> 1));
            const float x1 = z[j], x2 = z[j + 1], x3 = z[j + 2], x4 = z[j + 3];
            z[j] = x1 * w.x - x2 * w.y;
            z[j + 1] = x2 * w.x + x1 * w.y;
            z[j + 2] = x3 * w.z - x4 * w.w;
            z[j + 3] = x4 * w.z + x3 * w.w;
          }
        }
      }
      store_vec<T, N>(dst + d1, x);
      store_vec<T, N>(dst + d2, y);
    }
  }
}

template <typename T>
cudaError_t launch_rope(const RopeArgs &a, bool vec, cudaStream_t stream) {
  const dim3 grid((a.rows + a.rows_per_cta - 1) / a.rows_per_cta);
  if (a.plan.interleaved) {
    if (vec) rope_kernel<T, true, true><<<grid, kThreads, 0, stream>>>(a);
    else rope_kernel<T, true, false><<<grid, kThreads, 0, stream>>>(a);
  } else {
    if (vec) rope_kernel<T, false, true><<<grid, kThreads, 0, stream>>>(a);
    else rope_kernel<T, false, false><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace simsd

using namespace simsd;

extern "C" simsd_status simsd_rope(const simsd_rope_desc *d, void *stream) {
  if (d == nullptr) return SIMSD_ERR_NULL;
  if (d->dtype != SIMSD_F32 && d->dtype != SIMSD_BF16) return SIMSD_ERR_DTYPE;
  if (d->rows < 0 || d->rows > (1 << 30) || d->num_heads0 < 1 || d->num_heads0 > 16384 ||
      d->num_heads1 < 0 || d->num_heads1 > 16384 || (d->head_dim != 64 && d->head_dim != 128) ||
      (d->inverse != 0 && d->inverse != 1))
    return SIMSD_ERR_SHAPE;
  RopeArgs a;
  const simsd_status st = make_rope_plan(d->rope, d->head_dim, &a.plan);
  if (st != SIMSD_OK) return st;
  if (d->rows == 0) return SIMSD_OK;             // (tensors without rows have no memory)
  const bool two = d->num_heads1 > 0;
  if (!d->positions || !d->x0 || !d->y0 || (two && (!d->x1 || !d->y1))) return SIMSD_ERR_NULL;
  const int es = d->dtype == SIMSD_BF16 ? 2 : 4;
  const void *p[4] = {d->x0, d->y0, two ? d->x1 : d->x0, two ? d->y1 : d->y0};
  const int64_t s[8] = {d->x0_row, d->x0_head, d->y0_row, d->y0_head,
                        two ? d->x1_row : 0, two ? d->x1_head : 0, two ? d->y1_row : 0, two ? d->y1_head : 0};
  bool vec = (a.plan.half * es) % 16 == 0;     // whole vectors on both sides of every border
  for (const void *q : p) {
    if ((uintptr_t)q % es != 0) return SIMSD_ERR_ALIGN;
    vec = vec && (uintptr_t)q % 16 == 0;
  }
  for (const int64_t t : s) vec = vec && (t * es) % 16 == 0;
  a.pos = d->positions;
  a.x0 = d->x0; a.y0 = d->y0; a.x1 = d->x1; a.y1 = d->y1;
  a.x0_row = d->x0_row; a.x0_head = d->x0_head; a.y0_row = d->y0_row; a.y0_head = d->y0_head;
  a.x1_row = d->x1_row; a.x1_head = d->x1_head; a.y1_row = d->y1_row; a.y1_head = d->y1_head;
  a.rows = d->rows;
  a.h0 = d->num_heads0;
  a.heads = d->num_heads0 + d->num_heads1;
  a.hd = d->head_dim;
  a.inverse = d->inverse;
  // as many rows a CTA (up to four: an angle per thread) as leave every SM one
  // (40 heads of 128, bf16, in CTAs of one / four rows: 152 rows 2.9 / 4.1 us, 608
  // 4.9 / 4.1, 9728 51 / 37, 65536 321 / 214)
  a.rows_per_cta = std::min(kMaxRows, std::max(1, d->rows / device_sm_count()));
  a.inv_heads = (uint32_t)(((1ull << 32) + a.heads - 1) / a.heads);
  const cudaError_t e = d->dtype == SIMSD_BF16 ? launch_rope<__nv_bfloat16>(a, vec, (cudaStream_t)stream)
                                               : launch_rope<float>(a, vec, (cudaStream_t)stream);
  return e == cudaSuccess ? SIMSD_OK : SIMSD_ERR_CUDA;
}
