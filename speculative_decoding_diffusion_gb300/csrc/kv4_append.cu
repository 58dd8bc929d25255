// kv4_append.cu -- simsd_kv4_append: rotated keys and values quantised into the
// 4-bit cache.
//
// Every token has scales of its own (one for 16 neighbouring elements), so no
// token's codes depend on another's and a row is written where it arrives.  A
// CTA takes 16 rows: their places and angles are made once for all heads, then
// a thread takes 32 elements of a key (two groups, partners of each other in
// the rotation where the pairs allow it, so that each element is read once and
// nothing is exchanged) or one group of a value.  A value byte holds two
// neighbouring tokens of an element: the thread of the pair's first token in
// the call takes both; where only one of them is written, it puts its four bits
// into the byte that is there (no other thread of the call touches it).
//
// 576,000 tokens of 8 heads of 128 in bf16: 637 us, 4.7 TB/s (0.71 of the copy rate;
// 739 without the prefetch into L2, 665 with tiles of 32 rows).  No unit is full (issue
// slots 67%, ALU 52%, DRAM 55%): the arithmetic of the scales and quotients and
// stores of 8 bytes into records beside the reads; fp32 rows, which have half as much
// of both a byte, take 485 us for 289,000 tokens (0.83).
// 64 x 8 tokens: 4.9 us, a chain of round trips (range, page, rows).
#include <limits.h>
#include <math.h>

#include "kv4.cuh"
#include "rope_spec.cuh"
#include "vec.cuh"

namespace simsd {
namespace {

constexpr int kThreads = 256;

struct Append4Args {
  RopePlan plan;
  Rows4 rows;
  const void *k, *v;
  uint8_t *cache;
  int64_t k_row, v_row;
  int Hkv;
  FastDiv by_kv;
};

// Sixteen elements, as pairs.
struct Pairs {
  float2 p[8];
};

template <typename T>
__device__ __forceinline__ Pairs load16(const T *row) {
  Pairs x;
  load_vec<T, 8>(row, reinterpret_cast<float *>(x.p));
  load_vec<T, 8>(row + 8, reinterpret_cast<float *>(x.p) + 8);
  return x;
}

__device__ __forceinline__ uint32_t scale_of(const Pairs &x) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = absmax_nan(amax, x.p[i].x, x.p[i].y);
  return scale4_of(amax);
}

// Sixteen elements to codes, two neighbours a byte.
__device__ __forceinline__ uint2 codes_of(const Pairs &x, uint32_t byte) {
  const Reciprocal r = scaler_of(byte);
  return make_uint2(pack_e2m1x8(over(x.p[0], r), over(x.p[1], r), over(x.p[2], r), over(x.p[3], r)),
                    pack_e2m1x8(over(x.p[4], r), over(x.p[5], r), over(x.p[6], r), over(x.p[7], r)));
}

// Where pair d's cosine (and, kPlane floats on, its sine) lies in a row of the
// fast path's angles: lanes read 16 pairs each, 80 bytes apart.
__device__ __forceinline__ int plane_at(int d) { return d + 4 * (d >> 4); }
template <int HD> constexpr int kPlane = HD / 2 + HD / 8;

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 4)
kv4_append_kernel(const __grid_constant__ Append4Args a) {
  using R = Record<HD>;
  __shared__ __align__(16) float angle_s[kTileRows][2 * kPlane<HD>];
  __shared__ Row4 row_s[kTileRows];
  __shared__ int lead_s[kTileRows], n_lead_s;        // rows that write their value pair
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = a.rows.tile, row0 = blockIdx.x * tile;
  grid_dep_wait();
  grid_dep_launch();
  // the rows are on their way to L2 while their places are looked up
  {
    const int lines = a.Hkv * HD * (int)sizeof(T) / 128, n = min(tile, a.rows.total_n - row0);
    for (int e = threadIdx.x; e < n * lines; e += kThreads) {
      const int r = e / lines, at = e % lines * 128;
      prefetch_l2((const char *)((const T *)a.k + (int64_t)(row0 + r) * a.k_row) + at);
      prefetch_l2((const char *)((const T *)a.v + (int64_t)(row0 + r) * a.v_row) + at);
    }
  }
  find_rows4<kThreads / 32>(a.rows, row0, warp, lane, row_s);
  check_rows4(a.rows);
  __syncthreads();
  if (warp == 0) {
    const bool leads = lane < tile && row_s[lane].leads();
    const uint32_t m = __ballot_sync(0xffffffffu, leads);
    if (leads) lead_s[__popc(m & ((1u << lane) - 1u))] = lane;
    if (lane == 0) n_lead_s = __popc(m);
  }
  // half pairs in whole groups: cosines and sines apart; else as rotate8 takes them
  const bool paired = !a.plan.interleaved && a.plan.half % 16 == 0;
  for (int e = threadIdx.x; e < tile * (HD / 2); e += kThreads) {
    const int r = e / (HD / 2), d = e % (HD / 2);
    if (row_s[r].page < 0) continue;
    const float2 cs = d < a.plan.half ? rope_plan_cs(plan_by_lane(a.plan), d, row_s[r].pos) : make_float2(1.f, 0.f);
    if (paired) {
      angle_s[r][plane_at(d)] = cs.x;
      angle_s[r][kPlane<HD> + plane_at(d)] = cs.y;
    } else {
      reinterpret_cast<float2 *>(angle_s[r])[angle_at(d)] = cs;
    }
  }
  __syncthreads();
  constexpr int KL = HD / 32, VL = HD / 16;          // threads of a key row, of a value row
  const int turned = a.plan.half / 16;               // pairs of groups that are each other's partners
  for (int e = threadIdx.x; e < tile * a.Hkv * KL; e += kThreads) {
    const int u = e % KL, rh = e / KL, r = div_by(rh, a.by_kv), h = rh - r * a.Hkv;
    const Row4 w = row_s[r];
    if (w.page < 0) continue;
    const T *src = (const T *)a.k + (int64_t)(row0 + r) * a.k_row + h * HD;
    const bool rot = paired && u < turned;
    const int g0 = rot ? u : paired ? 2 * turned + 2 * (u - turned) : 2 * u, g1 = rot ? u + turned : g0 + 1;
    Pairs x, y;
    if (paired) {
      x = load16(src + g0 * 16);
      y = load16(src + g1 * 16);
      if (rot) {
        const float *cs = angle_s[r] + plane_at(g0 * 16);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float4 c = *reinterpret_cast<const float4 *>(cs + 2 * i);
          const float4 s = *reinterpret_cast<const float4 *>(cs + kPlane<HD> + 2 * i);
          const float2 c2[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
          const float2 s2[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 p = x.p[i + k], q = y.p[i + k], ns = make_float2(-s2[k].x, -s2[k].y);
            x.p[i + k] = fma_f32x2(p, c2[k], mul_f32x2(q, ns));
            y.p[i + k] = fma_f32x2(q, c2[k], mul_f32x2(p, s2[k]));
          }
        }
      }
    } else {
      const float2 *cs = reinterpret_cast<const float2 *>(angle_s[r]);
#pragma unroll
      for (int c = 0; c < 16; c += 8) {
        rotate8(a.plan, cs, src, g0 * 16 + c, reinterpret_cast<float *>(x.p) + c);
        rotate8(a.plan, cs, src, g1 * 16 + c, reinterpret_cast<float *>(y.p) + c);
      }
    }
    uint8_t *rec = a.cache + ((int64_t)w.page * a.Hkv + h) * R::kBytes;
    const int slot = w.pos & (kPage - 1);
    const uint32_t b0 = scale_of(x), b1 = scale_of(y);
    const uint2 c0 = codes_of(x, b0), c1 = codes_of(y, b1);
    *reinterpret_cast<uint2 *>(rec + slot * (HD / 2) + g0 * 8) = c0;
    *reinterpret_cast<uint2 *>(rec + slot * (HD / 2) + g1 * 8) = c1;
    rec[R::kKs + slot * (HD / 16) + g0] = (uint8_t)b0;
    rec[R::kKs + slot * (HD / 16) + g1] = (uint8_t)b1;
  }
  const int n_lead = n_lead_s;
  for (int e = threadIdx.x; e < n_lead * a.Hkv * VL; e += kThreads) {
    const int g = e % VL, rh = e / VL, i = div_by(rh, a.by_kv), h = rh - i * a.Hkv, r = lead_s[i];
    const Row4 w = row_s[r];
    const bool even = w.has(0), odd = w.has(1);
    const T *src = (const T *)a.v + (int64_t)(row0 + r) * a.v_row + h * HD + g * 16;
    const T *src_odd = (w.pos & 1) ? src : src + a.v_row;
    Pairs x, y;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.p[i] = y.p[i] = make_float2(0.f, 0.f);
    if (even) x = load16(src);
    if (odd) y = load16(src_odd);
    uint8_t *rec = a.cache + ((int64_t)w.page * a.Hkv + h) * R::kBytes;
    const int pair = (w.pos & (kPage - 1)) >> 1;
    uint32_t *codes = reinterpret_cast<uint32_t *>(rec + R::v_at(pair, g));
    uint8_t *scales = rec + R::vs_at(pair, g);
    const uint32_t bx = scale_of(x), by = scale_of(y);
    const Reciprocal rx = scaler_of(bx), ry = scaler_of(by);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = over(x.p[2 * i], rx), u2 = over(x.p[2 * i + 1], rx);
      const float2 v = over(y.p[2 * i], ry), v2 = over(y.p[2 * i + 1], ry);
      c[i] = pack_e2m1x8(make_float2(u.x, v.x), make_float2(u.y, v.y), make_float2(u2.x, v2.x), make_float2(u2.y, v2.y));
    }
    if (even && odd) {
      *reinterpret_cast<uint4 *>(codes) = make_uint4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<uint16_t *>(scales) = (uint16_t)(bx | by << 8);
    } else {                                         // the other token's four bits stay
      const uint32_t keep = even ? 0xf0f0f0f0u : 0x0f0f0f0fu;
#pragma unroll
      for (int i = 0; i < 4; ++i) codes[i] = (codes[i] & keep) | (c[i] & ~keep);
      scales[even ? 0 : 1] = (uint8_t)(even ? bx : by);
    }
  }
}

template <typename T>
cudaError_t launch_append4(const Append4Args &a, int hd, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.rows.total_n + a.rows.tile - 1) / a.rows.tile)), block(kThreads);
  return hd == 128 ? launch_pdl(kv4_append_kernel<T, 128>, grid, block, 0, stream, a)
                   : launch_pdl(kv4_append_kernel<T, 64>, grid, block, 0, stream, a);
}

}  // namespace
}  // namespace simsd

using namespace simsd;

extern "C" simsd_status simsd_kv4_append(const simsd_kv4_append_desc *d, void *stream_ptr) {
  if (d == nullptr) return SIMSD_ERR_NULL;
  if (d->dtype != SIMSD_F32 && d->dtype != SIMSD_BF16) return SIMSD_ERR_DTYPE;
  if (d->batch < 1 || d->batch > (1 << 20) || d->num_kv_heads < 1 || d->num_kv_heads > 1024 ||
      (d->head_dim != 64 && d->head_dim != 128) || d->page_size != kPageTokens || d->num_pages < 1 ||
      d->max_pages_per_seq < 1 || d->max_pages_per_seq > (1 << 26) || d->total_n < 0 || d->total_n > (1 << 30) || d->k_row < 0 || d->v_row < 0)
    return SIMSD_ERR_SHAPE;
  Append4Args a;
  const simsd_status st = make_rope_plan(d->rope, d->head_dim, &a.plan);
  if (st != SIMSD_OK) return st;
  if ((d->total_n > 0 && (!d->k || !d->v)) || !d->start || !d->cu_n || !d->cache || !d->block_table)
    return SIMSD_ERR_NULL;
  const int es = d->dtype == SIMSD_BF16 ? 2 : 4;
  a.k_row = d->k_row ? d->k_row : (int64_t)d->num_kv_heads * d->head_dim;
  a.v_row = d->v_row ? d->v_row : (int64_t)d->num_kv_heads * d->head_dim;
  if (!aligned16(d->k) || !aligned16(d->v) || !aligned16(d->cache) || a.k_row * es % 16 != 0 || a.v_row * es % 16 != 0)
    return SIMSD_ERR_ALIGN;
  if (d->workspace == nullptr || (uintptr_t)d->workspace % kAlign != 0 || d->workspace_bytes < kAlign)
    return SIMSD_ERR_WORKSPACE;
  if (d->total_n == 0) return SIMSD_OK;
  a.rows = {d->block_table, d->start, d->cu_n, d->take, (uint32_t *)d->workspace,
            d->batch, d->max_pages_per_seq, d->num_pages, d->total_n, tile_rows4(d->total_n)};
  a.k = d->k;
  a.v = d->v;
  a.cache = (uint8_t *)d->cache;
  a.Hkv = d->num_kv_heads;
  a.by_kv = make_fast_div(a.Hkv);
  cudaStream_t stream = (cudaStream_t)stream_ptr;
  const cudaError_t e = d->dtype == SIMSD_BF16 ? launch_append4<__nv_bfloat16>(a, d->head_dim, stream)
                                               : launch_append4<float>(a, d->head_dim, stream);
  return e == cudaSuccess ? SIMSD_OK : SIMSD_ERR_CUDA;
}
