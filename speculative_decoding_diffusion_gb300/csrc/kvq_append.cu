// kvq_append.cu -- simsd_kvq_append: rotated keys and values into the e4m3
// paged cache.
//
// A page and head's scale is 2^E, E = min{e : amax <= 448 * 2^e}; a value x
// is stored as the e4m3 code nearest to x * 2^-E.  Scaling by a power of two
// keeps the mantissa, so a page that later holds larger tokens moves its
// older codes exactly (up to the subnormal codes) instead of reading the
// tokens again.
//
// One CTA per touched page, a warp per head: a lane holds eight-element
// chunks of the page's 16 rows, the maximum is a warp reduction, and the
// rotation's partners are exchanged between lanes.  Bytes in, half as many
// (bf16) out: DRAM bounds a prompt's append.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "kvq.cuh"
#include "rope_spec.cuh"
#include "vec.cuh"

namespace simsd {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 8;                 // elements a lane handles together

struct AppendArgs {
  RopePlan plan;
  const void *k, *v;
  uint8_t *k_cache, *v_cache, *k_scale, *v_scale;
  const int32_t *block_table, *start, *cu_n, *take;
  uint32_t *status;
  int64_t k_row, v_row;
  int batch, Hkv, max_pages, num_pages, total_n;
};

// Work items: a sequence's touched pages, at most ceil((n + 15) / 16) <=
// floor(n / 16) + 2 of them, numbered from first_item(b); items in the gaps
// do nothing.
__host__ __device__ __forceinline__ int64_t first_item(int32_t cu, int b) { return cu / kPage + 2LL * b; }

// Rotates one chunk (elements 8 ch .. 8 ch + 7 of a head) whose row has the
// angles cs; every lane of the warp calls it (the partners of half pairs are
// shuffled in where they are whole chunks).  Rows that are not new (have
// false) hold zeros and no angles.
template <typename T, int HD>
__device__ __forceinline__ void rotate_chunk(const RopePlan &p, const float2 *cs, const T *row,
                                             bool have, int ch, int lane, float *x) {
  const int e0 = ch * kChunk, rd = 2 * p.half;
  if (p.interleaved) {
#pragma unroll
    for (int j = 0; j < kChunk; j += 2) {
      if (have && e0 + j < rd) {
        const float2 w = cs[(e0 + j) >> 1];
        const float a = x[j], b = x[j + 1];
        x[j] = a * w.x - b * w.y;
        x[j + 1] = b * w.x + a * w.y;
      }
    }
  } else if (p.half % kChunk == 0) {
    const int step = p.half / kChunk;     // chunks between partners
    const bool turned = e0 < rd, low = e0 < p.half;
    const int src = lane + (turned ? (low ? step : -step) : 0);
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const float y = __shfl_sync(0xffffffffu, x[j], src);
      if (turned && have) {
        const float2 w = cs[low ? e0 + j : e0 + j - p.half];
        x[j] = low ? x[j] * w.x - y * w.y : x[j] * w.x + y * w.y;
      }
    }
  } else if (have) {
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const int e = e0 + j;
      if (e < rd) {
        const bool low = e < p.half;
        const float y = Elem<T>::load(row + (low ? e + p.half : e - p.half));
        const float2 w = cs[low ? e : e - p.half];
        x[j] = low ? x[j] * w.x - y * w.y : x[j] * w.x + y * w.y;
      }
    }
  }
}

// One page and head of K or V: rows r_lo..r_hi-1 of the page are new (row r
// at src + r * stride), the rows before r_lo older.
template <typename T, int HD, bool ROT>
__device__ __forceinline__ void put_page(const AppendArgs &a, const T *src, int64_t stride, int r_lo,
                                         int r_hi, uint8_t *codes, uint8_t *scale,
                                         const float2 (*cs)[64], int lane) {
  constexpr int PER_ROW = HD / kChunk, N = kPage * PER_ROW / 32;   // chunks of a row; of a lane
  float x[N][kChunk];
  const int ch = lane % PER_ROW;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = (lane + 32 * i) / PER_ROW;
    const bool have = r >= r_lo && r < r_hi;
#pragma unroll
    for (int j = 0; j < kChunk; ++j) x[i][j] = 0.f;
    if (have) load_vec<T, kChunk>(src + r * stride + ch * kChunk, x[i]);
  }
  uint2 was[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = (lane + 32 * i) / PER_ROW;
    was[i] = make_uint2(0u, 0u);
    if (r < r_lo) was[i] = *reinterpret_cast<const uint2 *>(codes + r * HD + ch * kChunk);
  }
  const int old_byte = r_lo > 0 ? *scale : 0;
  float amax = 0.f;
  bool odd = false;                        // a NaN or an infinity
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = (lane + 32 * i) / PER_ROW;
    const bool have = r >= r_lo && r < r_hi;
    if (ROT) rotate_chunk<T, HD>(a.plan, cs[r], src + r * stride, have, ch, lane, x[i]);
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      odd |= !(fabsf(x[i][j]) < INFINITY);
      amax = fmaxf(amax, fabsf(x[i][j]));
    }
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  odd = __any_sync(0xffffffffu, odd) || old_byte == kScaleNan;
  int e = scale_exponent(amax);
  // older tokens keep at least their scale (a byte that no append wrote is
  // brought into the range)
  const int old_e = min(max(old_byte - kScaleBias, kExpLo), kExpHi);
  if (r_lo > 0) e = max(e, old_e);
  const float down = pow2i(-e), move = pow2i(max(old_byte - kScaleBias - e, -126));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = (lane + 32 * i) / PER_ROW;
    uint2 w;
    if (r < r_lo) {
      if (odd || old_byte - kScaleBias == e) continue;
      const uint32_t c[4] = {was[i].x & 0xffffu, was[i].x >> 16, was[i].y & 0xffffu, was[i].y >> 16};
      uint32_t n[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack_e4m3x2(c[j]);
        n[j] = pack_e4m3x2(f.x * move, f.y * move);
      }
      w = make_uint2(n[0] | n[1] << 16, n[2] | n[3] << 16);
    } else if (r < r_hi) {
      const float *f = x[i];
      w = make_uint2(pack_e4m3x2(f[0] * down, f[1] * down) | pack_e4m3x2(f[2] * down, f[3] * down) << 16,
                     pack_e4m3x2(f[4] * down, f[5] * down) | pack_e4m3x2(f[6] * down, f[7] * down) << 16);
    } else {
      continue;
    }
    *reinterpret_cast<uint2 *>(codes + r * HD + ch * kChunk) = w;
  }
  if (lane == 0) *scale = (uint8_t)(odd ? kScaleNan : e + kScaleBias);
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads)
kvq_append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float2 cs[kPage][64];
  const int64_t item = blockIdx.x;
  // the item's sequence: the last one whose first item is not above it
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_item(__ldg(a.cu_n + mid), mid) <= item) lo = mid; else hi = mid - 1;
  }
  const int b = lo;
  const int c0 = __ldg(a.cu_n + b), rows = __ldg(a.cu_n + b + 1) - c0;
  const int start = __ldg(a.start + b);
  const int n = a.take != nullptr ? __ldg(a.take + b) : rows;
  const int64_t j = item - first_item(c0, b);        // index among the sequence's touched pages
  const int64_t end = (int64_t)start + n;
  if (c0 < 0 || rows < 0 || (int64_t)c0 + rows > a.total_n || n < 0 || n > rows || start < 0 || j < 0 ||
      end > (int64_t)a.max_pages * kPage) {
    if (threadIdx.x == 0) raise_status(a.status, kStatusBadInput);
    return;
  }
  const int64_t pg = start / kPage + j;               // page of the sequence
  if (n == 0 || pg * kPage >= end) return;
  const int page = __ldg(a.block_table + (int64_t)b * a.max_pages + pg);
  if (page < 0 || page >= a.num_pages) {
    if (threadIdx.x == 0) raise_status(a.status, kStatusBadInput);
    return;
  }
  const int pos0 = (int)(pg * kPage);
  const int r_lo = max(0, start - pos0), r_hi = (int)min((int64_t)kPage, end - pos0);
  for (int e = threadIdx.x; e < kPage * 64; e += kThreads) {
    const int r = e >> 6, d = e & 63;
    if (d < a.plan.half && r >= r_lo && r < r_hi) cs[r][d] = rope_plan_cs(a.plan, d, pos0 + r);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)c0 + pos0 - start;    // row of the page's first slot (may be before c0)
  for (int h = warp; h < a.Hkv; h += kWarps) {
    const int64_t at = (int64_t)page * a.Hkv + h;
    put_page<T, HD, true>(a, (const T *)a.k + row0 * a.k_row + h * HD, a.k_row, r_lo, r_hi,
                          a.k_cache + at * kPage * HD, a.k_scale + at, cs, lane);
    put_page<T, HD, false>(a, (const T *)a.v + row0 * a.v_row + h * HD, a.v_row, r_lo, r_hi,
                           a.v_cache + at * kPage * HD, a.v_scale + at, cs, lane);
  }
}

}  // namespace
}  // namespace simsd

using namespace simsd;

extern "C" simsd_status simsd_kvq_append(const simsd_kvq_append_desc *d, void *stream_ptr) {
  if (d == nullptr) return SIMSD_ERR_NULL;
  if (d->dtype != SIMSD_F32 && d->dtype != SIMSD_BF16) return SIMSD_ERR_DTYPE;
  if (d->batch < 1 || d->batch > (1 << 20) || d->num_kv_heads < 1 || d->num_kv_heads > 1024 ||
      (d->head_dim != 64 && d->head_dim != 128) || d->page_size != kPageTokens || d->num_pages < 1 ||
      d->max_pages_per_seq < 1 || d->max_pages_per_seq > (1 << 26) || d->total_n < 0 ||
      d->k_row < 0 || d->v_row < 0)
    return SIMSD_ERR_SHAPE;
  AppendArgs a;
  const simsd_status st = make_rope_plan(d->rope, d->head_dim, &a.plan);
  if (st != SIMSD_OK) return st;
  if (!d->k || !d->v || !d->start || !d->cu_n || !d->k_cache || !d->v_cache || !d->k_scale ||
      !d->v_scale || !d->block_table)
    return SIMSD_ERR_NULL;
  const int64_t row = (int64_t)d->num_kv_heads * d->head_dim;
  a.k_row = d->k_row ? d->k_row : row;
  a.v_row = d->v_row ? d->v_row : row;
  const int es = d->dtype == SIMSD_BF16 ? 2 : 4;
  if (!aligned16(d->k) || !aligned16(d->v) || !aligned16(d->k_cache) || !aligned16(d->v_cache) ||
      (a.k_row * es) % 16 != 0 || (a.v_row * es) % 16 != 0)
    return SIMSD_ERR_ALIGN;
  if (d->workspace == nullptr || ((uintptr_t)d->workspace % kAlign) != 0 || d->workspace_bytes < kAlign)
    return SIMSD_ERR_WORKSPACE;
  if (d->total_n == 0) return SIMSD_OK;
  a.k = d->k; a.v = d->v;
  a.k_cache = (uint8_t *)d->k_cache; a.v_cache = (uint8_t *)d->v_cache;
  a.k_scale = d->k_scale; a.v_scale = d->v_scale;
  a.block_table = d->block_table; a.start = d->start; a.cu_n = d->cu_n; a.take = d->take;
  a.status = (uint32_t *)d->workspace;
  a.batch = d->batch; a.Hkv = d->num_kv_heads; a.max_pages = d->max_pages_per_seq;
  a.num_pages = d->num_pages; a.total_n = d->total_n;
  const dim3 grid((unsigned)first_item(d->total_n, d->batch));
  cudaStream_t stream = (cudaStream_t)stream_ptr;
  if (d->dtype == SIMSD_BF16) {
    if (d->head_dim == 128) kvq_append_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, stream>>>(a);
    else kvq_append_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, stream>>>(a);
  } else {
    if (d->head_dim == 128) kvq_append_kernel<float, 128><<<grid, kThreads, 0, stream>>>(a);
    else kvq_append_kernel<float, 64><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? SIMSD_OK : SIMSD_ERR_CUDA;
}
