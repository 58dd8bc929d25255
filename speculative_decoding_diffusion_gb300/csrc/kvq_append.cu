// kvq_append.cu -- simsd_kvq_append: rotated keys and values into the e4m3
// paged cache.
//
// A page and head's scale is 2^E, E = min{e : amax <= 448 * 2^e}; a value x
// is stored as the e4m3 code nearest to x * 2^-E.  Scaling by a power of two
// keeps the mantissa, so a page that later holds larger tokens moves its
// older codes exactly (up to the subnormal codes) instead of reading the
// tokens again.
//
// A warp takes one page and head at a time, keys then values, sixteen elements
// of a row a lane (both halves of its rotated pairs, so nothing is exchanged);
// the maximum is a warp reduction.  Angles: a page's first position
// (two a lane), times the turn by 0..15 positions from a table that
// the CTA makes once -- one product instead of a sine and a cosine for each
// row.  Bytes in, half as many (bf16) out; what keeps a prompt's append from the
// copy rate is its arithmetic (69% of the issue slots) and latency: while a warp
// works on a page's values the next page's keys are copied into shared memory
// (16-byte asynchronous copies), and so in turn; 16 warps an SM.  256 prompts (1.07 M tokens, bf16,
// 8 heads of 128): 1.22 ms, 5.4 TB/s of its bytes (12 warps with two pages of
// buffers each 1.49; rows held in registers instead 1.50; angles by a sine
// and a cosine for each row and lanes that met in the same banks 1.70 and up).
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "kvq.cuh"
#include "rope_spec.cuh"
#include "vec.cuh"

namespace simsd {
namespace {

// Warps of a CTA (one CTA an SM): a page's raw rows, keys and values, each.
template <typename T, int HD> constexpr int kPageBytes = 2 * kPage * HD * (int)sizeof(T);
// 16 warps where their buffers fit, for rows of 512 bytes 12.
template <typename T, int HD> constexpr int kWarpsOf = kPageBytes<T, HD> <= 8192 ? 16 : 12;
constexpr int kStageSeqs = 1024;          // sequences whose prefix sums are staged in shared memory

struct AppendArgs {
  RopePlan plan;
  const void *k, *v;
  uint8_t *k_cache, *v_cache, *k_scale, *v_scale;
  const int32_t *block_table, *start, *cu_n, *take;
  uint32_t *status;
  int64_t k_row, v_row;
  int batch, Hkv, max_pages, num_pages, total_n;
  int64_t tasks;                          // (page item, head) pairs
};

// Work items: a sequence's touched pages, at most ceil((n + 15) / 16) <=
// floor(n / 16) + 2 of them, numbered from first_item(b); items in the gaps
// do nothing.
__host__ __device__ __forceinline__ int64_t first_item(int32_t cu, int b) { return cu / kPage + 2LL * b; }

__device__ __forceinline__ float2 turn(float2 a, float2 b) {   // complex product
  return make_float2(a.x * b.x - a.y * b.y, a.x * b.y + a.y * b.x);
}

// Where a lane's two chunks of eight elements lie in a head: partners of half
// pairs, else neighbours.
struct Chunks {
  int d1, d2;
  bool paired;                            // (d1 + i, d2 + i) are pairs
};

// Sixteen rotated elements of a lane: u at d1.., v at d2.. (row: the head's
// elements, for partners off the chunk grid); base: the angles of the page's
// first position, of this lane's pairs d1.. (half pairs: base[i] belongs to
// pair d1 + i; interleaved: base[i] to pair d1 / 2 + i, both chunks in turn);
// delta: the turn from there to this row, by pair.
template <typename T, bool IL>
__device__ __forceinline__ void rotate16(const RopePlan &p, const Chunks &c, const float2 *base, const float2 *delta,
                                         const float2 *base_all, const T *row, float *u, float *v) {
  if (IL) {
    const int p0 = c.d1 >> 1;                      // (d2 = d1 + 8: eight pairs in a row)
    float2 dl[8];
    load_angles8(delta, p0, dl);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (p0 + i < p.half) {
        const float2 w = turn(base[i], dl[i]);
        float *z = i < 4 ? u + 2 * i : v + 2 * (i - 4);
        const float a = z[0], b = z[1];
        z[0] = a * w.x - b * w.y;
        z[1] = b * w.x + a * w.y;
      }
    }
  } else if (p.half % 8 == 0) {
    if (c.paired) {
      float2 dl[8];
      load_angles8(delta, c.d1, dl);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 w = turn(base[i], dl[i]);
        const float a = u[i], b = v[i];
        u[i] = a * w.x - b * w.y;
        v[i] = b * w.x + a * w.y;
      }
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const int d = (i < 8 ? c.d1 : c.d2) + (i & 7);
      if (d < 2 * p.half) {
        const bool low = d < p.half;
        const int q = low ? d : d - p.half;
        const float x = Elem<T>::load(row + d), y = Elem<T>::load(row + (low ? d + p.half : q));
        const float2 w = turn(base_all[angle_at(q)], delta[angle_at(q)]);
        const float z = low ? x * w.x - y * w.y : x * w.x + y * w.y;
#pragma unroll
        for (int k = 0; k < 8; ++k) {              // no indexed registers
          u[k] = k == i ? z : u[k];
          v[k] = k + 8 == i ? z : v[k];
        }
      }
    }
  }
}

// One page and head of K or V: rows r_lo..r_hi-1 of the page are new (in
// shared memory, all 16 rows' places), the rows before r_lo older.
template <typename T, int HD, bool ROT, bool IL>
__device__ __forceinline__ void put_page(const RopePlan &plan, const T *rows, int r_lo, int r_hi, uint8_t *codes,
                                         uint8_t *scale, const Chunks &c, int r0, const float2 *base_all,
                                         const float2 (*delta)[64], int lane) {
  constexpr int L = HD / 16;                       // lanes of a row
  constexpr int N = kPage * L / 32;                // rows of a lane
  const int old_byte = r_lo > 0 ? *scale : 0;
  float2 base[8];
  if (ROT && (IL || c.paired)) load_angles8(base_all, IL ? c.d1 >> 1 : c.d1, base);
  float u[N][8], v[N][8], amax = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = r0 + i * (32 / L);
    if (r >= r_lo && r < r_hi) {
      load_vec<T, 8>(rows + r * HD + c.d1, u[i]);
      load_vec<T, 8>(rows + r * HD + c.d2, v[i]);
      if (ROT) rotate16<T, IL>(plan, c, base, delta[r], base_all, rows + r * HD, u[i], v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[i][e] = v[i][e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = absmax_nan(amax, u[i][e], v[i][e]);
  }
  // (non-negative: ordered as bits; a NaN is above the infinity)
  const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(amax) & 0x7fffffffu);
  const bool odd = top >= 0x7f800000u || old_byte == kScaleNan;   // a NaN or an infinity
  int e = scale_exponent(__uint_as_float(top));
  // older tokens keep at least their scale (a byte that no append wrote is
  // brought into the range)
  if (r_lo > 0) e = max(e, min(max(old_byte - kScaleBias, kExpLo), kExpHi));
  const float down = pow2i(-e);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = r0 + i * (32 / L);
    if (r < r_lo || r >= r_hi) continue;
    uint8_t *dst = codes + r * HD;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const float *f = s ? v[i] : u[i];
      *reinterpret_cast<uint2 *>(dst + (s ? c.d2 : c.d1)) =
          make_uint2(pack_e4m3x2(f[0] * down, f[1] * down) | pack_e4m3x2(f[2] * down, f[3] * down) << 16,
                     pack_e4m3x2(f[4] * down, f[5] * down) | pack_e4m3x2(f[6] * down, f[7] * down) << 16);
    }
  }
  // codes of older tokens move to a scale that grew
  if (r_lo > 0 && !odd && old_byte - kScaleBias != e) {
    const float move = pow2i(max(old_byte - kScaleBias - e, -126));
    for (int i = lane; i < r_lo * (HD / 4); i += 32) {
      uint32_t *at = reinterpret_cast<uint32_t *>(codes) + i;
      const uint32_t w = *at;
      const float2 f = unpack_e4m3x2(w & 0xffffu), g = unpack_e4m3x2(w >> 16);
      *at = pack_e4m3x2(f.x * move, f.y * move) | pack_e4m3x2(g.x * move, g.y * move) << 16;
    }
  }
  if (lane == 0) *scale = (uint8_t)(odd ? kScaleNan : e + kScaleBias);
}

template <typename T, int HD, bool IL>
__global__ void __launch_bounds__(32 * kWarpsOf<T, HD>, 1)
kvq_append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ __align__(16) float2 delta_s[kPage][64];
  const int n_threads = blockDim.x, n_warps = n_threads / 32;
  __shared__ __align__(16) float2 base_s[kWarpsOf<T, HD>][64];
  __shared__ int32_t cu_s[kStageSeqs + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RopePlan &plan = plan_by_lane(a.plan);
  const bool staged = a.batch <= kStageSeqs;
  if (staged)
    for (int i = threadIdx.x; i <= a.batch; i += n_threads) cu_s[i] = __ldg(a.cu_n + i);
  // turns by 1, 2, 4 and 8 positions, then the products for the rest
  for (int e = threadIdx.x; e < 4 * 64; e += n_threads) {
    const int r = 1 << (e >> 6), d = e & 63;
    if (d < a.plan.half) delta_s[r][angle_at(d)] = rope_plan_angle(plan, d, r);
  }
  if (threadIdx.x < 64) delta_s[0][threadIdx.x] = make_float2(1.f, 0.f);
  __syncthreads();
  for (int e = threadIdx.x; e < kPage * 64; e += n_threads) {
    const int r = e >> 6, d = angle_at(e & 63), low = r & -r;
    if (r != low && (e & 63) < a.plan.half) {
      float2 w = delta_s[low][d];
      for (int m = 2 * low; m < kPage; m <<= 1)
        if (r & m) w = turn(w, delta_s[m][d]);
      delta_s[r][d] = w;
    }
  }
  __syncthreads();
  auto cu = [&](int b) { return staged ? cu_s[b] : __ldg(a.cu_n + b); };
  // (a sequence whose range is turned round may own no work item)
  for (int i = blockIdx.x * n_threads + threadIdx.x; i < a.batch; i += gridDim.x * n_threads)
    if (cu(i) < 0 || cu(i + 1) < cu(i) || cu(i + 1) > a.total_n) raise_status(a.status, kStatusBadInput);
  extern __shared__ __align__(16) uint8_t pages_s[];         // [warp][K, V][16][HD]
  T *mine = reinterpret_cast<T *>(pages_s) + (int64_t)warp * 2 * kPage * HD;
  constexpr int L = HD / 16;
  const int ln = lane % L, r0 = lane / L;
  Chunks ck, cv;                                   // of keys and of values
  ck.paired = !IL && a.plan.half % 8 == 0 && ln * 8 < a.plan.half;
  ck.d1 = ck.paired ? ln * 8 : ln * 16;
  ck.d2 = ck.paired ? ck.d1 + a.plan.half : ck.d1 + 8;
  cv.paired = false;
  cv.d1 = ln * 16;
  cv.d2 = cv.d1 + 8;
  // A task: its page of the cache (looked up while the task before is worked
  // on), the rows of the page that are new, the row of its first slot.
  struct Task {
    int64_t row0;
    int page, pos0, r_lo, r_hi, h;
    bool any, bad;                                 // new rows; numbers out of range
  };
  int b = -1;                                      // the last task's sequence
  auto find = [&](int64_t task) {
    Task t;
    t.any = t.bad = false;
    t.page = -1;
    if (task >= a.tasks) return t;
    const int64_t item = task / a.Hkv;
    t.h = (int)(task - item * a.Hkv);
    // the item's sequence: the last one whose first item is not above it
    if (b < 0) {
      int lo = 0, hi = a.batch - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_item(cu(mid), mid) <= item) lo = mid; else hi = mid - 1;
      }
      b = lo;
    } else {
      while (b + 1 < a.batch && first_item(cu(b + 1), b + 1) <= item) ++b;
    }
    const int c0 = cu(b), rows = cu(b + 1) - c0;
    const int start = __ldg(a.start + b);
    const int n = a.take != nullptr ? __ldg(a.take + b) : rows;
    const int64_t j = item - first_item(c0, b);    // index among the sequence's touched pages
    const int64_t end = (int64_t)start + n;
    if (c0 < 0 || rows < 0 || (int64_t)c0 + rows > a.total_n || n < 0 || n > rows || start < 0 ||
        end > (int64_t)a.max_pages * kPage) {
      t.bad = true;
      return t;
    }
    const int64_t pg = start / kPage + j;          // page of the sequence
    if (j < 0 || n == 0 || pg * kPage >= end) return t;   // (j < 0: rows before the first sequence's)
    t.any = true;
    t.page = __ldg(a.block_table + (int64_t)b * a.max_pages + pg);
    t.pos0 = (int)(pg * kPage);
    t.r_lo = max(0, start - t.pos0);
    t.r_hi = (int)min((int64_t)kPage, end - t.pos0);
    t.row0 = (int64_t)c0 + t.pos0 - start;         // (may be before c0)
    return t;
  };
  auto good = [&](const Task &t) { return t.any && t.page >= 0 && t.page < a.num_pages; };
  // starts copying a task's new rows, keys (kv 0) or values
  auto fetch = [&](const Task &t, int kv) {
    if (good(t)) {
      constexpr int C = HD * (int)sizeof(T) / 16;  // 16-byte chunks of a row
      const int64_t stride = kv ? a.v_row : a.k_row;
      const T *src = (const T *)(kv ? a.v : a.k) + t.row0 * stride + t.h * HD;
      const uint32_t dst = smem_u32(mine + kv * kPage * HD);
#pragma unroll
      for (int e = lane; e < kPage * C; e += 32) {
        const int r = e / C, ch = e % C;
        if (r >= t.r_lo && r < t.r_hi)
          copy16_async(dst + e * 16, (const char *)(src + r * stride) + ch * 16, true);
      }
    }
    copy_async_commit();
  };
  const int64_t step = (int64_t)gridDim.x * n_warps;
  int64_t task = (int64_t)blockIdx.x * n_warps + warp;
  Task next = find(task);
  fetch(next, 0);
  fetch(next, 1);
  for (; task < a.tasks; task += step) {
    const Task t = next;
    next = find(task + step);
    if ((t.bad || (t.any && !good(t))) && lane == 0) raise_status(a.status, kStatusBadInput);
    if (good(t))
      for (int d = lane; d < a.plan.half; d += 32) base_s[warp][angle_at(d)] = rope_plan_cs(plan, d, t.pos0);
    const int64_t at = (int64_t)t.page * a.Hkv + t.h;
    copy_async_wait<1>();                          // the keys
    __syncwarp();
    if (good(t))
      put_page<T, HD, true, IL>(a.plan, mine, t.r_lo, t.r_hi, a.k_cache + at * kPage * HD, a.k_scale + at, ck, r0,
                                base_s[warp], delta_s, lane);
    __syncwarp();
    fetch(next, 0);
    copy_async_wait<1>();                          // the values
    __syncwarp();
    if (good(t))
      put_page<T, HD, false, IL>(a.plan, mine + kPage * HD, t.r_lo, t.r_hi, a.v_cache + at * kPage * HD, a.v_scale + at,
                                 cv, r0, base_s[warp], delta_s, lane);
    __syncwarp();
    fetch(next, 1);
  }
  copy_async_wait_all();
}

template <typename T, int HD, bool IL>
cudaError_t launch_append_il(const AppendArgs &a, cudaStream_t stream) {
  auto kern = kvq_append_kernel<T, HD, IL>;
  constexpr int W = kWarpsOf<T, HD>, smem = W * kPageBytes<T, HD>;
  static std::atomic<uint64_t> configured{0};   // one bit per device
  const int dev = current_device();
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0;
  if (!bit || !(configured.load() & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  // a CTA per SM, of fewer warps where there are few tasks (64 x 8 tokens: 8
  // warps 5.8 us, 16 on half the SMs 7.1)
  const int64_t sms = device_sm_count(), per_sm = (a.tasks + sms - 1) / sms;
  const int warps = (int)(per_sm < 4 ? 4 : per_sm > W ? W : per_sm);
  const int64_t ctas = (a.tasks + warps - 1) / warps;
  kern<<<(unsigned)(ctas < sms ? ctas : sms), 32 * warps, warps * kPageBytes<T, HD>, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int HD>
cudaError_t launch_append(const AppendArgs &a, cudaStream_t stream) {
  return a.plan.interleaved ? launch_append_il<T, HD, true>(a, stream) : launch_append_il<T, HD, false>(a, stream);
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
  if ((d->total_n > 0 && (!d->k || !d->v)) || !d->start || !d->cu_n || !d->k_cache || !d->v_cache || !d->k_scale ||
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
  a.tasks = first_item(d->total_n, d->batch) * d->num_kv_heads;
  cudaStream_t stream = (cudaStream_t)stream_ptr;
  cudaError_t e;
  if (d->dtype == SIMSD_BF16)
    e = d->head_dim == 128 ? launch_append<__nv_bfloat16, 128>(a, stream) : launch_append<__nv_bfloat16, 64>(a, stream);
  else
    e = d->head_dim == 128 ? launch_append<float, 128>(a, stream) : launch_append<float, 64>(a, stream);
  return e == cudaSuccess ? SIMSD_OK : SIMSD_ERR_CUDA;
}
