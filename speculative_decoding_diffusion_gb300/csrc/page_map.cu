// page_map.cu -- simsd_page_map: block tables and slot maps from request
// lengths.
//
// need_b = ceil((lens_b + n_b) / 16); grow_b and drop_b are what need_b is
// above and below held_b.  With their prefix sums D and E over the batch,
// page j of a growing row is ring entry head + D_b + (j - held_b), page j of
// a shrinking one goes to ring place head + count + E_b + (j - need_b), and a
// sequence is served iff D_b + grow_b <= count (so D needs no second pass:
// after the first sequence that is not served no growing one is).
//
// A few words per sequence, page and token: latency is what it costs, so one
// launch does all of it.  Every CTA scans the whole batch into its shared
// memory (a few KB out of L2) rather than wait for another CTA's scan, then
// takes its share of the pages and tokens; reads of the old state end before
// a CTA counts itself done, and the last one writes the new state.  Taken
// ring entries and given-back places never overlap, since pages held and
// free are at most the ring's entries.  256 decoding sequences 6.5 us (one CTA
// 10.8, one on every SM 7.9); 256 prompts of up to 8192 tokens, 1.07 M slots,
// 13.4 us: 8.6 MB of slots at 0.64 TB/s, after 7 us of launch and scan.
#include <limits.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace simsd {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxBatch = 16384;
constexpr int kStaged = 8192;              // sequences whose lengths and counts are kept as well
                                           // (256 prompts: 14.9 us when read again, 13.1)
constexpr size_t kMapWorkspace = kAlign;   // status word; the done counter at kClaimOffset

struct MapArgs {
  const int32_t *lens, *cu_n, *held, *queue;
  int32_t *ring, *table, *held_out, *queue_out, *served;
  int64_t *slots;
  uint32_t *status;
  int *done;
  int batch, cap, width, total_n;
};

struct Seq {
  int len, n, held, need, c0;
  bool ok, rows_ok;     // rows_ok: its range of cu_n is valid
};

__device__ __forceinline__ Seq make_seq(const MapArgs &a, int len, int held, int c0, int c1) {
  Seq s;
  s.len = len;
  s.held = held;
  s.c0 = c0;
  s.rows_ok = c0 >= 0 && c1 >= c0 && c1 <= a.total_n;
  s.n = s.rows_ok ? c1 - c0 : 0;
  const int64_t end = (int64_t)len + s.n, pages = (end + kPage - 1) / kPage;
  s.ok = s.rows_ok && len >= 0 && end <= INT_MAX && pages <= a.width && held >= 0 && held <= a.width;
  s.need = s.ok ? (int)pages : held;
  return s;
}

// Largest b in [0, n) with p[b] <= g (p non-decreasing, p[0] <= g).
__device__ __forceinline__ int last_not_above(const int *p, int n, int g) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p[mid] <= g) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int wrap(int64_t i, int cap) { return (int)(i >= cap ? i - cap : i); }

__global__ void __launch_bounds__(kThreads, 1)
page_map_kernel(const __grid_constant__ MapArgs a) {
  extern __shared__ int32_t smem[];
  const int n1 = a.batch + 1;
  int *D = smem, *E = D + n1, *C = E + n1;       // exclusive prefix sums; cu_n
  int *len_s = C + n1, *held_s = len_s + n1;     // (batches of up to kStaged)
  const bool staged = a.batch <= kStaged;
  auto seq = [&](int b) {
    return staged ? make_seq(a, len_s[b], held_s[b], C[b], C[b + 1])
                  : make_seq(a, __ldg(a.lens + b), __ldcg(a.held + b), C[b], C[b + 1]);
  };
  __shared__ uint64_t warp_sum[32];
  __shared__ int last_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = __ldcg(a.queue), count = __ldcg(a.queue + 1);
  // scan of (grow | drop << 32), a chunk of kThreads sequences at a time
  uint64_t carry = 0;
  bool bad = false, torn = false;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    uint64_t x = 0;
    if (b < a.batch) {
      const int len = __ldg(a.lens + b), held = __ldcg(a.held + b);
      const int c0 = a.cu_n != nullptr ? __ldg(a.cu_n + b) : 0, c1 = a.cu_n != nullptr ? __ldg(a.cu_n + b + 1) : 0;
      C[b] = c0;
      if (b == a.batch - 1) C[a.batch] = c1;
      if (staged) {
        len_s[b] = len;
        held_s[b] = held;
      }
      const Seq s = make_seq(a, len, held, c0, c1);
      bad |= !s.ok;
      torn |= !s.rows_ok;
      x = (uint64_t)(uint32_t)max(0, s.need - s.held) | (uint64_t)(uint32_t)max(0, s.held - s.need) << 32;
    }
    uint64_t incl = x;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint64_t w = warp_sum[lane], wi = w;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, wi, m);
      if (lane >= m) wi += y;
    }
    const uint64_t before = carry + __shfl_sync(0xffffffffu, wi - w, warp) + incl - x;
    if (b < a.batch) {
      D[b] = (int)(uint32_t)before;
      E[b] = (int)(before >> 32);
    }
    carry += __shfl_sync(0xffffffffu, wi, 31);
    __syncthreads();
  }
  const int wanted = (int)(uint32_t)carry, dropped = (int)(carry >> 32);
  if (threadIdx.x == 0) {
    D[a.batch] = wanted;
    E[a.batch] = dropped;
  }
  const bool falls = __syncthreads_or(torn);     // cu_n is no prefix sum: it cannot be searched
  const bool ring_ok = head >= 0 && head < a.cap && count >= 0 && count <= a.cap &&
                       (int64_t)count + dropped <= a.cap;
  if ((bad || !ring_ok) && blockIdx.x == 0) raise_status(a.status, kStatusBadInput);
  // pages taken: the largest prefix that the free pages cover
  const int taken = !ring_ok ? 0 : wanted <= count ? wanted : D[last_not_above(D, a.batch + 1, count)];
  const int t0 = blockIdx.x * kThreads + threadIdx.x, step = gridDim.x * kThreads;
  // pages given back, and pages taken
  if (ring_ok) {
    for (int g = t0; g < dropped; g += step) {
      const int b = last_not_above(E, a.batch, g);
      const Seq s = seq(b);
      a.ring[wrap((int64_t)head + count + g, a.cap)] =       // count + dropped <= cap: one wrap
          a.table[(int64_t)b * a.width + s.need + (g - E[b])];
    }
    for (int g = t0; g < taken; g += step) {
      const int b = last_not_above(D, a.batch, g);
      const int j = (staged ? held_s[b] : __ldcg(a.held + b)) + (g - D[b]);
      const int page = __ldcg(a.ring + wrap((int64_t)head + g, a.cap));
      if (page < 0 || page >= a.cap) raise_status(a.status, kStatusBadInput);
      a.table[(int64_t)b * a.width + j] = page;
    }
  }
  // slots of the new tokens
  if (a.slots != nullptr && a.cu_n != nullptr) {
    auto put = [&](int t, int b, const Seq &s) {
      const bool served = ring_ok && s.ok && (s.need <= s.held || D[b + 1] <= count);
      int64_t slot = -1;
      if (served) {
        const int pos = s.len + (t - s.c0), j = pos / kPage;
        const int page = j < s.held ? a.table[(int64_t)b * a.width + j]
                                    : __ldcg(a.ring + wrap((int64_t)head + D[b] + (j - s.held), a.cap));
        slot = (int64_t)page * kPage + pos % kPage;
      }
      a.slots[t] = slot;
    };
    if (!falls) {
      const uint32_t end = (uint32_t)max(0, min(a.total_n, C[a.batch]));
      for (uint32_t u = t0; u < end; u += step) {  // (unsigned: a step past the last token may pass 2^31)
        const int t = (int)u, b = find_seq_smem(C, a.batch, t);
        const Seq s = seq(b);
        if (t >= s.c0 && t < s.c0 + s.n) put(t, b, s);
      }
    } else {                                       // every valid range by itself, a token always by the same thread:
      for (int b = 0; b < a.batch; ++b) {          // where two claim it, the later sequence has it
        const Seq s = seq(b);
        if (!s.rows_ok) continue;
        const uint32_t skip = s.c0 > t0 ? ((uint32_t)(s.c0 - t0) + step - 1) / (uint32_t)step : 0u;
        for (uint32_t u = t0 + skip * step; u < (uint32_t)(s.c0 + s.n); u += step) put((int)u, b, s);
      }
    }
  }
  // the new state, once every CTA has read the old one
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last_s = atomicAdd(a.done, 1) == (int)gridDim.x - 1;
    if (last_s) { __threadfence(); *a.done = 0; }
  }
  __syncthreads();
  if (!last_s) return;
  for (int b = threadIdx.x; b < a.batch; b += kThreads) {
    const Seq s = seq(b);
    const bool served = ring_ok && s.ok && (s.need <= s.held || D[b + 1] <= count);
    a.served[b] = served;
    a.held_out[b] = served ? s.need : s.held;
  }
  if (threadIdx.x == 0) {
    a.queue_out[0] = ring_ok ? wrap((int64_t)head + taken, a.cap) : head;
    a.queue_out[1] = ring_ok ? count - taken + dropped : count;
  }
}

simsd_status check(const simsd_page_map_desc *d) {
  if (d == nullptr) return SIMSD_ERR_NULL;
  if (d->batch < 1 || d->batch > kMaxBatch || d->page_size != kPageTokens || d->num_pages < 1 ||
      d->num_pages >= (1 << 30) || d->max_pages_per_seq < 1 || d->total_n < 0 ||
      (int64_t)d->batch * d->max_pages_per_seq >= ((int64_t)1 << 31))
    return SIMSD_ERR_SHAPE;
  return SIMSD_OK;
}

}  // namespace
}  // namespace simsd

using namespace simsd;

extern "C" {

size_t simsd_page_map_workspace_size(const simsd_page_map_desc *d) {
  return check(d) == SIMSD_OK ? kMapWorkspace : 0;
}

simsd_status simsd_page_map(const simsd_page_map_desc *d, void *stream_ptr) {
  const simsd_status st = check(d);
  if (st != SIMSD_OK) return st;
  if (!d->lens || (!d->cu_n && d->total_n > 0) || !d->held || !d->queue || !d->free_pages ||
      !d->block_table || !d->held_out || !d->queue_out || !d->served)
    return SIMSD_ERR_NULL;
  if (d->workspace == nullptr || ((uintptr_t)d->workspace % kAlign) != 0 ||
      d->workspace_bytes < kMapWorkspace)
    return SIMSD_ERR_WORKSPACE;
  MapArgs a;
  a.lens = d->lens; a.cu_n = d->cu_n; a.held = d->held; a.queue = d->queue;
  a.ring = d->free_pages; a.table = d->block_table;
  a.held_out = d->held_out; a.queue_out = d->queue_out; a.served = d->served;
  a.slots = d->slots;
  a.status = (uint32_t *)d->workspace;
  a.done = (int *)((char *)d->workspace + kClaimOffset);
  a.batch = d->batch; a.cap = d->num_pages; a.width = d->max_pages_per_seq; a.total_n = d->total_n;
  // a CTA for every two tokens (or sixteen table entries) a thread, one per SM
  // at most (256 prompts: 38 CTAs 33 us, 76 20, 152 13.4)
  const int64_t work = std::max<int64_t>(d->total_n / (2 * kThreads),
                                         (int64_t)d->batch * d->max_pages_per_seq / (16 * kThreads));
  const int grid = (int)std::min<int64_t>(std::max<int64_t>(work, 1), device_sm_count());
  const size_t smem = (d->batch <= kStaged ? 5 : 3) * (size_t)(d->batch + 1) * sizeof(int32_t);
  if (smem > 48 * 1024) {
    static std::atomic<uint64_t> configured{0};   // one bit per device
    const int dev = current_device();
    const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0;
    if (!bit || !(configured.load() & bit)) {
      if (cudaFuncSetAttribute(page_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               3 * (kMaxBatch + 1) * (int)sizeof(int32_t)) != cudaSuccess)
        return SIMSD_ERR_CUDA;
      configured.fetch_or(bit);
    }
  }
  page_map_kernel<<<grid, kThreads, smem, (cudaStream_t)stream_ptr>>>(a);
  return cudaGetLastError() == cudaSuccess ? SIMSD_OK : SIMSD_ERR_CUDA;
}

}  // extern "C"
