// kv4_read.cu -- simsd_kv4_read: positions of the 4-bit cache back as rows.
//
// A CTA takes 16 rows of the output; codes are multiplied by their scale in f16
// (exact).  Bytes: 9 in for every 16 elements, 16 to 64 out.
// 262144 positions of 8 heads of 128 to bf16: 258 us, 5.3 TB/s (0.80 of the copy
// rate), to fp32 439 us (0.83), to e4m3 184 us (0.68).  No unit is full (bf16: DRAM 64%,
// issue slots 68%, ALU 53%; e4m3: 49%, 62%, 55%, and its 52 registers leave an SM four
// CTAs, whose warps wait for their reads five cycles of each instruction's eleven).
#include "kv4.cuh"
#include "kvq.cuh"
#include "vec.cuh"

namespace simsd {
namespace {

constexpr int kThreads = 256;

struct Read4Args {
  Rows4 rows;
  const uint8_t *cache;
  void *k, *v;
  int64_t k_row, v_row;
  int Hkv;
  FastDiv by_kv;
};

// Elements that a thread takes at a time: 16 bytes of the output or more.
template <typename T> constexpr int kItem = sizeof(T) == 1 ? 16 : 8;

// N elements, f16 pairs h, to a row.
__device__ __forceinline__ void store_item(float *dst, const uint32_t *h) {
  const float2 a = f16x2_to_float2(h[0]), b = f16x2_to_float2(h[1]), c = f16x2_to_float2(h[2]), d = f16x2_to_float2(h[3]);
  reinterpret_cast<float4 *>(dst)[0] = make_float4(a.x, a.y, b.x, b.y);
  reinterpret_cast<float4 *>(dst)[1] = make_float4(c.x, c.y, d.x, d.y);
}
__device__ __forceinline__ void store_item(__nv_bfloat16 *dst, const uint32_t *h) {
  const float2 a = f16x2_to_float2(h[0]), b = f16x2_to_float2(h[1]), c = f16x2_to_float2(h[2]), d = f16x2_to_float2(h[3]);
  *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y), pack_bf16x2(c.x, c.y),
                                               pack_bf16x2(d.x, d.y));
}
// Two f16 pairs as four e4m3 codes (nearest even, saturating).
__device__ __forceinline__ uint32_t pack_e4m3x4(uint32_t a, uint32_t b) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 lo, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 hi, %2;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}" : "=r"(w) : "r"(a), "r"(b));
  return w;
}
__device__ __forceinline__ void store_item(__nv_fp8_e4m3 *dst, const uint32_t *h) {
  *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_e4m3x4(h[0], h[1]), pack_e4m3x4(h[2], h[3]), pack_e4m3x4(h[4], h[5]),
                                               pack_e4m3x4(h[6], h[7]));
}

// A scale byte as the products take it: for e4m3, which has no infinity (and
// whose conversion would make 448 of one), what is not finite is a NaN.
template <typename T>
__device__ __forceinline__ uint32_t scale_for(uint32_t byte) {
  return sizeof(T) == 1 && byte >= 0xf8u ? kScale4Nan : byte;
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const __grid_constant__ Read4Args a) {
  using R = Record<HD>;
  __shared__ Row4 row_s[kTileRows];
  __shared__ int lead_s[kTileRows], n_lead_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = a.rows.tile, row0 = blockIdx.x * tile;
  grid_dep_wait();
  grid_dep_launch();
  find_rows4<kThreads / 32>(a.rows, row0, warp, lane, row_s);
  check_rows4(a.rows);
  __syncthreads();
  if (warp == 0) {
    const bool leads = lane < tile && row_s[lane].leads();
    const uint32_t m = __ballot_sync(0xffffffffu, leads);
    if (leads) lead_s[__popc(m & ((1u << lane) - 1u))] = lane;
    if (lane == 0) n_lead_s = __popc(m);
  }
  __syncthreads();
  // A thread takes N neighbouring elements of a key, or of the two values that
  // share their bytes, so that neighbouring threads write neighbouring bytes; U of
  // them are requested before the first is used.
  constexpr int N = kItem<T>, L = HD / N, W = N / 8, U = sizeof(T) == 2 ? 1 : 2;  // L: threads of a row; W: words of a key's codes
  const int n_lead = n_lead_s;
  if (a.k != nullptr)
    for (int e0 = threadIdx.x; e0 < tile * a.Hkv * L; e0 += U * kThreads) {
      uint32_t c[U][W], sc[U];
      T *dst[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int e = e0 + i * kThreads, u = e % L, rh = e / L, r = div_by(rh, a.by_kv), h = rh - r * a.Hkv;
        const int page = r < tile ? row_s[r].page : -1;
        sc[i] = 0u;
        dst[i] = nullptr;
#pragma unroll
        for (int j = 0; j < W; ++j) c[i][j] = 0u;
        if (page < 0) continue;
        const uint8_t *rec = a.cache + ((int64_t)page * a.Hkv + h) * R::kBytes;
        const int slot = row_s[r].pos & (kPage - 1);
        const uint8_t *src = rec + slot * (HD / 2) + u * (N / 2);
        if constexpr (W == 2) {
          const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src));
          c[i][0] = x.x;
          c[i][1] = x.y;
        } else {
          c[i][0] = __ldg(reinterpret_cast<const uint32_t *>(src));
        }
        sc[i] = __ldg(rec + R::kKs + slot * (HD / 16) + u * N / 16);
        dst[i] = (T *)a.k + (int64_t)(row0 + r) * a.k_row + h * HD + u * N;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (dst[i] == nullptr) continue;
        const uint32_t s = scale4_twice(scale_for<T>(sc[i]), 0);
        uint32_t x[4 * W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint4 p = unpack_e2m1x8(c[i][j]);
          x[4 * j] = mul_f16x2(p.x, s);
          x[4 * j + 1] = mul_f16x2(p.y, s);
          x[4 * j + 2] = mul_f16x2(p.z, s);
          x[4 * j + 3] = mul_f16x2(p.w, s);
        }
        store_item(dst[i], x);
      }
    }
  if (a.v != nullptr)
    for (int e0 = threadIdx.x; e0 < n_lead * a.Hkv * L; e0 += U * kThreads) {
      uint32_t c[U][2 * W], sc[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int e = e0 + i * kThreads, u = e % L, rh = e / L, lead = div_by(rh, a.by_kv), h = rh - lead * a.Hkv;
        sc[i] = 0u;
#pragma unroll
        for (int j = 0; j < 2 * W; ++j) c[i][j] = 0u;
        if (lead >= n_lead) continue;
        const Row4 w = row_s[lead_s[lead]];
        const uint8_t *rec = a.cache + ((int64_t)w.page * a.Hkv + h) * R::kBytes;
        const int pair = (w.pos & (kPage - 1)) >> 1, g = u * N / 16;
        const uint8_t *src = rec + R::v_at(pair, g) + u * N % 16;
        if constexpr (W == 2) {
          const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src));
          c[i][0] = x.x; c[i][1] = x.y; c[i][2] = x.z; c[i][3] = x.w;
        } else {
          const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src));
          c[i][0] = x.x; c[i][1] = x.y;
        }
        sc[i] = __ldg(reinterpret_cast<const uint16_t *>(rec + R::vs_at(pair, g)));
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int e = e0 + i * kThreads, u = e % L, rh = e / L, lead = div_by(rh, a.by_kv), h = rh - lead * a.Hkv;
        if (lead >= n_lead) continue;
        const int r = lead_s[lead];
        const Row4 w = row_s[r];
        const uint32_t s = scale4_pair(scale_for<T>(sc[i] & 0xffu) | scale_for<T>(sc[i] >> 8) << 8);
        uint32_t x[4 * W], y[4 * W];                         // of the even and of the odd token
#pragma unroll
        for (int j = 0; j < 2 * W; ++j) {
          const uint4 p = unpack_e2m1x8(c[i][j]);            // an element a pair: (even, odd)
          const uint32_t p0 = mul_f16x2(p.x, s), p1 = mul_f16x2(p.y, s), p2 = mul_f16x2(p.z, s), p3 = mul_f16x2(p.w, s);
          x[2 * j] = __byte_perm(p0, p1, 0x5410);
          x[2 * j + 1] = __byte_perm(p2, p3, 0x5410);
          y[2 * j] = __byte_perm(p0, p1, 0x7632);
          y[2 * j + 1] = __byte_perm(p2, p3, 0x7632);
        }
        T *dst = (T *)a.v + (int64_t)(row0 + r) * a.v_row + h * HD + u * N;
        if (w.has(0)) store_item(dst, x);
        if (w.has(1)) store_item((w.pos & 1) ? dst : dst + a.v_row, y);
      }
    }
}

template <typename T>
cudaError_t launch_read4(const Read4Args &a, int hd, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.rows.total_n + a.rows.tile - 1) / a.rows.tile)), block(kThreads);
  return hd == 128 ? launch_pdl(kv4_read_kernel<T, 128>, grid, block, 0, stream, a)
                   : launch_pdl(kv4_read_kernel<T, 64>, grid, block, 0, stream, a);
}

}  // namespace
}  // namespace simsd

using namespace simsd;

extern "C" simsd_status simsd_kv4_read(const simsd_kv4_read_desc *d, void *stream_ptr) {
  if (d == nullptr) return SIMSD_ERR_NULL;
  if (d->dtype != SIMSD_F32 && d->dtype != SIMSD_BF16 && d->dtype != SIMSD_E4M3) return SIMSD_ERR_DTYPE;
  if (d->batch < 1 || d->batch > (1 << 20) || d->num_kv_heads < 1 || d->num_kv_heads > 1024 ||
      (d->head_dim != 64 && d->head_dim != 128) || d->page_size != kPageTokens || d->num_pages < 1 ||
      d->max_pages_per_seq < 1 || d->max_pages_per_seq > (1 << 26) || d->total_n < 0 || d->total_n > (1 << 30) || d->k_row < 0 || d->v_row < 0)
    return SIMSD_ERR_SHAPE;
  if ((d->total_n > 0 && !d->k && !d->v) || !d->start || !d->cu_n || !d->cache || !d->block_table)
    return SIMSD_ERR_NULL;
  const int es = d->dtype == SIMSD_F32 ? 4 : d->dtype == SIMSD_BF16 ? 2 : 1;
  Read4Args a;
  const int64_t row = (int64_t)d->num_kv_heads * d->head_dim;
  a.k_row = d->k_row ? d->k_row : row;
  a.v_row = d->v_row ? d->v_row : row;
  if ((d->k && a.k_row < row && d->total_n > 1) || (d->v && a.v_row < row && d->total_n > 1))
    return SIMSD_ERR_SHAPE;                                  // rows that share memory
  if (!aligned16(d->k) || !aligned16(d->v) || !aligned16(d->cache) || a.k_row * es % 16 != 0 || a.v_row * es % 16 != 0)
    return SIMSD_ERR_ALIGN;
  if (d->workspace == nullptr || (uintptr_t)d->workspace % kAlign != 0 || d->workspace_bytes < kAlign)
    return SIMSD_ERR_WORKSPACE;
  if (d->total_n == 0) return SIMSD_OK;
  a.rows = {d->block_table, d->start, d->cu_n, nullptr, (uint32_t *)d->workspace,
            d->batch, d->max_pages_per_seq, d->num_pages, d->total_n, tile_rows4(d->total_n)};
  a.cache = (const uint8_t *)d->cache;
  a.k = d->k;
  a.v = d->v;
  a.Hkv = d->num_kv_heads;
  a.by_kv = make_fast_div(a.Hkv);
  cudaStream_t stream = (cudaStream_t)stream_ptr;
  const cudaError_t e = d->dtype == SIMSD_F32    ? launch_read4<float>(a, d->head_dim, stream)
                        : d->dtype == SIMSD_BF16 ? launch_read4<__nv_bfloat16>(a, d->head_dim, stream)
                                                 : launch_read4<__nv_fp8_e4m3>(a, d->head_dim, stream);
  return e == cudaSuccess ? SIMSD_OK : SIMSD_ERR_CUDA;
}
