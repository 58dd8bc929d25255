// kv4_read.cu -- simsd_kv4_read: positions of the 4-bit cache back as rows.
//
// A CTA takes 16 rows of the output; codes are multiplied by their scale in f16
// (exact).  Bytes bound it: 9 in for every 16 elements, 16 to 64 out.
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
};

// Eight elements, f16 pairs h, to a row.
__device__ __forceinline__ void store8(float *dst, const uint4 &h) {
  const float2 a = f16x2_to_float2(h.x), b = f16x2_to_float2(h.y), c = f16x2_to_float2(h.z), d = f16x2_to_float2(h.w);
  reinterpret_cast<float4 *>(dst)[0] = make_float4(a.x, a.y, b.x, b.y);
  reinterpret_cast<float4 *>(dst)[1] = make_float4(c.x, c.y, d.x, d.y);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *dst, const uint4 &h) {
  const float2 a = f16x2_to_float2(h.x), b = f16x2_to_float2(h.y), c = f16x2_to_float2(h.z), d = f16x2_to_float2(h.w);
  *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y), pack_bf16x2(c.x, c.y),
                                               pack_bf16x2(d.x, d.y));
}
__device__ __forceinline__ uint32_t e4m3x2(uint32_t h) {
  const float2 f = f16x2_to_float2(h);                       // (the conversion would saturate an infinity)
  return pack_e4m3x2(fabsf(f.x) < INFINITY ? f.x : NAN, fabsf(f.y) < INFINITY ? f.y : NAN);
}
__device__ __forceinline__ void store8(__nv_fp8_e4m3 *dst, const uint4 &h) {
  *reinterpret_cast<uint2 *>(dst) = make_uint2(e4m3x2(h.x) | e4m3x2(h.y) << 16, e4m3x2(h.z) | e4m3x2(h.w) << 16);
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
  for (int r = warp; r < tile; r += kThreads / 32) {
    const Row4 w = find_row4(a.rows, row0 + r, lane);
    if (lane == 0) row_s[r] = w;
  }
  check_rows4(a.rows);
  __syncthreads();
  if (warp == 0) {
    const bool leads = lane < tile && row_s[lane].leads();
    const uint32_t m = __ballot_sync(0xffffffffu, leads);
    if (leads) lead_s[__popc(m & ((1u << lane) - 1u))] = lane;
    if (lane == 0) n_lead_s = __popc(m);
  }
  __syncthreads();
  // A thread takes eight elements of a key, or of the two values that share their
  // bytes, so that neighbouring threads write neighbouring bytes; U of them are
  // requested before the first is used.
  constexpr int L = HD / 8, U = 4;                           // threads of a row
  const int n_lead = n_lead_s;
  if (a.k != nullptr)
    for (int e0 = threadIdx.x; e0 < tile * a.Hkv * L; e0 += U * kThreads) {
      uint32_t c[U], sc[U];
      T *dst[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int e = e0 + i * kThreads, u = e % L, rh = e / L, h = rh % a.Hkv, r = rh / a.Hkv;
        const int page = r < tile ? row_s[r].page : -1;
        c[i] = sc[i] = 0u;
        dst[i] = nullptr;
        if (page < 0) continue;
        const uint8_t *rec = a.cache + ((int64_t)page * a.Hkv + h) * R::kBytes;
        const int slot = row_s[r].pos & (kPage - 1);
        c[i] = __ldg(reinterpret_cast<const uint32_t *>(rec + slot * (HD / 2) + u * 4));
        sc[i] = __ldg(rec + R::kKs + slot * (HD / 16) + (u >> 1));
        dst[i] = (T *)a.k + (int64_t)(row0 + r) * a.k_row + h * HD + u * 8;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (dst[i] == nullptr) continue;
        const uint32_t s = scale4_twice(sc[i], 0);
        const uint4 p = unpack_e2m1x8(c[i]);
        store8(dst[i], make_uint4(mul_f16x2(p.x, s), mul_f16x2(p.y, s), mul_f16x2(p.z, s), mul_f16x2(p.w, s)));
      }
    }
  if (a.v != nullptr)
    for (int e0 = threadIdx.x; e0 < n_lead * a.Hkv * L; e0 += U * kThreads) {
      uint2 c[U];
      uint32_t sc[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int e = e0 + i * kThreads, u = e % L, rh = e / L, h = rh % a.Hkv, lead = rh / a.Hkv;
        c[i] = make_uint2(0u, 0u);
        sc[i] = 0u;
        if (lead >= n_lead) continue;
        const Row4 w = row_s[lead_s[lead]];
        const uint8_t *rec = a.cache + ((int64_t)w.page * a.Hkv + h) * R::kBytes;
        const int pair = (w.pos & (kPage - 1)) >> 1;
        c[i] = __ldg(reinterpret_cast<const uint2 *>(rec + R::v_at(pair, u >> 1) + (u & 1) * 8));
        sc[i] = __ldg(reinterpret_cast<const uint16_t *>(rec + R::vs_at(pair, u >> 1)));
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int e = e0 + i * kThreads, u = e % L, rh = e / L, h = rh % a.Hkv, lead = rh / a.Hkv;
        if (lead >= n_lead) continue;
        const int r = lead_s[lead];
        const Row4 w = row_s[r];
        const uint32_t s = scale4_pair(sc[i]);
        uint4 p = unpack_e2m1x8(c[i].x), q = unpack_e2m1x8(c[i].y);     // an element a pair: (even, odd) token
        p = make_uint4(mul_f16x2(p.x, s), mul_f16x2(p.y, s), mul_f16x2(p.z, s), mul_f16x2(p.w, s));
        q = make_uint4(mul_f16x2(q.x, s), mul_f16x2(q.y, s), mul_f16x2(q.z, s), mul_f16x2(q.w, s));
        T *dst = (T *)a.v + (int64_t)(row0 + r) * a.v_row + h * HD + u * 8;
        if (w.has(0))
          store8(dst, make_uint4(__byte_perm(p.x, p.y, 0x5410), __byte_perm(p.z, p.w, 0x5410),
                                 __byte_perm(q.x, q.y, 0x5410), __byte_perm(q.z, q.w, 0x5410)));
        if (w.has(1))
          store8((w.pos & 1) ? dst : dst + a.v_row,
                 make_uint4(__byte_perm(p.x, p.y, 0x7632), __byte_perm(p.z, p.w, 0x7632),
                            __byte_perm(q.x, q.y, 0x7632), __byte_perm(q.z, q.w, 0x7632)));
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
      d->max_pages_per_seq < 1 || d->max_pages_per_seq > (1 << 26) || d->total_n < 0 || d->k_row < 0 || d->v_row < 0)
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
  cudaStream_t stream = (cudaStream_t)stream_ptr;
  const cudaError_t e = d->dtype == SIMSD_F32    ? launch_read4<float>(a, d->head_dim, stream)
                        : d->dtype == SIMSD_BF16 ? launch_read4<__nv_bfloat16>(a, d->head_dim, stream)
                                                 : launch_read4<__nv_fp8_e4m3>(a, d->head_dim, stream);
  return e == cudaSuccess ? SIMSD_OK : SIMSD_ERR_CUDA;
}
