// kv4_read.cu -- simsd_kv4_read: positions of the 4-bit cache back as rows.
//
// A CTA takes 16 rows of the output.  A thread takes one group: 16 elements of
// a key, or of the two values that share their bytes; it multiplies codes by
// their scale in f16 (exact) and writes 16 neighbouring elements of a row.
// Bytes bound it: 9 in for every 16 elements, 16 to 64 out.
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

// Four elements of type T from two f16 pairs, as they lie in memory.
template <typename T> struct Out4;
template <> struct Out4<float> {
  using type = float4;
  static __device__ type of(float2 a, float2 b) { return make_float4(a.x, a.y, b.x, b.y); }
};
template <> struct Out4<__nv_bfloat16> {
  using type = uint2;
  static __device__ type of(float2 a, float2 b) { return make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y)); }
};
template <> struct Out4<__nv_fp8_e4m3> {
  using type = uint32_t;
  static __device__ float2 kept(float2 a) {                  // (the conversion would saturate an infinity)
    return make_float2(fabsf(a.x) < INFINITY ? a.x : NAN, fabsf(a.y) < INFINITY ? a.y : NAN);
  }
  static __device__ type of(float2 a, float2 b) {
    a = kept(a);
    b = kept(b);
    return pack_e4m3x2(a.x, a.y) | pack_e4m3x2(b.x, b.y) << 16;
  }
};

// Sixteen elements, f16 pairs h, to a row.
template <typename T>
__device__ __forceinline__ void store16(T *dst, const uint32_t *h) {
  constexpr int N = 16 / (4 * (int)sizeof(T));               // runs of four in 16 bytes
#pragma unroll
  for (int i = 0; i < 4; i += N) {
    union { typename Out4<T>::type o[N]; uint4 v; } u;
#pragma unroll
    for (int j = 0; j < N; ++j)
      u.o[j] = Out4<T>::of(f16x2_to_float2(h[2 * (i + j)]), f16x2_to_float2(h[2 * (i + j) + 1]));
    *reinterpret_cast<uint4 *>(dst + 4 * i) = u.v;
  }
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const __grid_constant__ Read4Args a) {
  using R = Record<HD>;
  __shared__ Row4 row_s[kTileRows];
  __shared__ int lead_s[kTileRows], n_lead_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * kTileRows;
  grid_dep_wait();
  grid_dep_launch();
  for (int r = warp; r < kTileRows; r += kThreads / 32) {
    const Row4 w = find_row4(a.rows, row0 + r, lane);
    if (lane == 0) row_s[r] = w;
  }
  check_rows4(a.rows);
  __syncthreads();
  if (warp == 0) {
    const bool leads = lane < kTileRows && row_s[lane].leads();
    const uint32_t m = __ballot_sync(0xffffffffu, leads);
    if (leads) lead_s[__popc(m & ((1u << lane) - 1u))] = lane;
    if (lane == 0) n_lead_s = __popc(m);
  }
  __syncthreads();
  constexpr int L = HD / 16;                                 // threads of a row
  const int n_lead = n_lead_s;
  if (a.k != nullptr)
    for (int e = threadIdx.x; e < kTileRows * a.Hkv * L; e += kThreads) {
      const int g = e % L, rh = e / L, h = rh % a.Hkv, r = rh / a.Hkv;
      const Row4 w = row_s[r];
      if (w.page < 0) continue;
      const uint8_t *rec = a.cache + ((int64_t)w.page * a.Hkv + h) * R::kBytes;
      const int slot = w.pos & (kPage - 1);
      const uint2 c = __ldg(reinterpret_cast<const uint2 *>(rec + slot * (HD / 2) + g * 8));
      const uint32_t s = scale4_twice(__ldg(rec + R::kKs + slot * (HD / 16) + g), 0);
      const uint4 p = unpack_e2m1x8(c.x), q = unpack_e2m1x8(c.y);
      uint32_t x[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = mul_f16x2(x[i], s);
      store16((T *)a.k + (int64_t)(row0 + r) * a.k_row + h * HD + g * 16, x);
    }
  if (a.v != nullptr)
    for (int e = threadIdx.x; e < n_lead * a.Hkv * L; e += kThreads) {
      const int g = e % L, rh = e / L, h = rh % a.Hkv, r = lead_s[rh / a.Hkv];
      const Row4 w = row_s[r];
      const uint8_t *rec = a.cache + ((int64_t)w.page * a.Hkv + h) * R::kBytes;
      const int pair = (w.pos & (kPage - 1)) >> 1;
      const uint4 c = __ldg(reinterpret_cast<const uint4 *>(rec + R::v_at(pair, g)));
      const uint32_t s = scale4_pair(__ldg(reinterpret_cast<const uint16_t *>(rec + R::vs_at(pair, g))));
      const uint32_t w4[4] = {c.x, c.y, c.z, c.w};
      uint32_t x[8], y[8];                                   // of the even and of the odd token
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 p = unpack_e2m1x8(w4[i]);                // an element a pair: (even, odd)
        const uint32_t a0 = mul_f16x2(p.x, s), a1 = mul_f16x2(p.y, s), a2 = mul_f16x2(p.z, s), a3 = mul_f16x2(p.w, s);
        x[2 * i] = __byte_perm(a0, a1, 0x5410);
        x[2 * i + 1] = __byte_perm(a2, a3, 0x5410);
        y[2 * i] = __byte_perm(a0, a1, 0x7632);
        y[2 * i + 1] = __byte_perm(a2, a3, 0x7632);
      }
      T *dst = (T *)a.v + (int64_t)(row0 + r) * a.v_row + h * HD + g * 16;
      if (w.has(0)) store16(dst, x);
      if (w.has(1)) store16((w.pos & 1) ? dst : dst + a.v_row, y);
    }
}

template <typename T>
cudaError_t launch_read4(const Read4Args &a, int hd, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.rows.total_n + kTileRows - 1) / kTileRows)), block(kThreads);
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
            d->batch, d->max_pages_per_seq, d->num_pages, d->total_n};
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
