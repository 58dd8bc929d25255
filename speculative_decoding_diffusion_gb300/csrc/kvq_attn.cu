// kvq_attn.cu -- simsd_kvq_verify: the host side (checks, key-split plan), the
// CUDA-core attention kernel and the merge of key splits.
//
// For a query row r (new token and query head) with visible keys j,
//   out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = scale q_r . k_j
// (scale holds log2 e), the keys being the prompt's e4m3 codes times their
// page's scale and the new tokens' own rotated keys; a running maximum m and
// sum per row, one pass over the keys.
//
// The CUDA-core kernel (fp32 data: fp32 arithmetic throughout) takes 16 rows
// of a (sequence, KV head) against tiles of 64 keys that are decoded into
// shared memory once for all rows; a warp owns four rows, its lanes two keys
// each for the scores and four columns each for the values.  It serves fp32
// callers and checks; the FMA pipes and shared memory bound it.  One sequence
// of 64 keys, 8 tokens, 4 heads of 64: 10.3 us (a launch and the chain set-up, new
// tile, one tile of the prompt, store; 14.1 with rows loaded element by
// element).
#include <limits.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "kv4.cuh"
#include "kvq.cuh"
#include "kvq_attn.cuh"
#include "vec.cuh"

namespace simsd {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 16;                // rows of a CTA
constexpr int kRowsPerWarp = 4;
constexpr int kTile = 64;                // keys of a tile = the most new tokens
static_assert(kTile == kMaxNew, "the new tokens are one tile");

template <int HD>
struct SimtSmem {
  static constexpr int kLd = HD + 4;     // row stride of q and k: lanes on different banks
  float q[kRows][kLd];
  float k[kTile][kLd];
  float v[kTile][HD];                    // also the angles of the new tokens' positions
  float p[kRows][kTile];
};

// A tile of the prompt's keys and values, decoded; zeros past its end and for
// pages outside the cache.
template <int HD>
__device__ __forceinline__ void load_tile8(const KvqParams &a, const KvqWork &w, const int32_t *bt, int base,
                                           SimtSmem<HD> &s) {
  constexpr int CH = HD / 16;                        // 16-byte chunks of a row
  for (int e = threadIdx.x; e < 2 * kTile * CH; e += kThreads) {
    const bool is_v = e >= kTile * CH;
    const int j = (is_v ? e - kTile * CH : e) / CH, c = e % CH, key = base + j;
    uint4 raw = make_uint4(0, 0, 0, 0);
    float sc = 0.f;
    if (key < w.k_end) {
      const int page = __ldg(bt + key / kPage);
      if (page >= 0 && page < a.num_pages) {
        const int64_t at = (int64_t)page * a.Hkv + w.kvh;
        raw = __ldg(reinterpret_cast<const uint4 *>((is_v ? a.v_cache : a.k_cache) + (at * kPage + key % kPage) * HD) + c);
        sc = scale_value(__ldg((is_v ? a.v_scale : a.k_scale) + at));
      } else {
        raise_status(a.status, kStatusBadInput);
      }
    }
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
    float *dst = is_v ? &s.v[j][c * 16] : &s.k[j][c * 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_e4m3x2(u[i] & 0xffffu), g = unpack_e4m3x2(u[i] >> 16);
      reinterpret_cast<float4 *>(dst)[i] = make_float4(f.x * sc, f.y * sc, g.x * sc, g.y * sc);
    }
  }
}

// The same of a 4-bit cache: a thread takes 16 elements of a key, or of the two
// values that share their bytes.
template <int HD>
__device__ __forceinline__ void load_tile4(const KvqParams &a, const KvqWork &w, const int32_t *bt, int base,
                                           SimtSmem<HD> &s) {
  using R = Record<HD>;
  constexpr int CH = HD / 16;
  for (int e = threadIdx.x; e < (kTile + kTile / 2) * CH; e += kThreads) {
    const bool is_v = e >= kTile * CH;
    const int j = is_v ? (e - kTile * CH) / CH * 2 : e / CH, c = e % CH, key = base + j;
    const uint8_t *rec = nullptr;
    if (key < w.k_end) {
      const int page = __ldg(bt + key / kPage);
      if (page >= 0 && page < a.num_pages) rec = a.k_cache + ((int64_t)page * a.Hkv + w.kvh) * R::kBytes;
      else raise_status(a.status, kStatusBadInput);
    }
    const int slot = key % kPage;
    uint32_t x[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, y[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (rec != nullptr && !is_v) {
      const uint2 q = __ldg(reinterpret_cast<const uint2 *>(rec + slot * (HD / 2) + c * 8));
      const uint32_t sc = scale4_twice(__ldg(rec + R::kKs + slot * (HD / 16) + c), 0);
      const uint4 h = unpack_e2m1x8(q.x), g = unpack_e2m1x8(q.y);
      const uint32_t u[8] = {h.x, h.y, h.z, h.w, g.x, g.y, g.z, g.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = mul_f16x2(u[i], sc);
    } else if (rec != nullptr) {
      const uint4 q = __ldg(reinterpret_cast<const uint4 *>(rec + R::v_at(slot >> 1, c)));
      const uint32_t sc = scale4_pair(__ldg(reinterpret_cast<const uint16_t *>(rec + R::vs_at(slot >> 1, c))));
      const uint32_t q4[4] = {q.x, q.y, q.z, q.w};
      const bool both = key + 1 < w.k_end;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 h = unpack_e2m1x8(q4[i]);
        const uint32_t a0 = mul_f16x2(h.x, sc), a1 = mul_f16x2(h.y, sc), a2 = mul_f16x2(h.z, sc), a3 = mul_f16x2(h.w, sc);
        x[2 * i] = __byte_perm(a0, a1, 0x5410);
        x[2 * i + 1] = __byte_perm(a2, a3, 0x5410);
        y[2 * i] = both ? __byte_perm(a0, a1, 0x7632) : 0u;
        y[2 * i + 1] = both ? __byte_perm(a2, a3, 0x7632) : 0u;
      }
    }
    float *dst = is_v ? &s.v[j][c * 16] : &s.k[j][c * 16];
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<float2 *>(dst + 2 * i) = f16x2_to_float2(x[i]);
    if (is_v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) *reinterpret_cast<float2 *>(&s.v[j + 1][c * 16 + 2 * i]) = f16x2_to_float2(y[i]);
    }
  }
}

template <typename T, int HD, bool FOUR>
__global__ void __launch_bounds__(kThreads)
kvq_simt_kernel(const __grid_constant__ KvqParams a) {
  constexpr int PER = HD / 32;           // columns of a lane
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem<HD> &s = *reinterpret_cast<SimtSmem<HD> *>(smem_raw);
  __shared__ int tau_s[kMaxB];
  __shared__ uint32_t odd_s[kTile / 32];                 // new tokens whose values hold a NaN or an infinity
  grid_dep_wait();
  grid_dep_launch();
  const KvqWork w = kvq_work(a);
  if (!w.ok) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = min(kRows, w.M - w.row0);
  if (threadIdx.x < kTile / 32) odd_s[threadIdx.x] = 0u;
  if (a.order == SIMSD_ORDER_PAIRED && threadIdx.x < w.B) tau_s[threadIdx.x] = __ldg(a.tau + w.c0 + threadIdx.x);
  const int npos = a.order == SIMSD_ORDER_PAIRED ? w.B : a.order == SIMSD_ORDER_NODES ? a.node_size : w.n;
  float2 *cs = reinterpret_cast<float2 *>(&s.v[0][0]);   // [kMaxNew][HD / 2]
  for (int e = threadIdx.x; e < npos * (HD / 2); e += kThreads) {
    const int d = e % (HD / 2);
    cs[e - d + angle_at(d)] = d < a.plan.half ? rope_plan_cs(plan_by_lane(a.plan), d, w.P + e / (HD / 2)) : make_float2(1.f, 0.f);
  }
  __syncthreads();
  const int64_t t0 = (int64_t)a.per * w.c0;              // first new token's row
  constexpr int CH = HD / 8;
  for (int e = threadIdx.x; e < kRows * CH; e += kThreads) {
    const int r = e / CH, c = e % CH;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (r < rows) {
      const int tok = div_by(w.row0 + r, a.by_G), head = w.kvh * a.G + (w.row0 + r) - tok * a.G;
      rotate8(a.plan, cs + kvq_offset(a, w.B, tok) * (HD / 2), (const T *)a.q + (t0 + tok) * a.q_row + head * HD, c * 8, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= a.scale;
    }
    store_vec<float, 8>(&s.q[r][c * 8], x);
  }
  if (w.first) {                                         // keys past the last new token are masked, their values zero
    for (int e = threadIdx.x; e < w.n * CH; e += kThreads) {
      const int j = e / CH, c = e % CH;
      float x[8];
      rotate8(a.plan, cs + kvq_offset(a, w.B, j) * (HD / 2), (const T *)a.k_new + (t0 + j) * a.k_row + w.kvh * HD, c * 8, x);
      store_vec<float, 8>(&s.k[j][c * 8], x);
    }
    __syncthreads();                                     // the angles are read
    for (int e = threadIdx.x; e < kTile * CH; e += kThreads) {
      const int j = e / CH, c = e % CH;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
      if (j < w.n) load_vec<T, 8>((const T *)a.v_new + (t0 + j) * a.v_row + w.kvh * HD + c * 8, x);
      bool odd = false;                                  // (times a weight of 0 it would reach every row)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        odd |= !(fabsf(x[i]) < INFINITY);
        x[i] = fabsf(x[i]) < INFINITY ? x[i] : 0.f;
      }
      if (odd) atomicOr(odd_s + (j >> 5), 1u << (j & 31));
      store_vec<float, 8>(&s.v[j][c * 8], x);
    }
  }
  uint64_t newvis[kRowsPerWarp];
  const int r0 = warp * kRowsPerWarp;
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i)
    newvis[i] = r0 + i < rows ? kvq_visible(a, w.B, tau_s, div_by(w.row0 + r0 + i, a.by_G)) : 0ull;
  float m[kRowsPerWarp], l[kRowsPerWarp], o[kRowsPerWarp][PER];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < PER; ++c) o[i][c] = 0.f;
  }
  const int32_t *bt = a.block_table + (int64_t)w.b * a.max_pages;
  for (int base = w.first ? w.k_begin - kTile : w.k_begin; base < w.k_end; base += kTile) {
    const bool fresh = base < w.k_begin;                 // the new tokens' tile
    uint64_t there = ~0ull;                              // keys of the tile that exist
    if (!fresh) {
      __syncthreads();                                   // the last tile is read
      there = kvq_low_bits(w.k_end - base);
      if constexpr (FOUR) load_tile4<HD>(a, w, bt, base, s);
      else load_tile8<HD>(a, w, bt, base, s);
      // keys of pages outside the cache count as absent
      for (int q = 0; q < kTile / kPage; ++q) {
        const int key = base + q * kPage;
        const int page = key < w.k_end ? __ldg(bt + key / kPage) : 0;
        if (page < 0 || page >= a.num_pages) there &= ~(0xffffull << (q * kPage));
      }
    }
    __syncthreads();
    // scores of the warp's rows: keys lane and lane + 32
    float acc[kRowsPerWarp][2];
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) acc[i][0] = acc[i][1] = 0.f;
#pragma unroll 8
    for (int d = 0; d < HD; d += 4) {
      const float4 k0 = *reinterpret_cast<const float4 *>(&s.k[lane][d]);
      const float4 k1 = *reinterpret_cast<const float4 *>(&s.k[lane + 32][d]);
#pragma unroll
      for (int i = 0; i < kRowsPerWarp; ++i) {
        const float4 q = *reinterpret_cast<const float4 *>(&s.q[r0 + i][d]);
        acc[i][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, acc[i][0]))));
        acc[i][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, acc[i][1]))));
      }
    }
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
      const uint64_t vis = fresh ? newvis[i] : there;
      const float s0 = (vis >> lane) & 1ull ? acc[i][0] : -INFINITY;
      const float s1 = (vis >> (lane + 32)) & 1ull ? acc[i][1] : -INFINITY;
      float mx = fmaxf(s0, s1);
#pragma unroll
      for (int t = 16; t > 0; t >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, t));
      const float m_new = fmaxf(m[i], mx), mu = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2f(m[i] - mu);              // m = -inf: 0
      const float p0 = exp2f(s0 - mu), p1 = exp2f(s1 - mu);
      float ps = p0 + p1;
#pragma unroll
      for (int t = 16; t > 0; t >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, t);
      l[i] = l[i] * alpha + ps;
      m[i] = m_new;
#pragma unroll
      for (int c = 0; c < PER; ++c) o[i][c] *= alpha;
      s.p[r0 + i][lane] = p0;
      s.p[r0 + i][lane + 32] = p1;
    }
    __syncwarp();
    // values: columns lane * PER ..
#pragma unroll 2
    for (int j = 0; j < kTile; j += 4) {
      float4 p[kRowsPerWarp];
#pragma unroll
      for (int i = 0; i < kRowsPerWarp; ++i) p[i] = *reinterpret_cast<const float4 *>(&s.p[r0 + i][j]);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        float v[PER];
#pragma unroll
        for (int c = 0; c < PER; ++c) v[c] = s.v[j + jj][lane * PER + c];
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i) {
          const float pj = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
#pragma unroll
          for (int c = 0; c < PER; ++c) o[i][c] = fmaf(pj, v[c], o[i][c]);
        }
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    if (r0 + i >= rows) continue;
    if (w.first && (newvis[i] & ((uint64_t)odd_s[1] << 32 | odd_s[0])) != 0ull) l[i] = __uint_as_float(0x7fc00000u);
    const int grow = w.row0 + r0 + i;
    const int tok = div_by(grow, a.by_G);
    const int64_t row = (t0 + tok) * a.Hq + w.kvh * a.G + grow - tok * a.G;
    if (w.n_splits == 1) {
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
      for (int c = 0; c < PER; ++c) Elem<T>::store((T *)a.out + row * HD + lane * PER + c, o[i][c] * inv);
    } else {
      const int64_t prow = (int64_t)w.split * a.T * a.Hq + row;
#pragma unroll
      for (int c = 0; c < PER; ++c) a.o_part[prow * HD + lane * PER + c] = o[i][c];
      if (lane == 0) a.ml_part[prow] = make_float2(m[i], l[i]);
    }
  }
}

// The order in which a launch of a few waves takes its sequences: longest
// prompt first, so that its last CTAs are short (64 sequences of up to 4096
// keys, 3.4 waves: 99 us in the batch's order, 87 in this one; equal sequences
// lose the 2.5 us of this kernel, and 13 waves of ragged ones gain nothing: 592
// and 595 us).  Thread i counts the sequences ahead of its own.
constexpr int kOrderMax = 512;
constexpr int kOrderWaves = 8;

__global__ void __launch_bounds__(kOrderMax) kvq_order_kernel(const __grid_constant__ KvqParams a) {
  __shared__ __align__(16) int P[kOrderMax];
  const int i = threadIdx.x;
  grid_dep_launch();
  const int mine = i < a.batch ? __ldg(a.lens + i) : INT_MIN;
  const int c0 = i < a.batch ? __ldg(a.cu_B + i) : 0, c1 = i < a.batch ? __ldg(a.cu_B + i + 1) : 0;
  P[i] = mine;
  __syncthreads();
  if (i >= a.batch) return;
  int rank = 0;
  for (int j = 0; j < a.batch; j += 4) {
    const int4 x = *reinterpret_cast<const int4 *>(P + j);
    rank += (x.x > mine || (x.x == mine && j < i)) + (x.y > mine || (x.y == mine && j + 1 < i)) +
            (x.z > mine || (x.z == mine && j + 2 < i)) + (x.w > mine || (x.w == mine && j + 3 < i));
  }
  a.order_ws[rank] = make_int4(i, c0, c1 - c0, mine);
}

// Merge: out = sum_s 2^(m_s - m*) O_s / sum_s 2^(m_s - m*) l_s, a warp per
// (token, head) row of a split unit; blockIdx.x: a token of one of the last
// merge_seqs sequences in the units' order.
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = kMergeThreads / 32;

template <typename T, int HD>
__global__ void __launch_bounds__(kMergeThreads)
kvq_merge_kernel(const __grid_constant__ KvqParams a) {
  constexpr int PER = HD / 32;
  const int max_n = a.per * a.B_max, lane = threadIdx.x & 31;
  const int hq = blockIdx.y * kMergeRows + (threadIdx.x >> 5), tok = (int)blockIdx.x % max_n;
  const int rank = a.batch - a.merge_seqs + (int)blockIdx.x / max_n;
  grid_dep_wait();
  const int4 seq = kvq_sequence(a, rank);
  const int c0 = seq.y, B = seq.z, P = seq.w;
  if (hq >= a.Hq || kvq_bad(a, c0, B, P) || tok >= a.per * B) return;
  const int64_t tok_row = (int64_t)a.per * c0 + tok;
  const int g = hq / a.G;
  const int rtile = (tok * a.G + hq % a.G) / a.rows_per_tile;
  const int unit = rank * a.Hkv * a.row_tiles + rtile * a.Hkv + g;
  const int ns = unit >= a.tail_from ? (P + a.chunk_tail - 1) / a.chunk_tail : 1;
  if (ns <= 1) return;
  const int64_t row = tok_row * a.Hq + hq, step = (int64_t)a.T * a.Hq;
  float m = -INFINITY;
  for (int s = lane; s < ns; s += 32) m = fmaxf(m, __ldcg(a.ml_part + row + s * step).x);
#pragma unroll
  for (int t = 16; t > 0; t >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, t));
  const float mu = m == -INFINITY ? 0.f : m;
  float den = 0.f, o[PER];
#pragma unroll
  for (int c = 0; c < PER; ++c) o[c] = 0.f;
#pragma unroll 4
  for (int s = 0; s < ns; ++s) {
    const float2 ml = __ldcg(a.ml_part + row + s * step);
    const float wgt = exp2f(ml.x - mu);
    den = fmaf(wgt, ml.y, den);
    const float *src = a.o_part + (row + s * step) * HD + lane * PER;
    float v[PER];
    if constexpr (PER == 4) {
      const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
      const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
      v[0] = x.x; v[1] = x.y;
    }
#pragma unroll
    for (int c = 0; c < PER; ++c) o[c] = fmaf(wgt, v[c], o[c]);
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  T *dst = (T *)a.out + row * HD + lane * PER;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int c = 0; c < PER; c += 2)
      reinterpret_cast<uint32_t *>(dst)[c / 2] = pack_bf16x2(o[c] * inv, o[c + 1] * inv);
  } else {
#pragma unroll
    for (int c = 0; c < PER; ++c) dst[c] = o[c] * inv;
  }
}

template <typename T, int HD, bool FOUR>
cudaError_t launch_simt_t(const KvqPlan &p, const KvqParams &a, cudaStream_t stream) {
  auto kern = kvq_simt_kernel<T, HD, FOUR>;
  const int smem = (int)sizeof(SimtSmem<HD>);
  static std::atomic<uint64_t> configured{0};   // one bit per device
  const int dev = current_device();
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0;
  if (!bit || !(configured.load() & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  return launch_pdl(kern, dim3((unsigned)p.grid), dim3(kThreads), smem, stream, a);
}

// Key splits, in block-times of 128 keys on an SM: a CTA costs its blocks plus
// a ramp (set-up, rows, epilogue; over ten shapes of 3 to 64 sequences 6 is the
// best or within 1% of it, 3 and 12 up to 5% worse), and splits the merge's
// launch and reads.  A partial wave costs as much as a full one: the softmax's
// chain bounds an SM's rate, so idle SMs do not speed up the others.
constexpr int64_t kRamp = 6;
constexpr int kMaxSplits = 64;

struct Cut {
  int64_t per, n;                        // blocks of a piece but the last of a unit; pieces
  double time;
};

// The best cut of `units` units of `blocks` blocks each: equal pieces, or (if
// `uneven`) as many long ones as fit the SMs at once while the units' short
// ends take turns on the SMs that are left (8 sequences of 32768 keys, 8 heads:
// 64 units in halves 179 us, in 112 + 112 + 33 blocks 164).
Cut cut_units(int64_t units, int64_t blocks, int64_t slots, bool uneven, int64_t ramp) {
  Cut best = {blocks, 1, (double)((units + slots - 1) / slots * (blocks + ramp))};
  auto merged = [&](int64_t n) { return 2.0 + 2.0 * (double)(units * n) / (double)slots; };
  const int64_t most = std::min<int64_t>(std::min<int64_t>(kMaxSplits, blocks), 4 * slots / units + 1);
  for (int64_t s = 2; s <= most; ++s) {
    const int64_t per = (blocks + s - 1) / s;
    if ((blocks + per - 1) / per < s) continue;            // same split as a smaller s
    const double t = (double)((units * s + slots - 1) / slots * (per + ramp)) + merged(s);
    if (t < best.time) best = {per, s, t};
  }
  const int64_t e = std::min<int64_t>(slots / units, kMaxSplits - 1), left = slots - e * units;
  if (uneven && e > 0 && left > 0) {
    const int64_t k = (units + left - 1) / left;           // ends an SM takes in turn
    const int64_t per = (k * (blocks + ramp) - ramp + k * e) / (1 + k * e);
    if (per > 0 && e * per < blocks && blocks - e * per <= per) {
      const double t = (double)std::max(per + ramp, k * (blocks - e * per + ramp)) + merged(e + 1);
      if (t < best.time) best = {per, e + 1, t};
    }
  }
  return best;
}

// Every unit alike, or whole waves of whole units and the rest cut in equal
// pieces to fill the last wave, as simsd_verify_attn's plan (64 sequences of
// 4096 keys, 56 units of 512 in the fourth wave: 162 us whole, 156 in halves, 158
// in 15 + 15 + 3 blocks).
void plan_splits(int64_t batch, int64_t units_per_seq, int64_t max_keys, int64_t slots, int64_t ramp, KvqPlan *p) {
  const int64_t blocks = std::max<int64_t>(1, (max_keys + kBlockKeys - 1) / kBlockKeys);
  const int64_t pairs = batch * units_per_seq, W = pairs / slots, r = pairs - W * slots;
  Cut cut = cut_units(pairs, blocks, slots, true, ramp);
  int64_t whole = cut.n > 1 ? 0 : pairs;
  if (W > 0 && r > 0) {
    const Cut tail = cut_units(r, blocks, slots, false, ramp);
    if (tail.n > 1 && (double)(W * (blocks + ramp)) + tail.time < cut.time) {
      cut = tail;
      whole = W * slots;
    }
  }
  p->n_splits = p->s_tail = (int)cut.n;
  p->chunk_tail = (int)(cut.per * kBlockKeys);
  p->tail_from = (int)whole;
  p->tail_first = whole > 0 && whole < pairs && W <= 4;    // few full waves: the cut units' SMs start offset
  p->grid = (int)(whole + (pairs - whole) * cut.n);
  p->merge_seqs = (int)(whole == 0 ? batch : std::min<int64_t>(batch, (r + units_per_seq - 1) / units_per_seq + 1));
  p->ranked = p->grid > slots && pairs < kOrderWaves * slots && batch > 1 && batch <= kOrderMax;
}

simsd_status kvq_plan(const simsd_kvq_verify_desc *d, bool four, KvqPlan *p) {
  if (d == nullptr) return SIMSD_ERR_NULL;
  if (d->dtype != SIMSD_F32 && d->dtype != SIMSD_BF16) return SIMSD_ERR_DTYPE;
  const bool paired = d->order == SIMSD_ORDER_PAIRED;
  if (d->batch < 1 || d->num_q_heads < 1 || d->num_kv_heads < 1 || d->num_q_heads % d->num_kv_heads != 0 ||
      d->num_q_heads > 65535 || (d->head_dim != 64 && d->head_dim != 128) || d->page_size != kPageTokens ||
      d->num_pages < 1 || d->max_pages_per_seq < 1 || d->max_pages_per_seq >= (1 << 26) ||
      d->order < SIMSD_ORDER_PAIRED || d->order > SIMSD_ORDER_CAUSAL || d->B_max < 1 ||
      d->B_max > (paired ? kMaxB : kMaxNew) || d->total_B < d->batch || d->total_B > (1 << 28) ||
      (int64_t)d->total_B > (int64_t)d->batch * d->B_max || !(d->sm_scale > 0.0f) ||
      !(d->sm_scale < INFINITY) || d->q_row < 0 || d->k_row < 0 || d->v_row < 0 ||
      (d->order == SIMSD_ORDER_NODES ? d->node_size < 1 || d->node_size > kMaxNew : d->node_size != 0))
    return SIMSD_ERR_SHAPE;
  RopePlan rope;
  const simsd_status st = make_rope_plan(d->rope, d->head_dim, &rope);
  if (st != SIMSD_OK) return st;
  memset(p, 0, sizeof(*p));
  p->per = paired ? 2 : 1;
  p->T = p->per * d->total_B;
  p->G = d->num_q_heads / d->num_kv_heads;
  p->esize = d->dtype == SIMSD_BF16 ? 2 : 4;
  const int max_n = p->per * d->B_max;
  const bool tc = d->dtype == SIMSD_BF16;
  const int64_t max_rows = (int64_t)max_n * p->G;
  p->four = four;
  p->rows_per_tile = !tc ? kRows : four ? kv4_rows_per_tile(max_rows) : 128;
  p->row_tiles = (int)((max_rows + p->rows_per_tile - 1) / p->rows_per_tile);
  const int64_t per_seq = (int64_t)d->num_kv_heads * p->row_tiles;
  if (per_seq * d->batch * 64 >= ((int64_t)1 << 31)) return SIMSD_ERR_SHAPE;
  const bool few = p->few = tc && four && p->rows_per_tile <= kFewRows;
  const int sms = device_sm_count();
  // CTAs of an SM.  Few rows of a 4-bit cache: two, or where there are units for
  // two waves of them four of half as many warps (256 sequences of 256..8192 keys,
  // 4 rows: 214 and not 230 us; 64 of up to 4096, less than a wave: 55 and not 39);
  // six warps for 16 rows, whose sums take twice the registers.
  p->warps = p->rows_per_tile == 16 ? 6 : per_seq * d->batch >= 8 * sms ? 4 : 8;
  const int ctas = !tc ? 2 : !few ? 1 : p->warps == 4 ? 4 : 2;
  plan_splits(d->batch, per_seq, (int64_t)d->max_pages_per_seq * kPageTokens, ctas * sms, few ? 2 : kRamp, p);
  if ((int64_t)p->merge_seqs * max_n >= ((int64_t)1 << 31)) return SIMSD_ERR_SHAPE;
  size_t off = kAlign;
  p->off_order = off;
  if (p->ranked) off = align_up(off + (size_t)d->batch * sizeof(int4), kAlign);
  p->off_opart = p->off_ml = off;
  if (p->n_splits > 1) {
    const size_t rows = (size_t)p->n_splits * p->T * d->num_q_heads;
    off = align_up(off + rows * d->head_dim * sizeof(float), kAlign);
    p->off_ml = off;
    off = align_up(off + rows * sizeof(float2), kAlign);
  }
  p->total = off;
  return SIMSD_OK;
}

}  // namespace

cudaError_t launch_kvq_simt(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a,
                            cudaStream_t stream) {
  if (p.four)
    return d->head_dim == 128 ? launch_simt_t<float, 128, true>(p, a, stream)
                              : launch_simt_t<float, 64, true>(p, a, stream);
  return d->head_dim == 128 ? launch_simt_t<float, 128, false>(p, a, stream)
                            : launch_simt_t<float, 64, false>(p, a, stream);
}

cudaError_t launch_kvq_merge(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a,
                             cudaStream_t stream) {
  const dim3 grid((unsigned)(p.merge_seqs * p.per * d->B_max), (unsigned)((d->num_q_heads + kMergeRows - 1) / kMergeRows));
  const dim3 block(kMergeThreads);
  if (d->dtype == SIMSD_BF16)
    return d->head_dim == 128 ? launch_pdl(kvq_merge_kernel<__nv_bfloat16, 128>, grid, block, 0, stream, a)
                              : launch_pdl(kvq_merge_kernel<__nv_bfloat16, 64>, grid, block, 0, stream, a);
  return d->head_dim == 128 ? launch_pdl(kvq_merge_kernel<float, 128>, grid, block, 0, stream, a)
                            : launch_pdl(kvq_merge_kernel<float, 64>, grid, block, 0, stream, a);
}

namespace {

// The 8-bit cache's call, or (four) the 4-bit cache's, whose descriptor has been
// brought to the same form: k_cache is its records, the other three are not read.
simsd_status run_verify(const simsd_kvq_verify_desc *d, bool four, void *stream_ptr) {
  KvqPlan p;
  const simsd_status st = kvq_plan(d, four, &p);
  if (st != SIMSD_OK) return st;
  if (!d->q || !d->k_cache || !d->v_cache || !d->k_scale || !d->v_scale || !d->block_table || !d->k_new ||
      !d->v_new || (d->order == SIMSD_ORDER_PAIRED && !d->tau) || !d->lens || !d->cu_B || !d->out)
    return SIMSD_ERR_NULL;
  KvqParams a;
  (void)make_rope_plan(d->rope, d->head_dim, &a.plan);
  a.q_row = d->q_row ? d->q_row : (int64_t)d->num_q_heads * d->head_dim;
  a.k_row = d->k_row ? d->k_row : (int64_t)d->num_kv_heads * d->head_dim;
  a.v_row = d->v_row ? d->v_row : (int64_t)d->num_kv_heads * d->head_dim;
  const int es = (int)p.esize;
  if (!aligned16(d->q) || !aligned16(d->k_cache) || !aligned16(d->v_cache) || !aligned16(d->k_new) ||
      !aligned16(d->v_new) || !aligned16(d->out) || (a.q_row * es) % 16 != 0 || (a.k_row * es) % 16 != 0 ||
      (a.v_row * es) % 16 != 0)
    return SIMSD_ERR_ALIGN;
  if (d->workspace == nullptr || ((uintptr_t)d->workspace % kAlign) != 0 || d->workspace_bytes < p.total)
    return SIMSD_ERR_WORKSPACE;
  char *ws = (char *)d->workspace;
  a.q = d->q; a.k_new = d->k_new; a.v_new = d->v_new; a.out = d->out;
  a.k_cache = (const uint8_t *)d->k_cache; a.v_cache = (const uint8_t *)d->v_cache;
  a.k_scale = d->k_scale; a.v_scale = d->v_scale;
  a.block_table = d->block_table; a.tau = d->tau; a.lens = d->lens; a.cu_B = d->cu_B;
  a.o_part = (float *)(ws + p.off_opart);
  a.ml_part = (float2 *)(ws + p.off_ml);
  a.status = (uint32_t *)ws;
  a.batch = d->batch; a.Hq = d->num_q_heads; a.Hkv = d->num_kv_heads; a.G = p.G; a.T = p.T;
  a.total_B = d->total_B; a.B_max = d->B_max; a.order = d->order; a.node_size = d->node_size; a.per = p.per;
  a.max_pages = d->max_pages_per_seq; a.num_pages = d->num_pages;
  a.rows_per_tile = p.rows_per_tile; a.row_tiles = p.row_tiles;
  a.tail_from = p.tail_from; a.s_tail = p.s_tail; a.chunk_tail = p.chunk_tail; a.tail_first = p.tail_first;
  a.order_ws = p.ranked ? (int4 *)(ws + p.off_order) : nullptr;
  a.merge_seqs = p.merge_seqs;
  a.n_tail = p.grid - p.tail_from;
  a.n_whole = p.s_tail > 1 ? a.n_tail / p.s_tail * (p.s_tail - 1) : a.n_tail;
  a.by_seq = make_fast_div(a.Hkv * a.row_tiles);
  a.by_kv = make_fast_div(a.Hkv);
  a.by_split = make_fast_div(std::max(1, p.s_tail - 1));
  a.by_G = make_fast_div(a.G);
  a.by_node = make_fast_div(std::max(1, a.node_size));
  a.polls = wait_polls_of(d->wait_polls);
  a.scale = d->sm_scale * 1.4426950408889634f;
  cudaStream_t stream = (cudaStream_t)stream_ptr;
  cudaError_t e = cudaSuccess;
  if (p.ranked) {
    kvq_order_kernel<<<1, kOrderMax, 0, stream>>>(a);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess)
    e = d->dtype != SIMSD_BF16 ? launch_kvq_simt(d, p, a, stream)
        : !four                ? launch_kvq_tc(d, p, a, stream)
        : p.few                ? launch_kv4_mma(d, p, a, stream) : launch_kv4_tc(d, p, a, stream);
  if (e == cudaSuccess && p.n_splits > 1) e = launch_kvq_merge(d, p, a, stream);
  return e == cudaSuccess ? SIMSD_OK : SIMSD_ERR_CUDA;
}

// A 4-bit call's descriptor in the 8-bit call's form.
simsd_kvq_verify_desc from_four(const simsd_kv4_verify_desc &f) {
  simsd_kvq_verify_desc d;
  d.batch = f.batch; d.num_q_heads = f.num_q_heads; d.num_kv_heads = f.num_kv_heads; d.head_dim = f.head_dim;
  d.page_size = f.page_size; d.num_pages = f.num_pages; d.max_pages_per_seq = f.max_pages_per_seq;
  d.total_B = f.total_B; d.B_max = f.B_max; d.dtype = f.dtype; d.order = f.order; d.node_size = f.node_size;
  d.rope = f.rope; d.sm_scale = f.sm_scale; d.wait_polls = f.wait_polls;
  d.q_row = f.q_row; d.k_row = f.k_row; d.v_row = f.v_row;
  d.q = f.q; d.k_cache = d.v_cache = f.cache;
  d.k_scale = d.v_scale = (const uint8_t *)f.cache;
  d.block_table = f.block_table; d.k_new = f.k_new; d.v_new = f.v_new; d.tau = f.tau; d.lens = f.lens;
  d.cu_B = f.cu_B; d.out = f.out; d.workspace = f.workspace; d.workspace_bytes = f.workspace_bytes;
  return d;
}

}  // namespace
}  // namespace simsd

using namespace simsd;

extern "C" {

size_t simsd_kvq_verify_workspace_size(const simsd_kvq_verify_desc *d) {
  KvqPlan p;
  return kvq_plan(d, false, &p) == SIMSD_OK ? p.total : 0;
}

simsd_status simsd_kvq_verify(const simsd_kvq_verify_desc *d, void *stream) { return run_verify(d, false, stream); }

size_t simsd_kv4_verify_workspace_size(const simsd_kv4_verify_desc *d) {
  if (d == nullptr) return 0;
  const simsd_kvq_verify_desc e = from_four(*d);
  KvqPlan p;
  return kvq_plan(&e, true, &p) == SIMSD_OK ? p.total : 0;
}

simsd_status simsd_kv4_verify(const simsd_kv4_verify_desc *d, void *stream) {
  if (d == nullptr) return SIMSD_ERR_NULL;
  const simsd_kvq_verify_desc e = from_four(*d);
  return run_verify(&e, true, stream);
}

}  // extern "C"
