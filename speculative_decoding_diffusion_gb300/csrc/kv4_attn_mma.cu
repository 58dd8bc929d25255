// kv4_attn_mma.cu -- simsd_kv4_verify for bf16 data, few query rows a KV head
// (decode steps, short blocks).
//
// A CTA owns up to 16 rows of a (sequence, KV head) and a range of its keys; its
// warps take 32 keys (two pages) in turns, each with a running reference, sums and
// an output of its own, merged at the end.  Codes go from shared memory to
// registers, where a conversion and a product with the group's scale make them the
// f16 operand of an MMA: S^T = K Q^T and O^T += V^T P^T, so that keys (and the
// head's elements) fill the 16 rows of an MMA and the query rows its 8 columns,
// nothing decoded is ever stored, and the cache's order of bytes is that of the
// operands: a lane's elements of a key lie together, and a value byte holds the two
// neighbouring keys that share a register.  The weights P change from the product's
// layout to the operand's by transposing 8 x 8 tiles in registers.
//
// A page and head is one bulk copy of 18 hd bytes into the warp's own ring, so
// warps meet only for the set-up and the merge.
//
// Bytes bound it where there are many units: 256 sequences of 256..8192 keys, one
// token, 32 / 8 heads of 128, take 214 us, 0.92 of the copy rate; 64 of 1..4096 39 us
// (0.60: set-up, rows and the last wave), 8 of 32768 61 us (0.74).  With 16 rows no
// unit is full (64 x 4096, 92 us, 0.50: issue slots 46%, tensor pipe 34%, DRAM 42%): 168
// registers leave an SM twelve warps, too few to cover their own fixed latencies.
// Beyond 16 rows the tcgen05 kernel takes over.  At 24 rows this one, in six warps, takes
// 20 us of 16 x 1024 keys and 33 of 4 x 8192 where that one takes 15 and 26.5, but 123 of
// 64 x 4096 and 445 of 256 x 256..8192 where that one takes 128 and 495: the border is the
// few-unit one, and many units lose a tenth by it.  At 32 rows this one spills (215 us of
// 64 x 4096, that one 129).
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "kvq.cuh"
#include "kvq_attn.cuh"
#include "vec.cuh"

namespace simsd {
namespace {

constexpr int kBlock = 32;                 // keys that a warp takes at a time
constexpr float kHeadroom = 8.f;           // log2 units a row's scores may outgrow its reference by
constexpr float kLift = 7.f;               // log2 of the largest weight right after it moved

template <int HD, int NT, int W>
struct Lay {
  static constexpr int kWarps = W, kThreads = 32 * W;
  static constexpr int kRows = 8 * NT;
  static constexpr int kRec = Record<HD>::kBytes, kStage = 2 * kRec;
  static constexpr int kStages = HD == 64 ? 4 : 2;
  static constexpr int kCtas = W == 4 ? 4 : 2;             // of an SM
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kXld = 68;                      // floats of a row in the merge
  static constexpr int kOffQ = kRing;                  // query operands, lane by lane
  static constexpr int kOffRow = kOffQ + kRows * HD * 2;
  static constexpr int kOffVis = kOffRow + kRows * 4;  // new tokens that a row sees
  static constexpr int kOffMl = kOffVis + kRows * 8;   // [warps][rows] (reference, sum)
  static constexpr int kOffBar = kOffMl + kWarps * kRows * 8;
  static constexpr int kOffTau = kOffBar + kWarps * kStages * 8;
  static constexpr int kOffNewKv = kOffTau + kMaxB * 4;        // new tokens: 2^ke, ve; kShareLift - ve
  static constexpr int kOffNewShare = kOffNewKv + kMaxNew * 8;
  static constexpr int kOffMisc = kOffNewShare + kMaxNew * 4;  // odd new values, failure
  static constexpr int kOffDyn = kOffMisc + 16;
  static constexpr int kKnLd = HD * 2 + 16;            // bytes of a new key's row
  static_assert(kWarps * kRows * kXld * 4 <= kRing, "the merge fits the ring");
  static_assert(kOffVis % 8 == 0 && kOffBar % 8 == 0 && kOffNewKv % 8 == 0 && kOffDyn % 16 == 0, "alignment");
  // the query rows as they come; new keys and values of up to n tokens, and as
  // they come; the angles of npos positions
  static int bytes(int n, int npos) {
    const int pad = (n + 15) & ~15;
    return kOffDyn + kRows * HD * 2 + pad * kKnLd + pad / 2 * HD * 4 + 2 * n * HD * 2 + npos * (HD / 2) * 8;
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D += A (16 x 16, row) B (16 x 8, col), f16 with fp32 sums.
__device__ __forceinline__ void mma_f16(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// N 32-bit words (2 or 4) of shared memory.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *w) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x; w[1] = v.y;
  }
}

__device__ __forceinline__ uint4 mul4(uint4 h, uint32_t s) {
  return make_uint4(mul_f16x2(h.x, s), mul_f16x2(h.y, s), mul_f16x2(h.z, s), mul_f16x2(h.w, s));
}

template <int V> struct IntC { static constexpr int value = V; };

template <int HD, int NT, int W>
__global__ void __launch_bounds__((Lay<HD, NT, W>::kThreads), (Lay<HD, NT, W>::kCtas))
kv4_mma_kernel(const __grid_constant__ KvqParams a) {
  using L = Lay<HD, NT, W>;
  using R = Record<HD>;
  constexpr int kWarps = L::kWarps, kThreads = L::kThreads;
  constexpr int J = HD / 32;               // words of codes of a lane and key = runs of 8 elements
  constexpr int MT = HD / 16;              // MMA tiles of the head's elements
  extern __shared__ __align__(128) uint8_t sb[];
  float *row_s = reinterpret_cast<float *>(sb + L::kOffRow);
  uint64_t *vis_s = reinterpret_cast<uint64_t *>(sb + L::kOffVis);
  float2 *ml_s = reinterpret_cast<float2 *>(sb + L::kOffMl);
  int *tau_s = reinterpret_cast<int *>(sb + L::kOffTau);
  float2 *new_kv_s = reinterpret_cast<float2 *>(sb + L::kOffNewKv);
  float *new_share_s = reinterpret_cast<float *>(sb + L::kOffNewShare);
  uint32_t *odd_s = reinterpret_cast<uint32_t *>(sb + L::kOffMisc);
  int *flag_s = reinterpret_cast<int *>(sb + L::kOffMisc + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  grid_dep_wait();
  grid_dep_launch();
  const KvqWork w = kvq_work(a);
  if (!w.ok) return;
  const int rows = min(L::kRows, w.M - w.row0);
  const int fresh = w.first ? (w.n + kBlock - 1) / kBlock : 0;          // blocks of new tokens
  const int n_past = max(0, w.k_end - w.k_begin + kBlock - 1) / kBlock;
  const int mine = max(0, n_past - warp + kWarps - 1) / kWarps;         // this warp's of them
  const int32_t *bt = a.block_table + (int64_t)w.b * a.max_pages + w.k_begin / kPage;
  // ------------------------------------------------- this warp's stream of pages
  const uint32_t ring = smem_u32(sb) + warp * L::kStages * L::kStage;
  const uint8_t *ring_p = sb + warp * L::kStages * L::kStage;
  const uint32_t bars = smem_u32(sb + L::kOffBar) + warp * L::kStages * 8;
  if (lane < L::kStages) mbar_init(bars + 8 * lane, 1);
  fence_barrier_init();
  __syncwarp();
  // table entries of the warp's blocks mb .. mb + 15 (two pages each) and of the
  // sixteen blocks after them; -1: no key there
  auto entries = [&](int m) {
    const int p = 2 * (warp + kWarps * (m + (lane >> 1))) + (lane & 1);
    return w.k_begin + p * kPage < w.k_end ? __ldg(bt + p) : -1;
  };
  int mb = 0, cur = entries(0), nxt = entries(16);
  uint32_t gone = 0;                       // of each stage's two pages: bits 2 s and 2 s + 1
  auto issue = [&](int m) {                // copies of block m
    if (m == mb + 16) {
      mb = m;
      cur = nxt;
      nxt = entries(m + 16);
    }
    const int s = m % L::kStages;
    const int page = __shfl_sync(0xffffffffu, cur, 2 * (m - mb) + (lane & 1));
    const bool there = page >= 0 && page < a.num_pages;
    const uint32_t have = __ballot_sync(0xffffffffu, there) & 3u;
    gone = (gone & ~(3u << (2 * s))) | ((have ^ 3u) << (2 * s));
    if (lane == 0) mbar_arrive_expect_tx(bars + 8 * s, __popc(have) * L::kRec);
    __syncwarp();
    if (lane < 2) {
      if (there)
        bulk_load(ring + s * L::kStage + lane * L::kRec, a.k_cache + ((int64_t)page * a.Hkv + w.kvh) * L::kRec, L::kRec,
                  bars + 8 * s);
      else if (w.k_begin + (2 * (warp + kWarps * m) + lane) * kPage < w.k_end)
        raise_status(a.status, kStatusBadInput);
    }
  };
  int issued = 0;
  for (; issued < min(mine, L::kStages); ++issued) issue(issued);
  // ------------------------------------------------------------------ set-up
  const int n_pad = (w.n + 15) & ~15;
  __nv_bfloat16 *q_raw = reinterpret_cast<__nv_bfloat16 *>(sb + L::kOffDyn), *k_raw = q_raw + L::kRows * HD;
  __nv_bfloat16 *v_raw = k_raw + w.n * HD;
  uint8_t *kn = reinterpret_cast<uint8_t *>(v_raw + w.n * HD);         // [n_pad][kKnLd], f16
  uint8_t *vn = kn + n_pad * L::kKnLd;                 // [n_pad / 2][HD] pairs of tokens, f16
  float2 *cs = reinterpret_cast<float2 *>(vn + n_pad / 2 * HD * 4);
  const int64_t t0 = (int64_t)a.per * w.c0;            // first new token's row
  {
    constexpr int CH = HD / 8;                         // 16-byte chunks of a row
    const __nv_bfloat16 *qg = (const __nv_bfloat16 *)a.q + t0 * a.q_row + w.kvh * a.G * HD;
    for (int e = threadIdx.x; e < L::kRows * CH; e += kThreads) {
      const int r = e / CH, row = w.row0 + r, tok = div_by(row, a.by_G);
      const bool take = r < rows;
      copy16_async(smem_u32(q_raw + e * 8), take ? qg + tok * a.q_row + (row - tok * a.G) * HD + e % CH * 8 : (const void *)a.q, take);
    }
    if (fresh) {
      const __nv_bfloat16 *kg = (const __nv_bfloat16 *)a.k_new + t0 * a.k_row + w.kvh * HD;
      const __nv_bfloat16 *vg = (const __nv_bfloat16 *)a.v_new + t0 * a.v_row + w.kvh * HD;
      for (int e = threadIdx.x; e < w.n * CH; e += kThreads) {
        const int j = e / CH, c = e % CH * 8;
        copy16_async(smem_u32(k_raw + e * 8), kg + j * a.k_row + c, true);
        copy16_async(smem_u32(v_raw + e * 8), vg + j * a.v_row + c, true);
      }
    }
  }
  const int npos = a.order == SIMSD_ORDER_PAIRED ? w.B : a.order == SIMSD_ORDER_NODES ? a.node_size : w.n;
  if (threadIdx.x < 2) odd_s[threadIdx.x] = 0u;
  if (threadIdx.x == 0) *flag_s = 0;
  for (int e = threadIdx.x; e < npos * (HD / 2); e += kThreads) {
    const int d = e % (HD / 2);
    cs[e - d + angle_at(d)] =
        d < a.plan.half ? rope_plan_cs(plan_by_lane(a.plan), d, w.P + e / (HD / 2)) : make_float2(1.f, 0.f);
  }
  if (a.order == SIMSD_ORDER_PAIRED && threadIdx.x < w.B) tau_s[threadIdx.x] = __ldg(a.tau + w.c0 + threadIdx.x);
  copy_async_wait_all();
  __syncthreads();
  constexpr int PL = HD / 16;                          // lanes of a row
  const int n_q = L::kRows * PL, n_all = n_q + (fresh ? n_pad * PL : 0);   // (both whole warps)
#pragma unroll 1
  for (int e = threadIdx.x; e < n_all; e += kThreads) {
    const bool query = e < n_q;
    const int r = (query ? e : e - n_q) / PL, c = e % PL;
    const bool real = query ? r < rows : r < w.n;
    const int tok = !real ? 0 : query ? div_by(w.row0 + r, a.by_G) : r;
    int c0, c1;
    float x[16], amax = 0.f, nan = 0.f;                // (query rows that do not exist are zeros)
    rotate16(a.plan, cs + kvq_offset(a, w.B, tok) * (HD / 2), query ? q_raw + r * HD : k_raw + tok * HD, c, c0, c1, x);
#pragma unroll
    for (int i = 0; i < 16; ++i) {                     // (a NaN is not the maximum)
      nan = fmaf(x[i], 0.f, nan);
      amax = fmaxf(amax, fabsf(x[i]));
    }
#pragma unroll
    for (int m = PL / 2; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    // a NaN or an infinity: the row's, or the key's, scores become NaN
    const uint32_t odds = (__ballot_sync(0xffffffffu, nan != 0.f) >> (lane & ~(PL - 1))) & ((1u << PL) - 1u);
    const int ex = scale_exponent(amax, -100, 119);
    const float down = pow2i(-ex);
    if (c == 0) {
      const float up = odds != 0u ? __uint_as_float(0x7fc00000u) : pow2i(ex);
      if (query) row_s[r] = real ? a.scale * up : 0.f;
      else if (real) new_kv_s[r].x = up;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float *y = x + 8 * i;
      const uint4 h = make_uint4(pack_f16x2(y[0] * down, y[1] * down), pack_f16x2(y[2] * down, y[3] * down),
                                 pack_f16x2(y[4] * down, y[5] * down), pack_f16x2(y[6] * down, y[7] * down));
      const int k = i ? c1 : c0;
      uint8_t *dst = query ? sb + L::kOffQ + (((r >> 3) * J + k % J) * 32 + (r & 7) * 4 + k / J) * 16
                           : kn + r * L::kKnLd + k * 16;
      *reinterpret_cast<uint4 *>(dst) = h;
    }
  }
  for (int r = threadIdx.x; r < L::kRows; r += kThreads)
    vis_s[r] = fresh && r < rows ? kvq_visible(a, w.B, tau_s, div_by(w.row0 + r, a.by_G)) : 0ull;
  if (fresh) {                                         // new values, relative to a power of two of each token's
    constexpr int CH = HD / 8;
#pragma unroll 1
    for (int e = threadIdx.x; e < n_pad * CH; e += kThreads) {            // (whole warps)
      const int j = e / CH, c = e % CH;
      float v[8], va = 0.f;
      bool odd = false;
      if (j < w.n) {
        load_vec<__nv_bfloat16, 8>(v_raw + e * 8, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {                    // (an odd one times a weight of 0 would reach every row)
        odd |= !(fabsf(v[i]) < INFINITY);
        v[i] = fabsf(v[i]) < INFINITY ? v[i] : 0.f;
        va = fmaxf(va, fabsf(v[i]));
      }
      if (odd) atomicOr(odd_s + (j >> 5), 1u << (j & 31));
#pragma unroll
      for (int m = CH / 2; m > 0; m >>= 1) va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, m));
      const int ve = value_exponent(va);
      const float down = pow2i(-ve);
      if (c == 0) {
        new_kv_s[j].y = (float)ve;
        new_share_s[j] = kShareLift - (float)ve;
      }
      __half *dst = reinterpret_cast<__half *>(vn) + ((j >> 1) * HD + c * 8) * 2 + (j & 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[2 * i] = __float2half_rn(v[i] * down);
    }
  }
  __syncthreads();
  // --------------------------------------------------------------- the keys
  const uint4 *q_s = reinterpret_cast<const uint4 *>(sb + L::kOffQ) + lane;
  float f[NT][2], m[NT][2], l[NT][2], o[MT][NT][4];    // rows 8 nt + 2 t and the next one
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      f[nt][r] = row_s[8 * nt + 2 * t + r];
      m[nt][r] = -INFINITY;
      l[nt][r] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][nt][c] = 0.f;
  }
  // A block of 32 keys: of the new tokens from j0 on, or of the pages in stage
  // `rec` (lim: keys of it that exist; miss: pages that do not, one bit each).
  auto block = [&](auto newc, int j0, const uint8_t *rec, int lim, uint32_t miss) {
    constexpr bool is_new = decltype(newc)::value != 0;
    float s[2][NT][4];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[p][nt][c] = 0.f;
    uint32_t kw[2][2][J], ks[2][2];                    // [page][key g, g + 8]
    if constexpr (!is_new) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t *base = rec + p * L::kRec;
          load_words<J>(base + (g + 8 * r) * (HD / 2) + t * (HD / 8), kw[p][r]);
          if constexpr (HD == 128) ks[p][r] = *reinterpret_cast<const uint16_t *>(base + R::kKs + (g + 8 * r) * 8 + 2 * t);
          else ks[p][r] = base[R::kKs + (g + 8 * r) * 4 + t];
        }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      uint4 q[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) q[nt] = q_s[(nt * J + j) * 32];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint4 k0, k1;
        if constexpr (is_new) {
          if (j0 + 16 * p >= n_pad) continue;
          const uint8_t *row = kn + (j0 + 16 * p + g) * L::kKnLd + (t * J + j) * 16;
          k0 = *reinterpret_cast<const uint4 *>(row);
          k1 = *reinterpret_cast<const uint4 *>(row + 8 * L::kKnLd);
        } else {
          constexpr int shift = HD == 128 ? 1 : 2;     // words of a scale: 2 (16 elements)
          k0 = mul4(unpack_e2m1x8(kw[p][0][j]), scale4_twice(ks[p][0], j >> shift));
          k1 = mul4(unpack_e2m1x8(kw[p][1][j]), scale4_twice(ks[p][1], j >> shift));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(s[p][nt], k0.x, k1.x, k0.y, k1.y, q[nt].x, q[nt].y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(s[p][nt], k0.z, k1.z, k0.w, k1.w, q[nt].z, q[nt].w);
      }
    }
    // scores t = f s (log2 units); where some keys do not count, here and now
    const bool whole = !is_new && lim >= kBlock && miss == 0u;
    float ff[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) ff[nt][r] = whole ? f[nt][r] : 1.f;
    if (!whole) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = 16 * p + 8 * h + g;
          bool there = !is_new && key < lim && !((miss >> p) & 1u);
          float2 kv = make_float2(1.f, 0.f);
          if (is_new && j0 + key < w.n) kv = new_kv_s[j0 + key];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (is_new) there = j0 + key < w.n && ((vis_s[8 * nt + 2 * t + r] >> (j0 + key)) & 1ull);
              float &x = s[p][nt][2 * h + r];
              x = there ? fmaf(x, f[nt][r] * kv.x, kv.y) : -INFINITY;
            }
        }
    }
    // references move only when a score outgrows them
    constexpr float lift = is_new ? kNewLift : kLift;
    bool grows = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mx = fmaxf(fmaxf(s[0][nt][r], s[0][nt][r + 2]), fmaxf(s[1][nt][r], s[1][nt][r + 2]));
        grows |= mx * ff[nt][r] > m[nt][r] + (kLift + kHeadroom);
      }
    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = fmaxf(fmaxf(s[0][nt][r], s[0][nt][r + 2]), fmaxf(s[1][nt][r], s[1][nt][r + 2])) * ff[nt][r];
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
          if (mx > m[nt][r] + (kLift + kHeadroom)) {
            const float alpha = ex2(m[nt][r] - (mx - lift));          // m = -inf -> 0
            m[nt][r] = mx - lift;
            l[nt][r] *= alpha;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[i][nt][r] *= alpha;
              o[i][nt][r + 2] *= alpha;
            }
          }
        }
    }
    // weights 2^(t - m) as f16 operands (keys down, rows across -> transposed)
    uint32_t pw[2][NT][2];
    float share[2][2];
    if (is_new) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = j0 + 16 * p + 8 * h + g;
          share[p][h] = key < w.n ? new_share_s[key] : 0.f;
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mu[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) mu[r] = m[nt][r] == -INFINITY ? 0.f : m[nt][r];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float e0 = ex2(fmaf(s[p][nt][2 * h], ff[nt][0], -mu[0])), e1 = ex2(fmaf(s[p][nt][2 * h + 1], ff[nt][1], -mu[1]));
          if (is_new) {
            l[nt][0] = fmaf(ex2(s[p][nt][2 * h] - mu[0] + share[p][h]), kShareUnlift, l[nt][0]);
            l[nt][1] = fmaf(ex2(s[p][nt][2 * h + 1] - mu[1] + share[p][h]), kShareUnlift, l[nt][1]);
          } else {
            l[nt][0] += e0;
            l[nt][1] += e1;
          }
          pw[p][nt][h] = transpose8(pack_f16x2(e0, e1));
        }
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (is_new && j0 + 16 * p >= n_pad) continue;
      uint32_t va[J], vb[J], sa = 0u, sc = 0u;         // pairs t and t + 4
      const uint8_t *base = rec + p * L::kRec;
      if constexpr (!is_new) {
        const uint8_t *v = base + R::kV + (HD == 128 ? (g >> 1) * 256 + (g & 1) * 16 : (g >> 2) * 256 + (g & 3) * 8) + t * 32;
        load_words<J>(v, va);
        load_words<J>(v + 128, vb);
        const uint8_t *vs = base + R::vs_at(t, HD == 128 ? g : g >> 1);
        sa = scale4_pair(*reinterpret_cast<const uint16_t *>(vs));
        sc = scale4_pair(*reinterpret_cast<const uint16_t *>(vs + 4 * (HD / 8)));
        if (!whole) {                                  // no key, no value: not even a NaN
          const int k = 16 * p + 2 * t;
          const bool none = (miss >> p) & 1u;
          sa &= (!none && k < lim ? 0xffffu : 0u) | (!none && k + 1 < lim ? 0xffff0000u : 0u);
          sc &= (!none && k + 8 < lim ? 0xffffu : 0u) | (!none && k + 9 < lim ? 0xffff0000u : 0u);
        }
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {                    // four elements: two tiles
        uint4 x, y;
        if constexpr (is_new) {
          const uint8_t *v = vn + (((j0 + 16 * p) / 2 + t) * HD + g * (HD / 8) + 4 * j) * 4;
          x = *reinterpret_cast<const uint4 *>(v);
          y = *reinterpret_cast<const uint4 *>(v + 4 * HD * 4);
        } else {
          x = mul4(unpack_e2m1x8(va[j]), sa);
          y = mul4(unpack_e2m1x8(vb[j]), sc);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(o[2 * j][nt], x.x, x.y, y.x, y.y, pw[p][nt][0], pw[p][nt][1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(o[2 * j + 1][nt], x.z, x.w, y.z, y.w, pw[p][nt][0], pw[p][nt][1]);
      }
    }
  };
  if (kWarps - 1 - warp < fresh) block(IntC<1>{}, kBlock * (kWarps - 1 - warp), nullptr, 0, 0u);
  bool ok = true;
  int done = 0;
#pragma unroll 1
  for (; done < mine; ++done) {
    const int s = done % L::kStages;
    ok = mbar_wait_warp(bars + 8 * s, (done / L::kStages) & 1, a.polls);
    if (!ok) break;
    block(IntC<0>{}, 0, ring_p + s * L::kStage, w.k_end - w.k_begin - (warp + kWarps * done) * kBlock, (gone >> (2 * s)) & 3u);
    __syncwarp();                                      // the stage is read
    if (issued < mine) {
      issue(issued);
      ++issued;
    }
  }
  if (!ok) {                                           // copies in flight land before the CTA can exit
    if (lane == 0) {
      raise_status(a.status, kStatusTimeout);
      atomicExch(flag_s, 1);
    }
    for (; done < issued; ++done) (void)mbar_wait_warp(bars + 8 * (done % L::kStages), (done / L::kStages) & 1);
  }
  // ------------------------------------------------------------------ merge
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) l[nt][r] += __shfl_xor_sync(0xffffffffu, l[nt][r], k);
      if (g == 0) ml_s[warp * L::kRows + 8 * nt + 2 * t + r] = make_float2(m[nt][r], l[nt][r]);
    }
  __syncthreads();                                     // rings are idle
  const bool failed = *(volatile int *)flag_s != 0;
  const uint64_t odd = (uint64_t)odd_s[1] << 32 | odd_s[0];
  float *part = reinterpret_cast<float *>(sb);         // [warps][rows][kXld]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml_s[k * L::kRows + 8 * nt + 2 * t + r].x);
      f[nt][r] = m[nt][r] == -INFINITY ? 0.f : ex2_low(m[nt][r] - top);   // (below fp32's normal range too)
    }
#pragma unroll
  for (int q = 0; q < MT / 4; ++q) {                   // 8 of a lane's elements at a time
    if (q > 0) __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float *dst = part + (warp * L::kRows + 8 * nt + 2 * t + r) * L::kXld + 8 * g;
        const float c = f[nt][r];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float *x = o[4 * q + 2 * i][nt], *y = o[4 * q + 2 * i + 1][nt];
          *reinterpret_cast<float4 *>(dst + 4 * i) = make_float4(x[r] * c, x[r + 2] * c, y[r] * c, y[r + 2] * c);
        }
      }
    __syncthreads();
    for (int e = threadIdx.x; e < rows * 8; e += kThreads) {
      const int r = e >> 3, ge = e & 7;
      float top = -INFINITY, sum = 0.f, v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml_s[k * L::kRows + r].x);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 ml = ml_s[k * L::kRows + r];
        sum = fmaf(ml.x == -INFINITY && ml.y == 0.f ? 0.f : ex2_low(ml.x - (top == -INFINITY ? 0.f : top)), ml.y, sum);
        const float4 *src = reinterpret_cast<const float4 *>(part + (k * L::kRows + r) * L::kXld + 8 * ge);
        const float4 x = src[0], y = src[1];
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
      }
      if (odd != 0ull && (vis_s[r] & odd) != 0ull) sum = __uint_as_float(0x7fc00000u);
      if (failed) continue;
      const int grow = w.row0 + r, tok = div_by(grow, a.by_G), col = ge * (HD / 8) + 8 * q;
      const int64_t orow = (t0 + tok) * a.Hq + w.kvh * a.G + grow - tok * a.G;
      if (w.n_splits == 1) {
        const float c = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= c;
        store_vec<__nv_bfloat16, 8>((__nv_bfloat16 *)a.out + orow * HD + col, v);
      } else {
        const int64_t prow = (int64_t)w.split * a.T * a.Hq + orow;
        store_vec<float, 8>(a.o_part + prow * HD + col, v);
        if (col == 0) a.ml_part[prow] = make_float2(top, sum);
      }
    }
  }
}

template <int HD, int NT, int W>
cudaError_t launch_nt(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a, cudaStream_t stream) {
  using L = Lay<HD, NT, W>;
  auto kern = kv4_mma_kernel<HD, NT, W>;
  static std::atomic<uint64_t> configured{0};   // one bit per device
  const int dev = current_device();
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0;
  if (!bit || !(configured.load() & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes(kMaxNew, kMaxNew));
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  const int n = p.per * d->B_max, npos = d->order == SIMSD_ORDER_NODES ? d->node_size : d->B_max;
  return launch_pdl(kern, dim3((unsigned)p.grid), dim3(L::kThreads), L::bytes(n, npos), stream, a);
}

template <int HD>
cudaError_t launch_hd(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a, cudaStream_t stream) {
  if (p.rows_per_tile == 16) return launch_nt<HD, 2, 6>(d, p, a, stream);
  if (p.rows_per_tile != 8) return cudaErrorInvalidValue;      // no kernel of that tile
  return p.warps == 4 ? launch_nt<HD, 1, 4>(d, p, a, stream) : launch_nt<HD, 1, 8>(d, p, a, stream);
}

}  // namespace

int kv4_rows_per_tile(int64_t max_rows) { return max_rows <= 8 ? 8 : max_rows <= kFewRows ? kFewRows : 128; }

cudaError_t launch_kv4_mma(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a, cudaStream_t stream) {
  return d->head_dim == 128 ? launch_hd<128>(d, p, a, stream) : launch_hd<64>(d, p, a, stream);
}

}  // namespace simsd
