// kvq_attn_tc.cu -- simsd_kvq_verify for bf16 data on the tensor cores.
//
// Scores of prompt keys come from the cache's e4m3 codes as they lie: a query
// row, scaled by a power of two to the codes' range, is split into hi =
// e4m3(q) and lo = e4m3(q - hi) (together 2^-8 of a value, a bf16 rounding),
// and S = hi K^T + lo K^T accumulates in fp32 (kind::f8f6f4, twice the bf16
// rate, so two products cost what one in bf16 does and no key is decoded).
// The page's key scale multiplies the score in the softmax.  The weights
// cannot be split like that (their range is too wide for e4m3), so four warps
// decode the value tiles to bf16, scale included (a multiply by a power of
// two), and O += P V runs in bf16.  The new tokens are a block of their own
// ahead of the prompt: keys rotated here, S from bf16 q and k.
//
// One CTA per (key split, KV head x 128-row tile, sequence); rows stack new
// tokens x heads of the group, so a cache byte is read once for all of them.
// HBM bounds it: 32 KB per 128-key block against ~1000 tensor-core cycles.
//   warp 0      keys: one 2 KB TMA box per page, swizzled for the MMA
//   warp 6      values: one 2 KB bulk copy per page
//   warp 1      TMEM owner, one lane issues every MMA as its inputs are ready
//   warps 2-5   softmax, one thread per row; rows of tiles of at most 64 rows
//               are replicated and the copies split each block's keys
//   warps 7-10  the new tokens' keys and values, then value tiles to bf16
// Every wait is bounded (status bit, drain, return).
#include <cuda.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "kvq.cuh"
#include "kvq_attn.cuh"
#include "tc.cuh"
#include "vec.cuh"

namespace simsd {
namespace {

constexpr int kRows = 128;           // query rows per CTA: the MMA's M
constexpr int kKeys = 128;           // keys per block
static_assert(kKeys == kBlockKeys, "split chunks are whole blocks");
constexpr int kStages = 4;
constexpr int kPagesPerBlock = kKeys / kPage;
constexpr int kVWarp = 6, kDecodeWarp = 7, kWarps = 11;
constexpr int kThreads = kWarps * 32;
constexpr int kSoftmax = 4 * 32, kDecode = 4 * 32;
constexpr float kHeadroom = 8.f;     // log2 units a row max may grow before O is rescaled
constexpr uint32_t kColS = 0;        // two score / weight tiles: columns 0 and kKeys
constexpr uint32_t kColO = 2 * kKeys;

enum { kBarKFull = 0, kBarVFull = kBarKFull + kStages, kBarKEmpty = kBarVFull + kStages,
       kBarVEmpty = kBarKEmpty + kStages, kBarSFull = kBarVEmpty + kStages,
       kBarPFull = kBarSFull + 2, kBarPvDone = kBarPFull + 2, kBarVbFull = kBarPvDone + 2,
       kBarQReady = kBarVbFull + 2, kBarKnReady, kNumBars };

template <int HD>
struct Smem {
  static constexpr int kCodes = kKeys * HD;                 // K or V codes of a block
  static constexpr int kStage = 2 * kCodes;
  static constexpr int kHalf = kKeys * 128;                 // 128 rows x 64 bf16 columns
  static constexpr int kVb = (HD / 64) * kHalf;             // decoded value tile
  static constexpr int kKnHalf = kMaxNew * 128;
  static constexpr int kOffRing = 0;
  static constexpr int kOffVb = kOffRing + kStages * kStage;   // [2]; [1] holds the angles first
  static constexpr int kOffKn = kOffVb + 2 * kVb;           // rotated new keys, bf16
  static constexpr int kOffBar = kOffKn + (HD / 64) * kKnHalf;
  static constexpr int kOffTau = kOffBar + kNumBars * 8;
  static constexpr int kOffMisc = kOffTau + kMaxB * 4;      // tmem address, error flag
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;              // 1024-byte alignment slack
  static constexpr uint32_t kColQb = kColO + HD;            // q as bf16: hd / 2 columns
  static constexpr uint32_t kColQ8 = kColQb + HD / 2;       // q hi and lo: hd / 4 columns each
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kColQ8 + HD / 2 <= kTmemCols, "TMEM budget");
  static_assert(4 * 32 * (HD + 4) * 4 <= kStages * kStage, "epilogue exchange fits the ring");
  static_assert(kMaxNew * (HD / 2) * 8 <= kVb, "angles fit the second value tile");
};

__device__ __forceinline__ uint32_t swz(int row, int chunk) {
  // byte offset of 16-byte chunk `chunk` (0..7) of `row` in a 128-byte
  // swizzled tile whose base is 1024-byte aligned
  return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
}

// 2^x on the MUFU (approximate; subnormal results flush to zero).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int V> struct IntC { static constexpr int value = V; };

__device__ __forceinline__ uint32_t word4(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ void named_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

__device__ __forceinline__ uint64_t shift_right(uint64_t x, int s) { return s >= 64 ? 0ull : x >> s; }

// Element i (a compile-time constant after unrolling) of a bf16 row held in
// 16-byte vectors.
template <int HD>
__device__ __forceinline__ float row_elem(const uint4 *qv, int i) {
  const uint32_t w = word4(qv[i >> 3], (i >> 1) & 3);
  return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}

// Four e4m3 codes to two bf16 pairs, times a power of two: a code's exponent
// and mantissa bits, moved to a bf16's, are its value times 2^-120 (subnormal
// codes become subnormal bf16 values), so `mul` is 2^(120 + E) twice.
__device__ __forceinline__ uint32_t decode2(uint32_t w, uint32_t sel, __nv_bfloat162 mul) {
  uint32_t x;                                    // each byte sign-extended to 16 bits
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(x) : "r"(w), "r"(sel));
  x = (x << 4) & 0x87f087f0u;
  const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&x), mul);
  return *reinterpret_cast<const uint32_t *>(&y);
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
kvq_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ KvqParams a) {
  using L = Smem<HD>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sb = smem_raw + (base - raw);
  auto bar = [&](int i) { return base + L::kOffBar + 8u * i; };
  int *tau_s = reinterpret_cast<int *>(sb + L::kOffTau);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sb + L::kOffMisc);
  int *flag_s = reinterpret_cast<int *>(sb + L::kOffMisc + 4);
  grid_dep_launch();                         // the split merge may be scheduled
  const KvqWork w = kvq_work(a);
  if (!w.ok) return;                         // uniform: nothing to do here
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int fresh = w.first ? 1 : 0;         // block 0 is the new tokens'
  const int n_past = max(0, w.k_end - w.k_begin + kKeys - 1) / kKeys;   // prompt blocks
  const int n_blocks = fresh + n_past;
  const int n_pad = (w.n + 15) & ~15;
  // copies of the tile's rows across the four TMEM lane quadrants, and the
  // softmax warps that own real rows
  const int n_groups = min(4, (w.M - w.row0 + 31) / 32);
  const int R = n_groups == 1 ? 4 : n_groups == 2 ? 2 : 1;
  const int n_valid = R > 1 ? 4 : n_groups;
  const int32_t *bt = a.block_table + (int64_t)w.b * a.max_pages;
  const int64_t t0 = (int64_t)a.per * w.c0;  // first new token's row
  // page id of page `lane` of prompt block j; -1: none (or not in the cache)
  auto block_page = [&](int j) {
    if (j >= n_past || lane >= kPagesPerBlock) return -1;
    const int key = w.k_begin + j * kKeys + lane * kPage;
    if (key >= w.k_end) return -1;
    const int page = __ldg(bt + key / kPage);
    if (page >= 0 && page < a.num_pages) return page;
    raise_status(a.status, kStatusBadInput);
    return -1;
  };
  int pages[kStages];
  const bool softmax_warp = warp >= 2 && warp < 6;
  if (warp == 0 || warp == kVWarp) {
    if (warp == 0 && lane == 0) prefetch_tmap(&tmK);
#pragma unroll
    for (int d = 0; d < kStages; ++d) pages[d] = block_page(d);
  }
  uint4 qv[HD / 8];
  if (softmax_warp) {
    const int r = w.row0 + 32 * ((warp & 3) % (4 / R)) + lane;
    if (r < w.M) {
      const uint4 *src = reinterpret_cast<const uint4 *>(
          (const __nv_bfloat16 *)a.q + (t0 + r / a.G) * a.q_row + (w.kvh * a.G + r % a.G) * HD);
#pragma unroll
      for (int e = 0; e < HD / 8; ++e) qv[e] = __ldg(src + e);
    } else {
#pragma unroll
      for (int e = 0; e < HD / 8; ++e) qv[e] = make_uint4(0, 0, 0, 0);
    }
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(kBarKFull + i), 1);
      mbar_init(bar(kBarVFull + i), 1);
      mbar_init(bar(kBarKEmpty + i), 1);
      mbar_init(bar(kBarVEmpty + i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarPFull + i), n_valid);
      mbar_init(bar(kBarPvDone + i), 1);
      mbar_init(bar(kBarVbFull + i), 4);
    }
    mbar_init(bar(kBarQReady), 4);
    mbar_init(bar(kBarKnReady), 4);
    *flag_s = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tc::alloc(smem_u32(tmem_slot), L::kTmemCols);
    tc::relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  int issued = 0;                            // producers: blocks whose loads were started
  float2 *cs_s = reinterpret_cast<float2 *>(sb + L::kOffVb + L::kVb);   // [kMaxNew][HD / 2]
  auto give_up = [&]() { raise_status(a.status, kStatusTimeout); atomicOr(flag_s, 1); };
  // angles of the new tokens' positions (identity past the rotated part),
  // by the softmax and decode warps together
  auto angles = [&](int t) {
    const int npos = a.order == SIMSD_ORDER_PAIRED ? w.B : a.order == SIMSD_ORDER_NODES ? a.node_size : w.n;
    for (int e = t; e < npos * (HD / 2); e += kSoftmax + kDecode) {
      const int d = e % (HD / 2);
      cs_s[e] = d < a.plan.half ? rope_plan_cs(a.plan, d, w.P + e / (HD / 2)) : make_float2(1.f, 0.f);
    }
    if (a.order == SIMSD_ORDER_PAIRED && t < w.B) tau_s[t] = __ldg(a.tau + w.c0 + t);
    named_sync(1, kSoftmax + kDecode);
  };

  if (warp == 0 || warp == kVWarp) {
    // --------------------------------------------------------- producers
    const bool kside = warp == 0;
    const int full0 = kside ? kBarKFull : kBarVFull, empty0 = kside ? kBarKEmpty : kBarVEmpty;
    bool ok = true;
    for (int j0 = 0; ok && j0 < n_past; j0 += kStages) {
#pragma unroll
      for (int s = 0; s < kStages; ++s) {    // s: stage of block j
        const int j = j0 + s;
        if (j >= n_past) break;
        const int page = pages[s];
        const int n_pages = __popc(__ballot_sync(0xffffffffu, page >= 0));
        if (j >= kStages && !mbar_wait_warp(bar(empty0 + s), ((j / kStages) - 1) & 1, a.polls)) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(bar(full0 + s), n_pages * kPage * HD);
        __syncwarp();
        if (page >= 0) {
          const uint32_t dst = base + L::kOffRing + s * L::kStage + (kside ? 0 : L::kCodes) + lane * kPage * HD;
          if (kside)
            tma_load_4d(dst, &tmK, bar(full0 + s), 0, 0, w.kvh, page);
          else
            bulk_load(dst, a.v_cache + ((int64_t)page * a.Hkv + w.kvh) * kPage * HD, kPage * HD, bar(full0 + s));
        }
        issued = j + 1;
        pages[s] = block_page(j + kStages);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS8 = tc::idesc_e4m3(kRows, kKeys);
      constexpr uint32_t idSn = tc::idesc_bf16(kRows, kMaxNew, 0);
      constexpr uint32_t idO = tc::idesc_bf16(kRows, HD, 1);
      bool ok = mbar_wait(bar(kBarQReady), 0, a.polls);
      int ns = 0, np = 0;
      uint64_t idle = 0;
      while (ok && np < n_blocks) {
        bool progressed = false;
        if (ns < n_blocks) {
          const int tb = ns & 1, jp = ns - fresh, s = jp & (kStages - 1);
          const bool is_new = jp < 0;
          if ((is_new ? mbar_test(bar(kBarKnReady), 0) : mbar_test(bar(kBarKFull + s), (jp / kStages) & 1)) &&
              (ns < 2 || mbar_test(bar(kBarPvDone + tb), ((ns >> 1) - 1) & 1))) {
            tc::fence_after_sync();
            const uint32_t tS = tmem + kColS + tb * kKeys;
            if (is_new) {
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk)
                tc::mma_bf16_ts(tS, tmem + L::kColQb + kk * 8,
                                tc::smem_desc_sw128(base + L::kOffKn + (kk >> 2) * L::kKnHalf + (kk & 3) * 32, 16, 1024),
                                idSn, kk > 0);
            } else {
              const uint32_t kt = base + L::kOffRing + s * L::kStage;
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < HD / 32; ++kk)
                  tc::mma_e4m3_ts(tS, tmem + L::kColQ8 + part * (HD / 4) + kk * 8,
                                  HD == 128 ? tc::smem_desc_sw128(kt + kk * 32, 16, 1024)
                                            : tc::smem_desc_sw64(kt + kk * 32, 16, 512),
                                  idS8, part > 0 || kk > 0);
            }
            tc::commit(bar(kBarSFull + tb));
            if (!is_new) tc::commit(bar(kBarKEmpty + s));
            ++ns;
            progressed = true;
          }
        }
        if (np < ns) {
          const int tb = np & 1;
          if (mbar_test(bar(kBarPFull + tb), (np >> 1) & 1) && mbar_test(bar(kBarVbFull + tb), (np >> 1) & 1)) {
            tc::fence_after_sync();
            const int jp = np - fresh;
            const int depth = jp < 0 ? n_pad : min(kKeys, (w.k_end - w.k_begin - jp * kKeys + 15) & ~15);
            const uint32_t vt = base + L::kOffVb + tb * L::kVb;
            for (int kk = 0; kk < depth / 16; ++kk)
              tc::mma_bf16_ts(tmem + kColO, tmem + kColS + tb * kKeys + kk * 8,
                              tc::smem_desc_sw128(vt + kk * 2048, L::kHalf, 1024), idO, (np > 0 || kk > 0));
            tc::commit(bar(kBarPvDone + tb));
            ++np;
            progressed = true;
          }
        }
        if (progressed) {
          idle = 0;
        } else if (++idle > ((uint64_t)a.polls << 4)) {  // bounded: give up, flag, drain
          ok = false;
        } else if (idle > 8) {
          __nanosleep(32);                   // leave the issue slots to the other warps
        }
      }
      if (!ok) give_up();
    }
  } else if (warp >= kDecodeWarp) {
    // ------------------------------------------------------------- decode
    const int dw = warp - kDecodeWarp, t = threadIdx.x - kDecodeWarp * 32;
    angles(kSoftmax + t);
    if (fresh) {
      // the new tokens' keys, rotated, and their values as they are (zeros up
      // to the MMA's depth)
      constexpr int CH = HD / 8;
      const __nv_bfloat16 *ks = (const __nv_bfloat16 *)a.k_new + t0 * a.k_row + w.kvh * HD;
      const __nv_bfloat16 *vs = (const __nv_bfloat16 *)a.v_new + t0 * a.v_row + w.kvh * HD;
      const RopePlan &p = a.plan;
      for (int e = t; e < n_pad * CH; e += kDecode) {
        const int j = e / CH, c = e % CH, e0 = c * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
        if (j < w.n) {
          v = __ldg(reinterpret_cast<const uint4 *>(vs + j * a.v_row + e0));
          const __nv_bfloat16 *row = ks + j * a.k_row;
          const float2 *cs = cs_s + kvq_offset(a, w.B, j) * (HD / 2);
          load_vec<__nv_bfloat16, 8>(row + e0, x);
          if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float2 z = cs[(e0 + i) >> 1];
              const float x1 = x[i], x2 = x[i + 1];
              x[i] = x1 * z.x - x2 * z.y;
              x[i + 1] = x2 * z.x + x1 * z.y;
            }
          } else if (p.half % 8 == 0) {
            if (e0 < 2 * p.half) {
              const bool low = e0 < p.half;
              float y[8];
              load_vec<__nv_bfloat16, 8>(row + (low ? e0 + p.half : e0 - p.half), y);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 z = cs[low ? e0 + i : e0 + i - p.half];
                x[i] = low ? x[i] * z.x - y[i] * z.y : x[i] * z.x + y[i] * z.y;
              }
            }
          } else {
            for (int i = 0; i < 8; ++i) {
              const int d = e0 + i;
              if (d >= 2 * p.half) break;
              const bool low = d < p.half;
              const float y = __bfloat162float(row[low ? d + p.half : d - p.half]);
              const float2 z = cs[low ? d : d - p.half];
              x[i] = low ? x[i] * z.x - y * z.y : x[i] * z.x + y * z.y;
            }
          }
        }
        *reinterpret_cast<uint4 *>(sb + L::kOffVb + (c >> 3) * L::kHalf + swz(j, c & 7)) = v;
        *reinterpret_cast<uint4 *>(sb + L::kOffKn + (c >> 3) * L::kKnHalf + swz(j, c & 7)) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      }
      fence_proxy_async_smem();
      named_sync(2, kDecode);                // every decode warp is done with the angles
      if (lane == 0) {
        mbar_arrive(bar(kBarKnReady));
        mbar_arrive(bar(kBarVbFull));
      }
    }
    // value tiles: this warp's rows are pages 2 dw and 2 dw + 1 of a block;
    // lanes 0 and 1 keep those pages' scales, requested a block ahead
    // (their page ids two)
    auto page_of = [&](int jp) {
      const int key = w.k_begin + jp * kKeys + (2 * dw + lane) * kPage;
      if (lane >= 2 || jp >= n_past || key >= w.k_end) return -1;
      const int page = __ldg(bt + key / kPage);
      return page < a.num_pages ? page : -1;
    };
    auto scale_of = [&](int page) -> uint32_t {   // multiplier 2^(120 + E) as two bf16, 0: no page
      if (page < 0) return 0u;
      const uint32_t byte = __ldg(a.v_scale + (int64_t)page * a.Hkv + w.kvh);
      const uint32_t h = byte == kScaleNan ? 0x7fc0u : min(byte + 120u, 254u) << 7;
      return h | h << 16;
    };
    uint32_t next = scale_of(page_of(0));
    int page1 = page_of(1);
    bool ok = true;
    for (int jp = 0; jp < n_past; ++jp) {
      const int j = jp + fresh, tb = j & 1, s = jp & (kStages - 1);
      const uint32_t mine = next;
      next = scale_of(page1);
      page1 = page_of(jp + 2);
      if (j == 1 && !mbar_wait_warp(bar(kBarQReady), 0, a.polls)) { ok = false; break; }   // angles are read
      if (!mbar_wait_warp(bar(kBarVFull + s), (jp / kStages) & 1, a.polls) ||
          (j >= 2 && !mbar_wait_warp(bar(kBarPvDone + tb), ((j >> 1) - 1) & 1, a.polls))) { ok = false; break; }
      const int valid = w.k_end - w.k_begin - jp * kKeys;    // rows from here on hold no key
      const uint8_t *src = sb + L::kOffRing + s * L::kStage + L::kCodes;
      uint8_t *dst = sb + L::kOffVb + tb * L::kVb;
      constexpr int C = HD / 16, RPI = 32 / C;               // 16-byte chunks of a row; rows an iteration
#pragma unroll
      for (int i = 0; i < 32 / RPI; ++i) {
        const int row = 32 * dw + i * RPI + lane / C, c = lane % C;
        const uint32_t m = __shfl_sync(0xffffffffu, mine, (i * RPI) / kPage);
        const __nv_bfloat162 mul = *reinterpret_cast<const __nv_bfloat162 *>(&m);
        const uint4 x = *reinterpret_cast<const uint4 *>(src + row * HD + c * 16);
        uint4 lo, hi;                                        // selectors: bytes 0, 1 and 2, 3 with their signs
        lo = make_uint4(decode2(x.x, 0x9180u, mul), decode2(x.x, 0xb3a2u, mul),
                        decode2(x.y, 0x9180u, mul), decode2(x.y, 0xb3a2u, mul));
        hi = make_uint4(decode2(x.z, 0x9180u, mul), decode2(x.z, 0xb3a2u, mul),
                        decode2(x.w, 0x9180u, mul), decode2(x.w, 0xb3a2u, mul));
        if (row >= valid) lo = hi = make_uint4(0, 0, 0, 0);
        uint8_t *tile = dst + (c >> 2) * L::kHalf;
        const int ch = 2 * (c & 3);
        // the two 64-column halves store their chunks in opposite order: no bank twice
        const bool flip = c >= 4;
        *reinterpret_cast<uint4 *>(tile + swz(row, flip ? ch + 1 : ch)) = flip ? hi : lo;
        *reinterpret_cast<uint4 *>(tile + swz(row, flip ? ch : ch + 1)) = flip ? lo : hi;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kBarVbFull + tb));
        mbar_arrive(bar(kBarVEmpty + s));
      }
    }
    if (!ok && lane == 0) give_up();
  } else {
    // ------------------------------------------------------------ softmax
    // With at most 64 real rows the tile's rows are replicated across the
    // four TMEM lane quadrants (R = 4 or 2 copies) and the copies split each
    // block's keys; every copy keeps its own reference and writes weights for
    // its keys (zeros elsewhere), and the epilogue merges the copies.
    const int q4 = warp & 3;                 // TMEM lane quadrant of this warp
    const int groups = 4 / R;
    const int g = q4 % groups, kp = q4 / groups;
    const int grow = w.row0 + 32 * g + lane;
    const bool row_valid = grow < w.M;
    const bool warp_valid = w.row0 + 32 * g < w.M;
    const int tok = row_valid ? grow / a.G : 0;
    const uint32_t trow = tmem + ((uint32_t)(32 * q4) << 16);
    // the row's power of two: rotated elements stay below 448 * 2^qe
    float amax = 0.f;
    bool odd = false;                        // a NaN or an infinity: the row's scores become NaN
#pragma unroll
    for (int e = 0; e < HD; ++e) {
      const float x = fabsf(row_elem<HD>(qv, e));
      odd |= !(x < INFINITY);
      amax = fmaxf(amax, x);
    }
    const uint32_t ab = __float_as_uint(amax * a.plan.mul * 1.41422f);
    const int qe = min(max((int)(ab >> 23) - 127 - 8 + ((ab & 0x7fffffu) > 0x600000u ? 1 : 0), -100), 120);
    const float down = pow2i(-qe);
    const float rscale = odd ? __uint_as_float(0x7fc00000u) : a.scale * pow2i(qe);
    angles(threadIdx.x - 64);
    {
      const float2 *cs = cs_s + kvq_offset(a, w.B, tok) * (HD / 2);
      // 32 rotated elements at a time: bf16 for the new tokens' scores, hi
      // and lo codes for the prompt's
      auto emit = [&](int d0, const float *y) {
        uint32_t wb[16], wh[8], wl[8];
#pragma unroll
        for (int i = 0; i < 16; ++i) wb[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y0 = y[4 * i] * down, y1 = y[4 * i + 1] * down, y2 = y[4 * i + 2] * down, y3 = y[4 * i + 3] * down;
          const uint32_t h0 = pack_e4m3x2(y0, y1), h1 = pack_e4m3x2(y2, y3);
          const float2 f0 = unpack_e4m3x2(h0), f1 = unpack_e4m3x2(h1);
          wh[i] = h0 | h1 << 16;
          wl[i] = pack_e4m3x2(y0 - f0.x, y1 - f0.y) | pack_e4m3x2(y2 - f1.x, y3 - f1.y) << 16;
        }
        tc::st16(trow + L::kColQb + d0 / 2, wb);
        tc::st8(trow + L::kColQ8 + d0 / 4, wh);
        tc::st8(trow + L::kColQ8 + HD / 4 + d0 / 4, wl);
      };
      float y[32];
      if (a.plan.interleaved) {
#pragma unroll
        for (int d0 = 0; d0 < HD; d0 += 32) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 z = cs[(d0 + i) >> 1];
            const float x1 = row_elem<HD>(qv, d0 + i), x2 = row_elem<HD>(qv, d0 + i + 1);
            y[i] = x1 * z.x - x2 * z.y;
            y[i + 1] = x2 * z.x + x1 * z.y;
          }
          emit(d0, y);
        }
      } else if (a.plan.half == HD / 2) {
#pragma unroll
        for (int d0 = 0; d0 < HD; d0 += 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int d = d0 + i, dp = d < HD / 2 ? d : d - HD / 2;
            const float2 z = cs[dp];
            const float x1 = row_elem<HD>(qv, dp), x2 = row_elem<HD>(qv, dp + HD / 2);
            y[i] = d < HD / 2 ? x1 * z.x - x2 * z.y : x2 * z.x + x1 * z.y;
          }
          emit(d0, y);
        }
      } else {
        // half pairs of part of the head: a partner's place is not known at
        // compile time, so the row goes through local memory
        uint32_t loc[HD / 2];
#pragma unroll
        for (int i = 0; i < HD / 2; ++i) loc[i] = word4(qv[i >> 2], i & 3);
        auto at = [&](int d) {
          const uint32_t u = loc[d >> 1];
          return __uint_as_float((d & 1) ? (u & 0xffff0000u) : (u << 16));
        };
        const int half = a.plan.half;
#pragma unroll 1
        for (int d0 = 0; d0 < HD; d0 += 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int d = d0 + i;
            const bool low = d < half, turned = d < 2 * half;
            const float2 z = turned ? cs[low ? d : d - half] : make_float2(1.f, 0.f);
            const float x2 = at(turned ? (low ? d + half : d - half) : d);
            y[i] = low ? at(d) * z.x - x2 * z.y : at(d) * z.x + x2 * z.y;
          }
          emit(d0, y);
        }
      }
      tc::wait_st();
      tc::fence_before_sync();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarQReady));
    const uint64_t newvis = fresh ? kvq_visible(a, w.B, tau_s, tok) : 0ull;
    const uint32_t tO = trow + kColO;
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    int j = 0;
    // lane i < 8: key scale of page i of a prompt block (-1: no such page),
    // requested a block ahead (its page id two)
    auto scale_of = [&](int page) {
      return page < 0 ? -1.f : scale_value(__ldg(a.k_scale + (int64_t)page * a.Hkv + w.kvh));
    };
    float next = scale_of(block_page(0));
    int page1 = block_page(1);
    // the key loop, compiled once per copy count
    auto key_loop = [&](auto rc) {
      constexpr int RC = decltype(rc)::value;
      constexpr int KW = kKeys / RC;         // this warp's keys per block
      constexpr int CB = KW < 64 ? KW : 64;  // columns per TMEM round trip
      constexpr int NV = (KW + 63) / 64;
      const int k_lo = kp * KW;
      for (; warp_valid && j < n_blocks; ++j) {
        const int tb = j & 1, jp = j - fresh;
        const bool is_new = jp < 0;
        const uint32_t tS = trow + kColS + tb * kKeys;
        const float page_scale = is_new ? 1.f : next;
        if (!is_new) {
          next = scale_of(page1);
          page1 = block_page(jp + 2);
        }
        // factor of this warp's 16-key groups: row scale x page scale
        const float rs = is_new ? a.scale : rscale;
        float sc[KW / 16];
#pragma unroll
        for (int i = 0; i < KW / 16; ++i) sc[i] = rs * __shfl_sync(0xffffffffu, page_scale, is_new ? 0 : k_lo / 16 + i);
        // keys that count, one bit each (all of a whole block's)
        uint64_t vis[NV];
        bool whole = false;
        if (is_new) {
#pragma unroll
          for (int h = 0; h < NV; ++h) vis[h] = shift_right(newvis, k_lo + 64 * h);
        } else {
          const int valid = w.k_end - w.k_begin - jp * kKeys;
          const uint32_t absent = __ballot_sync(0xffffffffu, lane < kPagesPerBlock && page_scale == -1.f);
          whole = absent == 0;
#pragma unroll
          for (int h = 0; h < NV; ++h) vis[h] = kvq_low_bits(valid - k_lo - 64 * h);
          whole = whole && valid >= kKeys;
          if (!whole) {
#pragma unroll
            for (int i = 0; i < KW / 16; ++i)
              if ((absent >> (k_lo / 16 + i)) & 1u) vis[i / 4] &= ~(0xffffull << (16 * (i % 4)));
          }
        }
        if (!mbar_wait_warp(bar(kBarSFull + tb), (j >> 1) & 1, a.polls)) { ok = false; break; }
        tc::fence_after_sync();
        // pass 1: the row's maximum over this warp's keys
        float mx = -INFINITY;
#pragma unroll
        for (int ck = 0; ck < KW; ck += CB) {
          uint32_t sr[CB];
#pragma unroll
          for (int q = 0; q < CB; q += 32) tc::ld32(tS + k_lo + ck + q, sr + q);
          tc::wait_ld();
          if (whole) {
#pragma unroll
            for (int i = 0; i < CB; i += 16) {
              float t4[4];
#pragma unroll
              for (int c = 0; c < 4; ++c)
                t4[c] = fmaxf(fmaxf(__uint_as_float(sr[i + c]), __uint_as_float(sr[i + c + 4])),
                              fmaxf(__uint_as_float(sr[i + c + 8]), __uint_as_float(sr[i + c + 12])));
              mx = fmaxf(mx, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * sc[(ck + i) / 16]);
            }
          } else {
            const uint64_t vh = vis[ck / 64];
#pragma unroll
            for (int i = 0; i < CB; ++i)
              if ((vh >> i) & 1ull) mx = fmaxf(mx, __uint_as_float(sr[i]) * sc[(ck + i) / 16]);
          }
        }
        // reference maximum: moves only when this block's max outgrows it
        const bool move = row_valid && mx > m_ref + kHeadroom;
        const float m_new = move ? mx : m_ref;
        const float alpha = move ? ex2(m_ref - m_new) : 1.f;     // m_ref = -inf -> 0
        if (j > 0 && __any_sync(0xffffffffu, move)) {
          // rescaling O needs the previous block's P V done
          if (!mbar_wait_warp(bar(kBarPvDone + (tb ^ 1)), ((j - 1) >> 1) & 1, a.polls)) { ok = false; break; }
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            tc::ld32(tO + 32 * c, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::st32(tO + 32 * c, o);
          }
          tc::wait_st();
        }
        l *= alpha;
        m_ref = m_new;
        // pass 2: weights 2^(s - m_ref) as bf16 pairs over the score tile
        // (columns k_lo/2 .. (k_lo + KW)/2), zeros in the other copies' keys
        const float mu = m_ref == -INFINITY ? 0.f : m_ref;
        float rs4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ck = 0; ck < KW; ck += CB) {
          uint32_t sr[CB], pw[CB / 2];
#pragma unroll
          for (int q = 0; q < CB; q += 32) tc::ld32(tS + k_lo + ck + q, sr + q);
          tc::wait_ld();
          const uint64_t vh = vis[ck / 64];
#pragma unroll
          for (int e = 0; e < CB / 2; ++e) {
            const float f = sc[(ck + 2 * e) / 16];
            float x0 = fmaf(__uint_as_float(sr[2 * e]), f, -mu), x1 = fmaf(__uint_as_float(sr[2 * e + 1]), f, -mu);
            if (!whole) {
              x0 = (vh >> (2 * e)) & 1ull ? x0 : -INFINITY;
              x1 = (vh >> (2 * e + 1)) & 1ull ? x1 : -INFINITY;
            }
            const float p0 = ex2(x0), p1 = ex2(x1);
            rs4[e & 3] += p0 + p1;
            pw[e] = pack_bf16x2(p0, p1);
          }
#pragma unroll
          for (int q = 0; q < CB / 2; q += 16) tc::st16(tS + (k_lo + ck) / 2 + q, pw + q);
        }
        if (RC > 1) {
          uint32_t z[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) z[e] = 0u;
#pragma unroll
          for (int c = 0; c < kKeys / 2; c += 16)
            if (c < k_lo / 2 || c >= (k_lo + KW) / 2) tc::st16(tS + c, z);
        }
        tc::wait_st();
        l += (rs4[0] + rs4[1]) + (rs4[2] + rs4[3]);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPFull + tb));
      }
    };
    if (R == 4) key_loop(IntC<4>{});
    else if (R == 2) key_loop(IntC<2>{});
    else key_loop(IntC<1>{});
    if (ok && j > 0 && !mbar_wait_warp(bar(kBarPvDone + ((j - 1) & 1)), ((j - 1) >> 1) & 1, a.polls)) ok = false;
    if (!ok && lane == 0) give_up();
    tc::fence_after_sync();
    // -------------------------------------------------------- epilogue
    const bool failed = !ok || *(volatile int *)flag_s != 0;
    const int64_t orow = (t0 + tok) * a.Hq + w.kvh * a.G + (row_valid ? grow % a.G : 0);
    // columns [c0, c0 + n) of this thread's row: sums v relative to reference
    // mr, weights' sum lt
    auto write_cols = [&](const float *v, int c0, int n, float lt, float mr) {
      if (w.n_splits == 1) {
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        uint4 *dst = reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.out + orow * HD + c0);
        for (int e = 0; e < n / 8; ++e)
          dst[e] = make_uint4(pack_bf16x2(v[8 * e] * inv, v[8 * e + 1] * inv),
                              pack_bf16x2(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                              pack_bf16x2(v[8 * e + 4] * inv, v[8 * e + 5] * inv),
                              pack_bf16x2(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
      } else {
        const int64_t prow = (int64_t)w.split * a.T * a.Hq + orow;
        float4 *dst = reinterpret_cast<float4 *>(a.o_part + prow * HD + c0);
        for (int e = 0; e < n / 4; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        if (c0 == 0) a.ml_part[prow] = make_float2(mr, lt);
      }
    };
    if (R == 1) {
      if (warp_valid) {
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t o[32];
          tc::ld32(tO + 32 * c, o);
          tc::wait_ld();
          if (!row_valid || failed) continue;
          write_cols(reinterpret_cast<const float *>(o), 32 * c, 32, l, m_ref);
        }
      }
    } else {
      // every copy puts its sums and reference in the idle ring; then copy kp
      // merges the R partials of columns [kp * HD/R, ..)
      float *part = reinterpret_cast<float *>(sb + L::kOffRing);   // [R][groups][32][HD + 4]
      float *mine = part + ((kp * groups + g) * 32 + lane) * (HD + 4);
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        tc::ld32(tO + 32 * c, o);
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<float4 *>(mine + 32 * c + 4 * e) =
              make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                          __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
      }
      mine[HD] = l;
      mine[HD + 1] = m_ref;
      named_sync(3, kSoftmax);
      if (row_valid && !failed) {
        const int cw = HD / R, cb = kp * cw;    // 16, 32 or 64 columns
        float mt = -INFINITY;
        for (int c = 0; c < R; ++c) mt = fmaxf(mt, part[((c * groups + g) * 32 + lane) * (HD + 4) + HD + 1]);
        float wc[4], lt = 0.f;
        for (int c = 0; c < R; ++c) {
          const float *pc = part + ((c * groups + g) * 32 + lane) * (HD + 4);
          wc[c] = ex2(pc[HD + 1] - (mt == -INFINITY ? 0.f : mt));   // -inf reference -> 0
          lt += wc[c] * pc[HD];
        }
        for (int q = 0; q < cw; q += 32) {
          const int n = min(32, cw - q);        // a multiple of 16
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0.f;
          for (int c = 0; c < R; ++c) {
            const float *src = part + ((c * groups + g) * 32 + lane) * (HD + 4) + cb + q;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (4 * e >= n) break;
              const float4 p4 = *reinterpret_cast<const float4 *>(src + 4 * e);
              v[4 * e] += wc[c] * p4.x; v[4 * e + 1] += wc[c] * p4.y;
              v[4 * e + 2] += wc[c] * p4.z; v[4 * e + 3] += wc[c] * p4.w;
            }
          }
          write_cols(v, cb + q, n, lt, mt);
        }
      }
    }
  }
  // -------------------------------------------------------------- teardown
  tc::fence_before_sync();
  __syncthreads();
  // after a wait that gave up, the copies still in flight land before the CTA
  // can exit (default limit)
  if ((warp == 0 || warp == kVWarp) && *(volatile int *)flag_s)
    for (int j = max(0, issued - kStages); j < issued; ++j)
      (void)mbar_wait_warp(bar((warp == 0 ? kBarKFull : kBarVFull) + j % kStages), (j / kStages) & 1);
  if (warp == 1) {
    tc::fence_after_sync();
    tc::dealloc(tmem, L::kTmemCols);
  }
}

static_assert(Smem<128>::kAlloc <= 227 * 1024, "shared memory budget");

template <int HD>
cudaError_t launch_tc_hd(const CUtensorMap &mk, const KvqPlan &p, const KvqParams &a, cudaStream_t stream) {
  auto kern = kvq_tc_kernel<HD>;
  const int smem = Smem<HD>::kAlloc;
  static std::atomic<uint64_t> configured{0};   // one bit per device
  const int dev = current_device();
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0;
  if (!bit || !(configured.load() & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  kern<<<p.grid, kThreads, smem, stream>>>(mk, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kvq_tc(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a,
                          cudaStream_t stream) {
  CUtensorMap mk;
  if (!make_cache_map(&mk, const_cast<void *>(d->k_cache), d->num_pages, d->num_kv_heads, d->head_dim, true))
    return cudaErrorInvalidValue;
  return d->head_dim == 128 ? launch_tc_hd<128>(mk, p, a, stream) : launch_tc_hd<64>(mk, p, a, stream);
}

}  // namespace simsd
