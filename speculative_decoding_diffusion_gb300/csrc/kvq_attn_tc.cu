// kvq_attn_tc.cu -- simsd_kvq_verify for bf16 data on the tensor cores.
//
// Scores of prompt keys come from the cache's e4m3 codes as they lie: a query
// row, scaled by a power of two to the codes' range, is split into hi =
// e4m3(q) and lo = e4m3(q - hi) (together within 2^-9 of an element, half of a
// bf16 rounding, or 2^-17 of the row's largest: lo's subnormal codes), and S =
// hi K^T + lo K^T accumulates in fp32 (kind::f8f6f4, twice the bf16 rate, so
// two products cost what one in bf16 does and no key is decoded).
// The page's key scale multiplies the score in the softmax.  The weights
// cannot be split like that (their range is too wide for e4m3), so four warps
// unpack the value codes to f16 (exact) and O += P V runs in f16.  A page's
// value scale 2^ve goes into its keys' weights: with t = s + ve and a row
// reference M over t, p = 2^(t - M + 7) multiplies the codes themselves, and
// the row's sum takes 2^-ve times the sum of a page's weights -- nothing per
// key or value.  M is at most 8 stale, so p <= 2^15 fits f16, whose 11 bits
// keep the error against 64 bits at 1.9e-3 of the result, 1.7e-3 of it the
// output's own rounding (weights rounded to bf16: 2.5e-3).  The new tokens are a block of
// their own ahead of the prompt: keys rotated and split here relative to a power
// of two of each token's, values as f16 relative to another that is the token's
// ve, so that no token's size reaches a row that does not see it.
// One CTA per (key split, KV head x 128-row tile, sequence); rows stack new
// tokens x heads of the group, so a cache byte is read once for all of them.
// A 128-key block is 32 KB, 1410 cycles of an SM's share of the HBM rate, and
// 1024 tensor-core cycles (an MMA of N = 128 takes 64, e4m3 at K = 32 like f16
// at K = 16; issued by one lane of a converged warp, whose addresses stay in
// uniform registers, 33 to 43 cycles each -- from a branch of a single thread
// it is 55 or more).  It takes 1400 cycles with up to 32 rows, 1700 with 64 and
// 2240 with 128, where the softmax's chain (scores, maximum, exchange,
// exponentials, weights) bounds it, and a CTA 15 to 20 thousand cycles more:
// set-up 3, angles 1.5, rows 2 to 5 (as much instruction fetch as work), the new
// tokens' block 3.5 to 4, epilogue 3.  Measured, bf16, 32 heads on 8 of 128: 64
// sequences of up to 4096 keys, one token each, 82 us (3.4 TB/s of its bytes);
// 64 of 4096, 64 rows a KV head, 149 us (3.7 TB/s, 460 TFLOP/s); 8 of 32768, 128
// rows, 149 us (3.6 TB/s, 920 TFLOP/s); 256 of 256..8192 577 us (4.2 TB/s).
//   warp 0       one 2 KB copy per page: keys by TMA, swizzled for the MMA,
//                values as they lie
//   warp 6       scales: page ids and scale bytes well ahead, what they mean
//                for a group of four blocks into shared memory
//   warp 1       TMEM owner; issues the score MMAs; warp 15 the P V MMAs
//   warps 2-5 and 11-14  softmax, two warps per 32 rows: one thread of each
//                per row, half of the block's keys each (scores stay in
//                registers from the maximum to the weights; the halves agree
//                on the row's reference through shared memory).  Rows of
//                tiles of at most 64 rows are replicated and the copies split
//                the keys again
//   warps 7-10   value tiles to f16
// Warps 2-5 and 7-14 first rotate and split the query rows and the new keys.
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
constexpr int kScaleWarp = 6, kDecodeWarp = 7, kSoftmaxB = 11, kPvWarp = 15, kWarps = 16;
constexpr int kGroup = 4, kGroupSlots = 4;   // blocks whose scales go together; groups in flight
constexpr int kThreads = kWarps * 32;
constexpr int kPrep = 12 * 32;         // threads of the softmax and decode warps
constexpr int kHalves = 2;            // softmax warps sharing 32 rows
constexpr float kHeadroom = 8.f;     // log2 units a row max may grow before O is rescaled
constexpr float kLift = 7.f;         // log2 of the largest weight right after that
constexpr int kNoPage = -1;          // instead of a scale byte
constexpr uint32_t kColS = 0;        // two score tiles: columns 0 and kKeys
// The weights, f16, two keys a column, go over the scores they come from, so
// that a block's need not wait for the block before to leave its own; the next
// scores of that buffer wait for the product instead.  (Weights in columns of
// their own: 128 rows, 8 x 32768 keys, 160 us and not 149; 32 rows, 16 x 1024,
// 16.2 and not 16.0.)
constexpr uint32_t kColO = 2 * kKeys;

enum { kBarKFull = 0, kBarVFull = kBarKFull + kStages, kBarKEmpty = kBarVFull + kStages,
       kBarVEmpty = kBarKEmpty + kStages, kBarSFull = kBarVEmpty + kStages,
       kBarPFull = kBarSFull + 2, kBarPvDone = kBarPFull + 2,
       kBarVbFull = kBarPvDone + 2,
       kBarQReady = kBarVbFull + 2, kBarKnReady = kBarQReady + 1, kBarNewRead = kBarKnReady + 1,
       kBarGFull = kBarNewRead + 1, kBarGEmpty = kBarGFull + kGroupSlots, kNumBars = kBarGEmpty + kGroupSlots };

// What the scales of four blocks mean; entry 8 q + i: page i of block q.
struct Scales {
  float2 kv[8 * kGroup];               // factor of a page's scores; ve
  float inv[8 * kGroup];               // 2^-ve
  uint32_t gone[kGroup];               // pages missing from the block (bits)
};

template <int HD>
struct Smem {
  static constexpr int kCodes = kKeys * HD;                 // K or V codes of a block
  static constexpr int kStage = 2 * kCodes;
  static constexpr int kHalf = kKeys * 128;                 // 128 rows x 64 f16 columns
  static constexpr int kVb = (HD / 64) * kHalf;             // decoded value tile, f16
  static constexpr int kKn = kMaxNew * HD;                  // one part of the new keys
  static constexpr int kOffRing = 0;
  // before their first use the last two stages hold the new keys and values
  // as they came and the query parts, the value tiles the query rows as they
  // came and the angles
  static constexpr int kOffNew = (kStages - 2) * kStage;
  static constexpr int kOffQ = (kStages - 1) * kStage;
  static constexpr int kOffVb = kOffRing + kStages * kStage;   // [2]
  static constexpr int kOffKn = kOffVb + 2 * kVb;           // rotated new keys, hi and lo
  static constexpr int kOffBar = kOffKn + 2 * kKn;
  static constexpr int kOffTau = kOffBar + (kNumBars + 1) / 2 * 16;
  static constexpr int kOffRow = kOffTau + kMaxB * 4;       // rows' score factors
  static constexpr int kOffMax = kOffRow + kRows * 4;       // [2 blocks][2 halves][4 quadrants][32]: row maxima, sums
  static constexpr int kOffNewKv = kOffMax + 2 * kHalves * kRows * 4;       // new tokens: 2^ke and ve of each,
  static constexpr int kOffNewInv = kOffNewKv + kKeys * 8;                  // and 2^-ve (zeros past the last)
  static constexpr int kOffScales = kOffNewInv + kKeys * 4;
  static constexpr int kOffMisc = kOffScales + kGroupSlots * (int)sizeof(Scales);   // tmem address, error flag, odd new
                                                            // values
  static constexpr int kBytes = kOffMisc + 32;
  static constexpr int kAlloc = kBytes + 1024;              // 1024-byte alignment slack
  static constexpr uint32_t kColQ = kColO + HD;             // q hi and lo: hd / 4 columns each
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kOffScales % 16 == 0 && sizeof(Scales) % 16 == 0, "16-byte reads of the scales");
  static_assert(kColQ + HD / 2 <= kTmemCols, "TMEM budget");
  static_assert(2 * kRows * HD <= kStage && 4 * kMaxNew * HD <= kStage && kRows * HD * 2 <= kVb, "first contents fit");
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

// 16 bytes of shared memory, read where it stands (a run of reads ahead of
// their use would not leave registers for the scores).
__device__ __forceinline__ float4 load_shared4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

template <int V> struct IntC { static constexpr int value = V; };

__device__ __forceinline__ void named_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

__device__ __forceinline__ uint64_t shift_right(uint64_t x, int s) { return s >= 64 ? 0ull : x >> s; }

// Byte offset of 16-byte chunk `k` of `row` in a tile of e4m3 rows: the
// 128-byte swizzle for 128-byte rows, the 64-byte one for 64-byte rows.
template <int HD>
__device__ __forceinline__ uint32_t code_off(int row, int k) {
  return HD == 128 ? (uint32_t)(row * 128 + ((k ^ (row & 7)) << 4))
                   : (uint32_t)(row * 64 + ((k ^ ((row >> 1) & 3)) << 4));
}

// Eight values in two e4m3 parts: hi, and lo = e4m3(x - hi).
__device__ __forceinline__ void split8(const float *x, uint2 &hi, uint2 &lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_e4m3x2(x[2 * i], x[2 * i + 1]);
    const float2 f = unpack_e4m3x2(h[i]);
    l[i] = pack_e4m3x2(x[2 * i] - f.x, x[2 * i + 1] - f.y);
  }
  hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

// Four e4m3 codes as two f16 pairs (exact).
__device__ __forceinline__ uint2 unpack4(uint32_t codes) {
  uint2 h;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(h.x), "=r"(h.y)
      : "r"(codes));
  return h;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two fp32 operations in one instruction (half the issue slots).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)),
        "l"(*reinterpret_cast<uint64_t *>(&c)));
  return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
  return *reinterpret_cast<float2 *>(&d);
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
  float *row_s = reinterpret_cast<float *>(sb + L::kOffRow);
  uint32_t *odd_s = reinterpret_cast<uint32_t *>(sb + L::kOffMisc + 8);   // new tokens whose values hold a NaN or an
                                                                          // infinity, one bit each
  float2 *new_kv_s = reinterpret_cast<float2 *>(sb + L::kOffNewKv);
  float *new_inv_s = reinterpret_cast<float *>(sb + L::kOffNewInv);
  Scales *scales_s = reinterpret_cast<Scales *>(sb + L::kOffScales);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 1) {
    tc::alloc(smem_u32(tmem_slot), L::kTmemCols);
    tc::relinquish();
  }
  // the threads that rotate and split rows, their index among them, and the
  // pair whose angles each of them makes (its plan requested here)
  const bool prep_warp = warp >= 2 && warp != kScaleWarp && warp != kPvWarp;
  const int pt = threadIdx.x - (warp < kScaleWarp ? 64 : 96), pair = (pt + 64) % (HD / 2);
  static_assert(kPrep % (HD / 2) == 0, "a thread's angles are of one pair");
  const float turn_hi = plan_by_lane(a.plan).hi[pair], turn_lo = plan_by_lane(a.plan).lo[pair];
  grid_dep_wait();                           // the units' order is there
  grid_dep_launch();                         // the split merge may be scheduled
  const KvqWork w = kvq_work(a);
  if (!w.ok) {                               // uniform: nothing to do here
    __syncthreads();
    if (warp == 1) tc::dealloc(*tmem_slot, L::kTmemCols);
    return;
  }
  const int fresh = w.first ? 1 : 0;         // block 0 is the new tokens'
  const int n_past = max(0, w.k_end - w.k_begin + kKeys - 1) / kKeys;   // prompt blocks
  const int n_blocks = fresh + n_past;
  const int n_pad = (w.n + 15) & ~15;
  // copies of the tile's rows across the four TMEM lane quadrants, and the
  // softmax warps that own real rows
  const int n_groups = min(4, (w.M - w.row0 + 31) / 32);
  const int R = n_groups == 1 ? 4 : n_groups == 2 ? 2 : 1;
  const int n_valid = kHalves * (R > 1 ? 4 : n_groups);
  const int32_t *bt = a.block_table + (int64_t)w.b * a.max_pages;
  const int64_t t0 = (int64_t)a.per * w.c0;  // first new token's row
  // Page ids are requested four blocks ahead of their use and looked at only
  // then: under load such a read takes longer than a block, and a test right
  // after it would hold the warp.
  auto in_cache = [&](int page) { return page >= 0 && page < a.num_pages; };
  // table entry of page `lane` & 7 of prompt block j (lanes 0-15); -1: none
  auto block_page = [&](int j) {
    const int key = w.k_begin + j * kKeys + (lane & 7) * kPage;
    return j < n_past && lane < 2 * kPagesPerBlock && key < w.k_end ? __ldg(bt + key / kPage) : -1;
  };
  // table entry of page `lane` of the four prompt blocks 4 g ..; -1: none
  auto group_page = [&](int g) {
    const int64_t key = w.k_begin + ((int64_t)g * 8 * kGroup + lane) * kPage;
    return key < w.k_end ? __ldg(bt + key / kPage) : -1;
  };
  // scale byte of page `page` and this head; kNoPage: none
  auto scale_byte = [&](const uint8_t *scale, int page) {
    return in_cache(page) ? (int)__ldg(scale + (int64_t)page * a.Hkv + w.kvh) : kNoPage;
  };
  int pages[kStages];
  constexpr int CH = HD / 8;                 // 16-byte chunks of a bf16 row
  if (warp == 0) {
    if (lane == 0) prefetch_tmap(&tmK);
#pragma unroll
    for (int d = 0; d < kStages; ++d) pages[d] = block_page(d);
  } else if (prep_warp) {
    // the query rows and the new tokens' keys and values come first of all,
    // ahead of the stream of codes
    const __nv_bfloat16 *qs = (const __nv_bfloat16 *)a.q + t0 * a.q_row + w.kvh * a.G * HD;
    for (int e = pt; e < n_groups * 32 * CH; e += kPrep) {
      const int r = e / CH, c = e % CH, row = w.row0 + r, tok = div_by(row, a.by_G);
      const bool take = row < w.M;
      copy16_async(base + L::kOffVb + r * HD * 2 + c * 16,
                   take ? qs + tok * a.q_row + (row - tok * a.G) * HD + c * 8 : (const void *)a.q, take);
    }
    if (fresh)
      for (int e = pt; e < w.n * CH; e += kPrep) {
        const int j = e / CH, c = e % CH;
        const uint32_t dst = base + L::kOffNew + j * HD * 2 + c * 16;
        copy16_async(dst, (const __nv_bfloat16 *)a.k_new + (t0 + j) * a.k_row + w.kvh * HD + c * 8, true);
        copy16_async(dst + kMaxNew * HD * 2, (const __nv_bfloat16 *)a.v_new + (t0 + j) * a.v_row + w.kvh * HD + c * 8, true);
      }
  }
  if (warp == kPvWarp) {
    for (int i = lane; i < kNumBars; i += 32) {
      const bool rows = i >= kBarPFull && i < kBarPFull + 2;
      const bool tiles = (i >= kBarVEmpty && i < kBarVEmpty + kStages) || (i >= kBarVbFull && i < kBarVbFull + 2) ||
                         i == kBarQReady || i == kBarKnReady || i == kBarNewRead;
      mbar_init(bar(i), i >= kBarGEmpty ? n_valid + 4 : rows ? n_valid : tiles ? 4 : 1);
    }
    if (lane == 0) {
      *flag_s = 0;
      odd_s[0] = odd_s[1] = 0u;
    }
    for (int i = lane; i < kKeys; i += 32) {
      new_kv_s[i] = make_float2(0.f, 0.f);
      new_inv_s[i] = 0.f;
    }
    fence_barrier_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  int issued = 0;                            // producers: blocks whose loads were started
  float2 *cs_s = reinterpret_cast<float2 *>(sb + L::kOffVb + L::kVb);   // [kMaxNew][HD / 2]
  auto give_up = [&]() { raise_status(a.status, kStatusTimeout); atomicOr(flag_s, 1); };
  // An issuing warp stays until its last product is done (default limit): after a
  // wait that gave up elsewhere nobody else waits for it, and the tiles and tensor
  // memory that it uses go with the CTA.
  auto drain = [&](int bars, int n, int sent) {   // n barriers in turn, one a block
    if (sent > 0) (void)mbar_wait_warp(bar(bars + (sent - 1) % n), ((sent - 1) / n) & 1);
  };
  // The softmax and decode warps together rotate the query rows into two e4m3
  // parts and, in the CTA that owns the new tokens, their keys likewise (the
  // decode warps then take their values); rolled loops, since each CTA runs them
  // once (unrolled per row they took as long as ten blocks, most of it
  // instruction fetch).
  auto prepare = [&]() {
    // angles of the new tokens' positions (identity past the rotated part)
    const int npos = a.order == SIMSD_ORDER_PAIRED ? w.B : a.order == SIMSD_ORDER_NODES ? a.node_size : w.n;
#pragma unroll 1
    for (int e = pt; e < npos * (HD / 2); e += kPrep) {
      float2 cs = make_float2(1.f, 0.f);
      if (pair < a.plan.half) {
        cs = rope_angle(plan_by_lane(a.plan), turn_hi, turn_lo, pair, w.P + e / (HD / 2));
        cs = make_float2(cs.x * a.plan.mul, cs.y * a.plan.mul);
      }
      cs_s[e - pair + angle_at(pair)] = cs;
    }
    if (a.order == SIMSD_ORDER_PAIRED && pt < w.B) tau_s[pt] = __ldg(a.tau + w.c0 + pt);
    copy_async_wait_all();
    const __nv_bfloat16 *ks = reinterpret_cast<const __nv_bfloat16 *>(sb + L::kOffNew), *vs = ks + kMaxNew * HD;
    if (fresh) {                             // each token's ve: its largest finite value (CH lanes hold its row, each
                                             // the chunk that it copied itself)
#pragma unroll 1
      for (int e = pt; e - lane < w.n * CH; e += kPrep) {
        float va = 0.f;
        if (e < w.n * CH) {
          float y[8];
          load_vec<__nv_bfloat16, 8>(vs + e * 8, y);
          bool odd = false;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            odd |= !(fabsf(y[i]) < INFINITY);
            va = fmaxf(va, fabsf(y[i]) < INFINITY ? fabsf(y[i]) : 0.f);
          }
          if (odd) atomicOr(odd_s + (e / CH >> 5), 1u << (e / CH & 31));
        }
#pragma unroll
        for (int m = CH / 2; m > 0; m >>= 1) va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, m));
        if (e < w.n * CH && e % CH == 0) {
          const int ve = scale_exponent(va, -64, 119);
          new_kv_s[e / CH].y = (float)ve;
          new_inv_s[e / CH] = pow2i(-ve);
        }
      }
    }
    named_sync(1, kPrep);
    // rows, query rows first: PL neighbouring lanes hold one (a warp's lanes
    // all have query rows or all new keys: both are multiples of 32 lanes)
    constexpr int PL = HD / 16;
    const __nv_bfloat16 *qs = reinterpret_cast<const __nv_bfloat16 *>(sb + L::kOffVb);
    const int n_q = n_groups * 32 * PL, n_all = n_q + (fresh ? n_pad * PL : 0);   // zeros up to the MMA's depth
#pragma unroll 1
    for (int e = pt; e < n_all; e += kPrep) {
      const bool query = e < n_q;
      const int r = (query ? e : e - n_q) / PL, first = r - (lane / PL);   // row; the warp's first row
      const int c = e % PL;
      uint8_t *dst = sb + (query ? L::kOffQ : L::kOffKn);
      uint8_t *dst_lo = dst + (query ? kRows * HD : L::kKn);
      if (query ? w.row0 + first >= w.M : first >= w.n) {                  // none of them exist
        *reinterpret_cast<uint4 *>(dst + code_off<HD>(r, c)) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(dst_lo + code_off<HD>(r, c)) = make_uint4(0, 0, 0, 0);
        if (query && c == 0) row_s[r] = 0.f;
        continue;
      }
      const int row = w.row0 + r;
      const int tok = !query ? min(r, w.n - 1) : row < w.M ? div_by(row, a.by_G) : 0;
      int c0, c1;
      float x[16], amax = 0.f, nan = 0.f;
      rotate16(a.plan, cs_s + kvq_offset(a, w.B, tok) * (HD / 2), query ? qs + r * HD : ks + tok * HD, c, c0, c1, x);
      if (!query) {
#pragma unroll
        for (int i = 0; i < 16; ++i)         // e4m3 has no infinity
          x[i] = r >= w.n ? 0.f : fabsf(x[i]) < INFINITY ? x[i] : __uint_as_float(0x7fc00000u);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {         // (a NaN is not the maximum)
        nan = fmaf(x[i], 0.f, nan);
        amax = fmaxf(amax, fabsf(x[i]));
      }
#pragma unroll
      for (int m = PL / 2; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
      // a NaN or an infinity: the query row's scores become NaN
      const uint32_t odds = (__ballot_sync(0xffffffffu, nan != 0.f) >> (lane & ~(PL - 1))) & ((1u << PL) - 1u);
      const int ex = scale_exponent(amax, -100, 119);
      const float down = pow2i(-ex);
      if (c == 0) {
        if (query) row_s[r] = odds != 0u ? __uint_as_float(0x7fc00000u) : a.scale * pow2i(ex);
        else if (r < w.n) new_kv_s[r].x = pow2i(ex);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= down;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint2 hi, lo;
        split8(x + 8 * i, hi, lo);
        const int k = i ? c1 : c0;
        const uint32_t off = code_off<HD>(r, k >> 1) + (k & 1) * 8;
        *reinterpret_cast<uint2 *>(dst + off) = hi;
        *reinterpret_cast<uint2 *>(dst_lo + off) = lo;
      }
    }
    fence_proxy_async_smem();
    named_sync(1, kPrep);
  };

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    const bool kside = lane < kPagesPerBlock;
    bool ok = true;
    for (int j0 = 0; ok && j0 < n_past; j0 += kStages) {
#pragma unroll
      for (int s = 0; s < kStages; ++s) {    // s: stage of block j
        const int j = j0 + s;
        if (j >= n_past) break;
        const int page = pages[s];
        const int n_pages = __popc(__ballot_sync(0xffffffffu, kside && in_cache(page)));
        // (the last two stages hold the rows of this CTA until they are split
        // and in TMEM)
        if ((j >= kStages && (!mbar_wait_warp(bar(kBarKEmpty + s), ((j / kStages) - 1) & 1, a.polls) ||
                              !mbar_wait_warp(bar(kBarVEmpty + s), ((j / kStages) - 1) & 1, a.polls))) ||
            ((j == kStages - 2 || j == kStages - 1) && !mbar_wait_warp(bar(kBarQReady), 0, a.polls)) ||
            (j == kStages - 2 && fresh && !mbar_wait_warp(bar(kBarNewRead), 0, a.polls))) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(kBarKFull + s), n_pages * kPage * HD);
          mbar_arrive_expect_tx(bar(kBarVFull + s), n_pages * kPage * HD);
        }
        __syncwarp();
        const uint32_t dst = base + L::kOffRing + s * L::kStage + (lane & 7) * kPage * HD;
        if (in_cache(page)) {
          if (kside)
            tma_load_4d(dst, &tmK, bar(kBarKFull + s), 0, 0, w.kvh, page);
          else
            bulk_load(dst + L::kCodes, a.v_cache + ((int64_t)page * a.Hkv + w.kvh) * kPage * HD, kPage * HD,
                      bar(kBarVFull + s));
        } else if (kside && w.k_begin + j * kKeys + lane * kPage < w.k_end) {
          raise_status(a.status, kStatusBadInput);
        }
        issued = j + 1;
        pages[s] = block_page(j + kStages);
      }
    }
  } else if (warp == kScaleWarp) {
    // ------------------------------------------------------------- scales
    // lane 8 q + i: page i of block 4 g + q; bytes requested a group ahead,
    // page ids two
    int page = group_page(0);
    int kb = scale_byte(a.k_scale, page), vb = scale_byte(a.v_scale, page);
    page = group_page(1);
    bool ok = true;
    const int groups = (n_past + kGroup - 1) / kGroup;
    for (int g = 0; ok && g < groups; ++g) {
      const int slot = g % kGroupSlots;
      if (g >= kGroupSlots && !mbar_wait_warp(bar(kBarGEmpty + slot), ((g / kGroupSlots) - 1) & 1, a.polls)) {
        ok = false;
        break;
      }
      Scales &s = scales_s[slot];
      const uint32_t missing = __ballot_sync(0xffffffffu, kb == kNoPage);
      const int ve = vb - kScaleBias;
      const bool nan = vb < 0 || vb == kScaleNan;
      s.kv[lane] = make_float2(scale_value(kb & 255), nan ? __uint_as_float(0x7fc00000u) : (float)ve);
      s.inv[lane] = nan ? 1.f : scale_value(2 * kScaleBias - vb);
      if (lane < kGroup) s.gone[lane] = (missing >> (8 * lane)) & 0xffu;
      kb = scale_byte(a.k_scale, page);
      vb = scale_byte(a.v_scale, page);
      page = group_page(g + 2);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarGFull + slot));
    }
    if (!ok && lane == 0) give_up();
  } else if (warp == 1) {
    // ------------------------------------------------------------- scores
    // The whole warp keeps the loop (uniform addresses), one lane issues.
    constexpr uint32_t idS8 = tc::idesc_e4m3(kRows, kKeys);
    constexpr uint32_t idSn = tc::idesc_e4m3(kRows, kMaxNew);
    const uint64_t dK0 = HD == 128 ? tc::smem_desc_sw128(base, 16, 1024) : tc::smem_desc_sw64(base, 16, 512);
    // scores of the part q0 of the query rows against the tile at offset off
    auto score = [&](uint32_t tS, uint32_t q0, uint32_t off, uint32_t idesc, bool more) {
#pragma unroll
      for (int kk = 0; kk < HD / 32; ++kk)
        tc::mma_e4m3_ts(tS, q0 + kk * 8, dK0 + ((off + kk * 32) >> 4), idesc, more || kk > 0);
    };
    const uint32_t qhi = tmem + L::kColQ, qlo = qhi + HD / 4;
    bool ok = mbar_wait_warp(bar(kBarQReady), 0, a.polls);
    int sent = 0;                            // blocks whose products were issued
    for (int j = 0; ok && j < n_blocks; ++j) {
      const int tb = j & 1, jp = j - fresh, s = jp & (kStages - 1);
      ok = (jp < 0 ? mbar_wait_warp(bar(kBarKnReady), 0, a.polls)
                   : mbar_wait_warp(bar(kBarKFull + s), (jp / kStages) & 1, a.polls)) &&
           (j < 2 || mbar_wait_warp(bar(kBarPvDone + tb), ((j >> 1) - 1) & 1, a.polls));
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t tS = tmem + kColS + tb * kKeys;
      if (tc::elect_one()) {
        if (jp < 0) {                        // both parts of q against both of the new keys
          score(tS, qhi, L::kOffKn, idSn, false);
          score(tS, qlo, L::kOffKn, idSn, true);
          score(tS, qhi, L::kOffKn + L::kKn, idSn, true);
          score(tS, qlo, L::kOffKn + L::kKn, idSn, true);
          tc::commit(bar(kBarSFull + tb));
        } else {
          score(tS, qhi, s * L::kStage, idS8, false);
          score(tS, qlo, s * L::kStage, idS8, true);
          tc::commit(bar(kBarSFull + tb));
          tc::commit(bar(kBarKEmpty + s));
        }
      }
      __syncwarp();
      sent = j + 1;
    }
    if (!ok && lane == 0) give_up();
    drain(kBarSFull, 2, sent);
    drain(kBarKEmpty, kStages, sent - fresh);
  } else if (warp == kPvWarp) {
    // ---------------------------------------------------------------- P V
    constexpr uint32_t idO = tc::idesc_f16(kRows, HD, 1);
    const uint64_t dV0 = tc::smem_desc_sw128(base + L::kOffVb, L::kHalf, 1024);
    bool ok = true;
    int sent = 0;
    for (int j = 0; j < n_blocks; ++j) {
      const int tb = j & 1, jp = j - fresh;
      ok = mbar_wait_warp(bar(kBarVbFull + tb), (j >> 1) & 1, a.polls) && mbar_wait_warp(bar(kBarPFull + tb), (j >> 1) & 1, a.polls);
      if (!ok) break;
      tc::fence_after_sync();
      const int depth = jp < 0 ? n_pad : min(kKeys, (w.k_end - w.k_begin - jp * kKeys + 15) & ~15);
      const uint64_t dV = dV0 + ((uint32_t)(tb * L::kVb) >> 4);
      const uint32_t tP = tmem + kColS + tb * kKeys;
      if (tc::elect_one()) {
        if (depth == kKeys) {
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            tc::mma_bf16_ts(tmem + kColO, tP + kk * 8, dV + kk * 128, idO, j > 0 || kk > 0);
        } else {
          for (int kk = 0; kk < depth / 16; ++kk)
            tc::mma_bf16_ts(tmem + kColO, tP + kk * 8, dV + kk * 128, idO, j > 0 || kk > 0);
        }
        tc::commit(bar(kBarPvDone + tb));
      }
      __syncwarp();
      sent = j + 1;
    }
    if (!ok && lane == 0) give_up();
    drain(kBarPvDone, 2, sent);
  } else if (warp >= kDecodeWarp && warp < kSoftmaxB) {
    // ------------------------------------------------------------- decode
    const int dw = warp - kDecodeWarp;
    prepare();
    if (fresh) {                             // the new values, as f16, are the first value tile
      if (lane == 0) mbar_arrive(bar(kBarKnReady));
      const __nv_bfloat16 *vs = reinterpret_cast<const __nv_bfloat16 *>(sb + L::kOffNew) + kMaxNew * HD;
#pragma unroll 1
      for (int e = 32 * dw + lane; e < n_pad * CH; e += 128) {
        const int j = e / CH, c = e % CH;
        const float vdown = new_inv_s[j];
        float v[8];
        load_vec<__nv_bfloat16, 8>(vs + e * 8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)          // (an odd one times a weight of 0 would reach every row)
          v[i] = j < w.n && fabsf(v[i]) < INFINITY ? v[i] * vdown : 0.f;
        *reinterpret_cast<uint4 *>(sb + L::kOffVb + (c >> 3) * L::kHalf + swz(j, c & 7)) =
            make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kBarNewRead));
        mbar_arrive(bar(kBarVbFull));
      }
    }
    // value tiles: this warp's rows are pages 2 dw and 2 dw + 1 of a block
    constexpr int C = HD / 8, RPI = 32 / C;                  // 8-byte chunks of a row; rows an iteration
    const int c = lane % C, r0 = 32 * dw + lane / C;
    bool ok = true;
    for (int jp = 0; jp < n_past; ++jp) {
      const int j = jp + fresh, tb = j & 1, s = jp & (kStages - 1), q = jp % kGroup, slot = jp / kGroup % kGroupSlots;
      if (q == 0 && !mbar_wait_warp(bar(kBarGFull + slot), (jp / (kGroup * kGroupSlots)) & 1, a.polls)) { ok = false; break; }
      if (!mbar_wait_warp(bar(kBarVFull + s), (jp / kStages) & 1, a.polls) ||
          (j >= 2 && !mbar_wait_warp(bar(kBarPvDone + tb), ((j >> 1) - 1) & 1, a.polls))) { ok = false; break; }
      const int valid = w.k_end - w.k_begin - jp * kKeys;    // rows from here on hold no key
      const uint32_t gone = scales_s[slot].gone[q];
      const uint8_t *src = sb + L::kOffRing + s * L::kStage + L::kCodes + r0 * HD + c * 8;
      uint8_t *dst = sb + L::kOffVb + tb * L::kVb + (c >> 3) * L::kHalf;
      if (valid >= kKeys && gone == 0u) {
#pragma unroll
        for (int i = 0; i < 32 / RPI; ++i) {                 // eight lanes write a 128-byte row: no bank twice
          const uint2 x = *reinterpret_cast<const uint2 *>(src + i * RPI * HD);
          const uint2 a0 = unpack4(x.x), a1 = unpack4(x.y);
          *reinterpret_cast<uint4 *>(dst + swz(r0 + i * RPI, c & 7)) = make_uint4(a0.x, a0.y, a1.x, a1.y);
        }
      } else {                                               // no key or no page: zeros
#pragma unroll 1
        for (int i = 0; i < 32 / RPI; ++i) {
          const int row = r0 + i * RPI;
          const uint2 x = *reinterpret_cast<const uint2 *>(src + i * RPI * HD);
          const uint2 a0 = unpack4(x.x), a1 = unpack4(x.y);
          const bool none = row >= valid || ((gone >> (row / kPage)) & 1u);
          *reinterpret_cast<uint4 *>(dst + swz(row, c & 7)) = none ? make_uint4(0, 0, 0, 0) : make_uint4(a0.x, a0.y, a1.x, a1.y);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kBarVbFull + tb));
        mbar_arrive(bar(kBarVEmpty + s));
        if (q == kGroup - 1 || jp == n_past - 1) mbar_arrive(bar(kBarGEmpty + slot));
      }
    }
    if (!ok && lane == 0) give_up();
  } else {
    // ------------------------------------------------------------ softmax
    // With at most 64 real rows the tile's rows are replicated across the
    // four TMEM lane quadrants (R = 4 or 2 copies) and the copies split each
    // block's keys; every copy keeps its own reference, its weights of the
    // other copies' keys stay zero, and the epilogue merges the copies.
    const int half = warp >= kSoftmaxB;
    const int q4 = warp & 3;                 // TMEM lane quadrant of this warp
    const int groups = 4 / R;
    const int g = q4 % groups, kp = q4 / groups;
    const int grow = w.row0 + 32 * g + lane;
    const bool row_valid = grow < w.M;
    const bool warp_valid = w.row0 + 32 * g < w.M;
    const int tok = row_valid ? div_by(grow, a.by_G) : 0;
    const uint32_t trow = tmem + ((uint32_t)(32 * q4) << 16);
    // this row's values of the two warps that share it: [block parity][half]
    float *both_s = reinterpret_cast<float *>(sb + L::kOffMax) + 32 * q4 + lane;
    auto pair_sync = [&]() { named_sync(4 + q4, 64); };
    prepare();
    const float rscale = row_s[32 * g + lane];
    if (half == 0) {
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int k = 0; k < HD / 16; k += 2) {
          const uint8_t *src = sb + L::kOffQ + part * kRows * HD;
          uint4 v[2];
          v[0] = *reinterpret_cast<const uint4 *>(src + code_off<HD>(32 * g + lane, k));
          v[1] = *reinterpret_cast<const uint4 *>(src + code_off<HD>(32 * g + lane, k + 1));
          tc::st8(trow + L::kColQ + part * (HD / 4) + k * 4, reinterpret_cast<const uint32_t *>(v));
        }
    }
    tc::wait_st();
    tc::fence_before_sync();
    if (half == 0 && lane == 0) mbar_arrive(bar(kBarQReady));
    const uint64_t newvis = fresh ? kvq_visible(a, w.B, tau_s, tok) : 0ull;
    const uint32_t tO = trow + kColO;
    // a row that sees a new token with an odd value is NaN
    const bool odd = (newvis & ((uint64_t)odd_s[1] << 32 | odd_s[0])) != 0ull;
    float m_ref = -INFINITY, l = odd ? __uint_as_float(0x7fc00000u) : 0.f;
    bool ok = true;
    int j = 0;
    // the key loop, compiled once per copy count, the new tokens' block by itself
    // (a factor and a ve for each key: in the loop they would not leave it its
    // registers, 64 x 4096 keys 171 us and not 149)
    auto key_loop = [&](auto rc) {
      constexpr int RC = decltype(rc)::value;
      constexpr int KW = kKeys / (RC * kHalves);   // this warp's keys per block: 64, 32 or 16
      const int k_lo = (kp * kHalves + half) * KW;
      // A warp whose wait gave up still meets its partner once, with a NaN in
      // the maximum's place (a maximum is never NaN), so both leave the loop.
      auto block = [&](auto newc) {            // block j; false: leave the loop
        constexpr bool is_new = decltype(newc)::value != 0;
        const int tb = is_new ? 0 : j & 1, jp = is_new ? -1 : j - fresh;
        const uint32_t tS = trow + kColS + tb * kKeys + k_lo;
        const int q = jp & (kGroup - 1), slot = jp / kGroup % kGroupSlots;
        if (!is_new && q == 0) ok = ok && mbar_wait_warp(bar(kBarGFull + slot), (jp / (kGroup * kGroupSlots)) & 1, a.polls);
        // a page's 16 keys: t = f s + ve, its weights' share of the sum 2^-ve
        constexpr int NP = KW / 16;
        float f[NP], ve[NP], inv[NP];
        uint32_t gone = 0u;
        if (is_new) {                        // (a factor and a ve for each key, below)
#pragma unroll
          for (int i = 0; i < NP; ++i) { f[i] = 1.f; ve[i] = 0.f; inv[i] = 0.f; }
        } else {
          const Scales &sc = scales_s[slot];
          const int e0 = 8 * q + k_lo / 16;
          gone = sc.gone[q];
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const float2 x = sc.kv[e0 + i];
            f[i] = x.x * rscale; ve[i] = x.y; inv[i] = sc.inv[e0 + i];
          }
        }
        // keys that count: all of a whole block's, else one bit each
        const int valid = is_new ? 0 : w.k_end - w.k_begin - jp * kKeys;
        const bool whole = !is_new && valid >= kKeys && gone == 0u;
        ok = ok && mbar_wait_warp(bar(kBarSFull + tb), (j >> 1) & 1, a.polls);
        tc::fence_after_sync();
        uint32_t sr[KW];
        if constexpr (KW == 16) {
          tc::ld16(tS, sr);
        } else {
#pragma unroll
          for (int q = 0; q < KW; q += 32) tc::ld32(tS + q, sr + q);
        }
        tc::wait_ld();
        tc::fence_before_sync();
        // the row's maximum over both warps' keys
        float mx = -INFINITY;
        if (!whole) {                        // keys that do not count score -inf from here on
          if (is_new) {
            const uint64_t vis = shift_right(newvis, k_lo);
#pragma unroll
            for (int i = 0; i < KW; i += 2) {
              const float4 x = load_shared4(base + L::kOffNewKv + (k_lo + i) * 8);   // of two keys
              sr[i] = __float_as_uint((vis >> i) & 1ull ? fmaf(__uint_as_float(sr[i]), x.x * rscale, x.y) : -INFINITY);
              sr[i + 1] = __float_as_uint((vis >> i) & 2ull ? fmaf(__uint_as_float(sr[i + 1]), x.z * rscale, x.w) : -INFINITY);
            }
          } else {
            uint64_t vis = kvq_low_bits(valid - k_lo);
            for (int i = 0; i < KW / 16; ++i)
              if ((gone >> (k_lo / 16 + i)) & 1u) vis &= ~(0xffffull << (16 * i));
#pragma unroll
            for (int i = 0; i < KW; ++i)
              sr[i] = __float_as_uint((vis >> i) & 1ull ? fmaf(__uint_as_float(sr[i]), f[i / 16], ve[i / 16]) : -INFINITY);
#pragma unroll
            for (int i = 0; i < NP; ++i) { f[i] = 1.f; ve[i] = 0.f; }
          }
        }
#pragma unroll
        for (int i = 0; i < KW; i += 16) {
          float v[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] = __uint_as_float(sr[i + c]);
          const float m0 = max3(max3(v[0], v[1], v[2]), v[3], v[4]), m1 = max3(max3(v[5], v[6], v[7]), v[8], v[9]);
          const float m2 = max3(max3(v[10], v[11], v[12]), v[13], v[14]);
          mx = fmaxf(mx, fmaf(max3(max3(m0, m1, m2), v[15], v[15]), f[i / 16], ve[i / 16]));
        }
        both_s[(tb * kHalves + half) * kRows] = ok ? mx : __uint_as_float(0x7fc00000u);
        pair_sync();
        const float theirs = both_s[(tb * kHalves + (half ^ 1)) * kRows];
        if (!ok || theirs != theirs) { ok = false; return false; }
        mx = fmaxf(mx, theirs);
        // both warps have their scores: weights may go over them, zeros for the
        // other copies' keys first (each warp half of them)
        const uint32_t tW = trow + kColS + tb * kKeys;
        tc::fence_after_sync();
        if constexpr (RC > 1) {
          uint32_t z[KW / 2];
#pragma unroll
          for (int e = 0; e < KW / 2; ++e) z[e] = 0u;
#pragma unroll
          for (int c = 1; c < RC; ++c) {
            const uint32_t at = tW + ((kp + c) % RC) * KW + half * (KW / 2);
            if constexpr (KW == 16) tc::st8(at, z);
            else tc::st16(at, z);
          }
        }
        // reference: moves only when this block's max outgrows it
        const bool move = row_valid && mx > m_ref + kLift + kHeadroom;
        const float m_new = move ? mx - kLift : m_ref;
        const float alpha = move ? ex2(m_ref - m_new) : 1.f;     // m_ref = -inf -> 0
        l *= alpha;
        m_ref = m_new;
        // weights 2^(t - m_ref) as f16 pairs
        const float mu = m_ref == -INFINITY ? 0.f : m_ref;
        if (is_new) {                        // the new tokens' share of the sum, key by key
#pragma unroll
          for (int i = 0; i < KW; i += 4) {
            const float4 x = load_shared4(base + L::kOffNewInv + (k_lo + i) * 4);
            l = fmaf(ex2(__uint_as_float(sr[i]) - mu), x.x, l);
            l = fmaf(ex2(__uint_as_float(sr[i + 1]) - mu), x.y, l);
            l = fmaf(ex2(__uint_as_float(sr[i + 2]) - mu), x.z, l);
            l = fmaf(ex2(__uint_as_float(sr[i + 3]) - mu), x.w, l);
          }
        }
        uint32_t pw[KW / 2];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const float2 f2 = make_float2(f[i], f[i]), b2 = make_float2(ve[i] - mu, ve[i] - mu);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 8 * i; e < 8 * i + 8; ++e) {
            const float2 x = fma2(make_float2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), f2, b2);
            const float2 p = make_float2(ex2(x.x), ex2(x.y));
            sum = add2(sum, p);
            pw[e] = pack_f16x2(p.x, p.y);
          }
          l = fmaf(sum.x + sum.y, inv[i], l);
        }
        // O's rows may be scaled once the previous block's P V is done
        if (!is_new && __any_sync(0xffffffffu, move) && j > 0) {
          if (!mbar_wait_warp(bar(kBarPvDone + (tb ^ 1)), ((j - 1) >> 1) & 1, a.polls)) { ok = false; return true; }
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {  // this half of its columns
            uint32_t o[16];
            tc::ld16(tO + half * (HD / 2) + 16 * c, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::st16(tO + half * (HD / 2) + 16 * c, o);
          }
        }
        const uint32_t tP = tW + k_lo / 2;
        if constexpr (KW == 16) {
          tc::st8(tP, pw);
        } else {
#pragma unroll
          for (int q = 0; q < KW / 2; q += 16) tc::st16(tP + q, pw + q);
        }
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kBarPFull + tb));   // (one for each parity: a warp may be a block ahead of another)
          if (!is_new && (q == kGroup - 1 || jp == n_past - 1)) mbar_arrive(bar(kBarGEmpty + slot));
        }
        return true;
      };
      if (!warp_valid) return;
      if (fresh) {
        if (!block(IntC<1>{})) return;
        j = 1;
      }
      for (; j < n_blocks; ++j)
        if (!block(IntC<0>{})) return;
    };
    if (R == 4) key_loop(IntC<4>{});
    else if (R == 2) key_loop(IntC<2>{});
    else key_loop(IntC<1>{});
    if (ok && j > 0 && !mbar_wait_warp(bar(kBarPvDone + ((j - 1) & 1)), ((j - 1) >> 1) & 1, a.polls)) ok = false;
    if (!ok && lane == 0) give_up();
    tc::fence_after_sync();
    // -------------------------------------------------------- epilogue
    const bool failed = !ok || *(volatile int *)flag_s != 0;
    const int64_t orow = (t0 + tok) * a.Hq + w.kvh * a.G + (row_valid ? grow - tok * a.G : 0);
    // columns [c0, c0 + n), n <= 32, of this thread's row: sums v relative to
    // reference mr, weights' sum lt
    auto write_cols = [&](const float *v, int c0, int n, float lt, float mr) {
      if (w.n_splits == 1) {
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        uint4 *dst = reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.out + orow * HD + c0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * e < n) dst[e] = make_uint4(pack_bf16x2(v[8 * e] * inv, v[8 * e + 1] * inv),
                              pack_bf16x2(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                              pack_bf16x2(v[8 * e + 4] * inv, v[8 * e + 5] * inv),
                              pack_bf16x2(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
      } else {
        const int64_t prow = (int64_t)w.split * a.T * a.Hq + orow;
        float4 *dst = reinterpret_cast<float4 *>(a.o_part + prow * HD + c0);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (4 * e < n) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        if (c0 == 0) a.ml_part[prow] = make_float2(mr, lt);
      }
    };
    // the row's sum over both warps' keys (the maxima's places, block parity 0)
    both_s[half * kRows] = l;
    named_sync(3, 8 * 32);
    l += both_s[(half ^ 1) * kRows];
    if (R == 1) {
      if (warp_valid) {
#pragma unroll 1
        for (int c = 0; c < HD / 64; ++c) {
          const int c0 = half * (HD / 2) + 32 * c;
          uint32_t o[32];
          tc::ld32(tO + c0, o);
          tc::wait_ld();
          if (!row_valid || failed) continue;
          write_cols(reinterpret_cast<const float *>(o), c0, 32, l, m_ref);
        }
      }
    } else {
      // every copy puts its sums and reference in the idle ring; then each
      // warp merges the R partials of its share of the columns
      float *part = reinterpret_cast<float *>(sb + L::kOffRing);   // [R][groups][32][HD + 4]
      float *mine = part + ((kp * groups + g) * 32 + lane) * (HD + 4);
#pragma unroll 1
      for (int c = 0; c < HD / 64; ++c) {
        const int c0 = half * (HD / 2) + 32 * c;
        uint32_t o[32];
        tc::ld32(tO + c0, o);
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<float4 *>(mine + c0 + 4 * e) =
              make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                          __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
      }
      if (half == 0) *reinterpret_cast<float2 *>(mine + HD) = make_float2(m_ref, l);
      named_sync(3, 8 * 32);
      if (row_valid && !failed) {
        const int cw = HD / (R * kHalves), cb = (kp * kHalves + half) * cw;    // 8, 16 or 32 columns
        const float *row = part + (g * 32 + lane) * (HD + 4);                  // copy 0; the others:
        const int next = groups * 32 * (HD + 4);
        float2 ml[4];                          // the copies' references and sums, read together
#pragma unroll
        for (int c = 0; c < 4; ++c)
          ml[c] = c < R ? *reinterpret_cast<const float2 *>(row + c * next + HD) : make_float2(-INFINITY, 0.f);
        const float mt = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
        float lt = 0.f, v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c >= R) break;
          const float wc = ex2(ml[c].x - (mt == -INFINITY ? 0.f : mt));   // -inf reference -> 0
          lt += wc * ml[c].y;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (4 * e >= cw) break;
            const float4 p4 = *reinterpret_cast<const float4 *>(row + c * next + cb + 4 * e);
            v[4 * e] += wc * p4.x; v[4 * e + 1] += wc * p4.y;
            v[4 * e + 2] += wc * p4.z; v[4 * e + 3] += wc * p4.w;
          }
        }
        write_cols(v, cb, cw, lt, mt);
      }
    }
  }
  // -------------------------------------------------------------- teardown
  tc::fence_before_sync();
  __syncthreads();
  // after a wait that gave up, the copies still in flight land before the CTA
  // can exit (default limit)
  if (warp == 0 && *(volatile int *)flag_s)
    for (int j = max(0, issued - kStages); j < issued; ++j) {
      (void)mbar_wait_warp(bar(kBarKFull + j % kStages), (j / kStages) & 1);
      (void)mbar_wait_warp(bar(kBarVFull + j % kStages), (j / kStages) & 1);
    }
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
  return launch_pdl(kern, dim3((unsigned)p.grid), dim3(kThreads), smem, stream, mk, a);
}

}  // namespace

cudaError_t launch_kvq_tc(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a,
                          cudaStream_t stream) {
  CUtensorMap mk;
  if (!make_codes_map(&mk, const_cast<void *>(d->k_cache), d->num_pages, d->num_kv_heads, d->head_dim))
    return cudaErrorInvalidValue;
  return d->head_dim == 128 ? launch_tc_hd<128>(mk, p, a, stream) : launch_tc_hd<64>(mk, p, a, stream);
}

}  // namespace simsd
