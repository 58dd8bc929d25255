// kv4_attn_tc.cu -- simsd_kv4_verify for bf16 data, many query rows a KV head,
// on the tensor cores.
//
// S = Q K^T and O += P V in f16 with fp32 sums (kind::f16).  The cache's values
// are exact in f16 (an e2m1 code times a scale of four bits); a query row and a
// new key or value is held relative to a power of two of its own.  A row's
// weights are p = 2^(t - M + 7), t its scores in log2 units and M a reference at
// most 8 stale, so p <= 2^15 fits f16.  One CTA per (key split, KV head x 128-row
// tile, sequence); rows stack new tokens x heads of the group, so a byte of the
// cache is read and decoded once for all of them.
//   warp 0       one bulk copy per page (18 hd bytes: keys, values, scales)
//   warp 1       TMEM owner; issues the score MMAs; warp 2 the P V MMAs
//   warp 3       nothing (its place keeps the softmax warps on their TMEM lanes)
//   warps 4-11   softmax, two warps per 32 rows: one thread of each per row,
//                half of the block's keys each; the halves agree on the row's
//                reference through shared memory.  Rows of tiles of at most 64
//                rows are replicated and the copies split the keys again
//   warps 12-15  codes times scales to f16 tiles, swizzled for the MMA: two pages
//                of a block's keys each; warps 16-19 of its values
// Warps 4-19 first rotate the query rows and the new keys; the new tokens are a
// block of their own ahead of the prompt.  Lanes of a decoding warp are set on
// elements so that neither their reads nor their writes meet in a bank.
// Every wait is bounded (status bit, drain, return).
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
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
constexpr int kPvWarp = 2, kSoftmaxWarp = 4, kDecodeWarp = 12, kValueWarp = 16, kWarps = 20;
constexpr int kDecoders = 4;          // warps for a tile
constexpr int kPagesPerWarp = kPagesPerBlock / kDecoders;
constexpr int kThreads = kWarps * 32;
constexpr int kPrep = 16 * 32;         // threads of the softmax and decoding warps
constexpr int kHalves = 2;            // softmax warps sharing 32 rows
constexpr int kGone = 16;             // blocks whose missing pages are kept (a producer is at most 7 ahead of a softmax)
constexpr float kHeadroom = 8.f;     // log2 units a row max may grow before O is rescaled
constexpr float kLift = 7.f;         // log2 of the largest weight right after that
constexpr uint32_t kColS = 0;        // two score tiles: columns 0 and kKeys
// The weights, f16, two keys a column, go over the scores they come from: those
// of keys 0..63 from the tile's first column on, those of 64..127 from its 65th,
// so that neither of a row's two warps writes where the other still reads.
__host__ __device__ constexpr uint32_t weight_col(int key) { return (uint32_t)((key & 64) + (key & 63) / 2); }
constexpr uint32_t kColO = 2 * kKeys;

enum { kBarFull = 0, kBarEmpty = kBarFull + kStages, kBarKbFull = kBarEmpty + kStages, kBarVbFull = kBarKbFull + 2,
       kBarSFull = kBarVbFull + 2, kBarPFull = kBarSFull + 2, kBarPvDone = kBarPFull + 2,
       kBarQReady = kBarPvDone + 2, kBarNewRead = kBarQReady + 1, kNumBars = kBarNewRead + 1 };

template <int HD>
struct Smem {
  static constexpr int kRec = Record<HD>::kBytes;
  static constexpr int kStage = kPagesPerBlock * kRec;
  static constexpr int kHalf = kKeys * 128;                 // 128 rows x 64 f16 columns
  static constexpr int kTile = (HD / 64) * kHalf;           // decoded tile, f16
  static constexpr int kOffKb = 0;                          // [2]
  static constexpr int kOffVb = kOffKb + 2 * kTile;         // [2]
  static constexpr int kOffRing = kOffVb + 2 * kTile;
  // before their first use the last two stages hold the new keys and values as
  // they came, the second value tile the query rows as they came, the second key
  // tile the angles, the first value tile the rotated query rows
  static constexpr int kOffNew = kOffRing + (kStages - 2) * kStage;
  static constexpr int kOffRaw = kOffVb + kTile;
  static constexpr int kOffCs = kOffKb + kTile;
  static constexpr int kOffQ = kOffVb;
  static constexpr int kOffBar = kOffRing + kStages * kStage;
  static constexpr int kOffTau = kOffBar + (kNumBars + 1) / 2 * 16;
  static constexpr int kOffRow = kOffTau + kMaxB * 4;       // rows' score factors
  static constexpr int kOffMax = kOffRow + kRows * 4;       // [2 blocks][2 halves][4 quadrants][32]: row maxima, sums
  static constexpr int kOffNewKv = kOffMax + 2 * kHalves * kRows * 4;       // new tokens: 2^ke and ve of each,
  static constexpr int kOffNewInv = kOffNewKv + kKeys * 8;                  // and 2^-ve (zeros past the last)
  static constexpr int kOffGone = kOffNewInv + kKeys * 4;
  static constexpr int kOffMisc = kOffGone + kGone * 4;     // tmem address, error flag, odd new values
  static constexpr int kBytes = kOffMisc + 32;
  static constexpr int kAlloc = kBytes + 1024;              // 1024-byte alignment slack
  static constexpr uint32_t kColQ = kColO + HD;             // the query: hd / 2 columns
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kColQ + HD / 2 <= kTmemCols, "TMEM budget");
  static_assert(4 * kMaxNew * HD <= 2 * kStage && kRows * HD * 2 <= kTile && kMaxNew * (HD / 2) * 8 <= kTile,
                "first contents fit");
  static_assert(4 * 32 * (HD + 4) * 4 <= kStages * kStage, "epilogue exchange fits the ring");
  static_assert(kOffRing % 128 == 0 && kStage % 16 == 0, "alignment");
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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ uint4 mul4(uint4 h, uint32_t s) {
  return make_uint4(mul_f16x2(h.x, s), mul_f16x2(h.y, s), mul_f16x2(h.z, s), mul_f16x2(h.w, s));
}

// One page's keys to a tile: lane (row r and r + 8, 32 elements).  Lanes of the
// upper half of the head take their runs of 8 in another order, so that eight
// lanes write to eight different 16-byte columns.
template <int HD>
__device__ __forceinline__ void decode_keys(const uint8_t *rec, uint8_t *tile, int page, int lane) {
  constexpr int C = HD / 32;                         // lanes of a row
  constexpr int RPI = 32 / C;                        // rows in a step
  const int c = lane % C, r0 = lane / C;
  const bool swap = (c & 2) != 0;
#pragma unroll
  for (int i = 0; i < kPage / RPI; ++i) {
    const int r = r0 + i * RPI, row = page * kPage + r;
    const uint4 w = *reinterpret_cast<const uint4 *>(rec + r * (HD / 2) + c * 16);
    const uint32_t two = *reinterpret_cast<const uint16_t *>(rec + Record<HD>::kKs + r * (HD / 16) + 2 * c);
    const uint32_t s0 = scale4_twice(two, 0), s1 = scale4_twice(two, 1);
    const uint32_t sa = swap ? s1 : s0, sb = swap ? s0 : s1;
    const uint32_t k[4] = {swap ? w.z : w.x, swap ? w.w : w.y, swap ? w.x : w.z, swap ? w.y : w.w};
    uint8_t *dst = tile + (c >> 1) * Smem<HD>::kHalf;
    const int c0 = (c & 1) * 4 + (swap ? 2 : 0);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint4 *>(dst + swz(row, c0 ^ q)) = mul4(unpack_e2m1x8(k[q]), q < 2 ? sa : sb);
  }
}

// One page's values to a tile: lane (pair of tokens, 16 elements of it), the
// upper half of 32 elements writing its odd token first.  mask0, mask1: tokens
// of the pair that count (f16 bits of the scales).
template <int HD>
__device__ __forceinline__ void decode_values(const uint8_t *rec, uint8_t *tile, int page, int valid, int lane) {
  using R = Record<HD>;
  const int half = lane & 1, pair = (lane >> 1) & 7, row = page * kPage + 2 * pair;
  const uint32_t sel_a = half ? 0x7632u : 0x5410u, sel_b = half ? 0x5410u : 0x7632u;
  const uint32_t keep = (row < valid ? 0xffffu : 0u) | (row + 1 < valid ? 0xffff0000u : 0u);
#pragma unroll
  for (int i = 0; i < HD / 64; ++i) {
    const int g = 2 * (2 * i + (lane >> 4)) + half;  // group of 16 elements
    const uint4 w = *reinterpret_cast<const uint4 *>(rec + R::kV + i * 512 + lane * 16);
    const uint32_t s = scale4_pair(*reinterpret_cast<const uint16_t *>(rec + R::vs_at(pair, g))) & keep;
    const uint32_t k[4] = {w.x, w.y, w.z, w.w};
    uint32_t a[8], b[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 h = mul4(unpack_e2m1x8(k[q]), s);  // an element a pair: (even, odd) token
      a[2 * q] = __byte_perm(h.x, h.y, sel_a);
      a[2 * q + 1] = __byte_perm(h.z, h.w, sel_a);
      b[2 * q] = __byte_perm(h.x, h.y, sel_b);
      b[2 * q + 1] = __byte_perm(h.z, h.w, sel_b);
    }
    uint8_t *dst = tile + (g >> 2) * Smem<HD>::kHalf;
    const int ch = (g & 3) * 2, ra = row + half, rb = row + 1 - half;
    *reinterpret_cast<uint4 *>(dst + swz(ra, ch)) = make_uint4(a[0], a[1], a[2], a[3]);
    *reinterpret_cast<uint4 *>(dst + swz(rb, ch)) = make_uint4(b[0], b[1], b[2], b[3]);
    *reinterpret_cast<uint4 *>(dst + swz(ra, ch + 1)) = make_uint4(a[4], a[5], a[6], a[7]);
    *reinterpret_cast<uint4 *>(dst + swz(rb, ch + 1)) = make_uint4(b[4], b[5], b[6], b[7]);
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
kv4_tc_kernel(const __grid_constant__ KvqParams a) {
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
  uint32_t *gone_s = reinterpret_cast<uint32_t *>(sb + L::kOffGone);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 1) {
    tc::alloc(smem_u32(tmem_slot), L::kTmemCols);
    tc::relinquish();
  }
  // the threads that rotate rows, their index among them, and the pair whose
  // angles each of them makes (its plan requested here)
  const bool prep_warp = warp >= kSoftmaxWarp;
  const int pt = threadIdx.x - 32 * kSoftmaxWarp, pair = threadIdx.x % (HD / 2);
  static_assert(kPrep % (HD / 2) == 0 && 32 * kSoftmaxWarp % (HD / 2) == 0, "a thread's angles are of one pair");
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
  // table entry of page `lane` & 7 of prompt block j; -1: none
  auto block_page = [&](int j) {
    const int key = w.k_begin + j * kKeys + (lane & 7) * kPage;
    return j < n_past && key < w.k_end ? __ldg(bt + key / kPage) : -1;
  };
  int pages[kStages];
  constexpr int CH = HD / 8;                 // 16-byte chunks of a bf16 row
  if (warp == 0) {
#pragma unroll
    for (int d = 0; d < kStages; ++d) pages[d] = block_page(d);
  } else if (prep_warp) {
    // the query rows and the new tokens' keys and values come first of all,
    // ahead of the stream of codes
    const __nv_bfloat16 *qs = (const __nv_bfloat16 *)a.q + t0 * a.q_row + w.kvh * a.G * HD;
    for (int e = pt; e < n_groups * 32 * CH; e += kPrep) {
      const int r = e / CH, c = e % CH, row = w.row0 + r, tok = div_by(row, a.by_G);
      const bool take = row < w.M;
      copy16_async(base + L::kOffRaw + r * HD * 2 + c * 16,
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
      const bool tiles = i >= kBarKbFull && i < kBarVbFull + 2;
      mbar_init(bar(i), rows ? n_valid : tiles ? kDecoders : i >= kBarEmpty && i < kBarEmpty + kStages ? 2 * kDecoders
                      : i == kBarQReady ? 4 : i == kBarNewRead ? kDecoders : 1);
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
  float2 *cs_s = reinterpret_cast<float2 *>(sb + L::kOffCs);            // [kMaxNew][HD / 2]
  auto give_up = [&]() { raise_status(a.status, kStatusTimeout); atomicOr(flag_s, 1); };
  // These warps together rotate the query rows and, in the CTA that owns the new
  // tokens, their keys, to f16 relative to a power of two of each row's; rolled
  // loops, since each CTA runs them once.
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
    const __nv_bfloat16 *qs = reinterpret_cast<const __nv_bfloat16 *>(sb + L::kOffRaw);
    const int n_q = n_groups * 32 * PL, n_all = n_q + (fresh ? n_pad * PL : 0);   // zeros up to the MMA's depth
#pragma unroll 1
    for (int e = pt; e < n_all; e += kPrep) {
      const bool query = e < n_q;
      const int r = (query ? e : e - n_q) / PL, first = r - (lane / PL);   // row; the warp's first row
      const int c = e % PL;
      // 16-byte chunk k of the row: query rows one after another, keys as the score MMA's tile
      auto place = [&](int k) {
        return sb + (query ? L::kOffQ + r * HD * 2 + ((k ^ (r & 7)) << 4)
                           : L::kOffKb + (k >> 3) * L::kHalf + (int)swz(r, k & 7));
      };
      if (query ? w.row0 + first >= w.M : first >= w.n) {                  // none of them exist
        *reinterpret_cast<uint4 *>(place(2 * c)) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(place(2 * c + 1)) = make_uint4(0, 0, 0, 0);
        if (query && c == 0) row_s[r] = 0.f;
        continue;
      }
      const int row = w.row0 + r;
      const int tok = !query ? min(r, w.n - 1) : row < w.M ? div_by(row, a.by_G) : 0;
      int c0, c1;
      float x[16], amax = 0.f, nan = 0.f;
      rotate16(a.plan, cs_s + kvq_offset(a, w.B, tok) * (HD / 2), query ? qs + r * HD : ks + tok * HD, c, c0, c1, x);
      if (!query && r >= w.n) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {         // (a NaN is not the maximum)
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
        if (query) row_s[r] = a.scale * up;
        else if (r < w.n) new_kv_s[r].x = up;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float *y = x + 8 * i;
        *reinterpret_cast<uint4 *>(place(i ? c1 : c0)) =
            make_uint4(pack_f16x2(y[0] * down, y[1] * down), pack_f16x2(y[2] * down, y[3] * down),
                       pack_f16x2(y[4] * down, y[5] * down), pack_f16x2(y[6] * down, y[7] * down));
      }
    }
    fence_proxy_async_smem();
    named_sync(1, kPrep);
  };

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    bool ok = true;
    for (int j0 = 0; ok && j0 < n_past; j0 += kStages) {
#pragma unroll
      for (int s = 0; s < kStages; ++s) {    // s: stage of block j
        const int j = j0 + s;
        if (j >= n_past) break;
        const int page = pages[s];
        const bool there = lane < kPagesPerBlock && in_cache(page);
        const uint32_t have = __ballot_sync(0xffffffffu, there);
        // (the last two stages hold the new tokens until they are converted)
        if ((j >= kStages && !mbar_wait_warp(bar(kBarEmpty + s), ((j / kStages) - 1) & 1, a.polls)) ||
            (j == kStages - 2 && fresh && !mbar_wait_warp(bar(kBarNewRead), 0, a.polls))) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        if (lane == 0) {
          gone_s[j & (kGone - 1)] = have ^ 0xffu;
          mbar_arrive_expect_tx(bar(kBarFull + s), __popc(have) * L::kRec);
        }
        __syncwarp();
        if (there)
          bulk_load(base + L::kOffRing + s * L::kStage + lane * L::kRec,
                    a.k_cache + ((int64_t)page * a.Hkv + w.kvh) * L::kRec, L::kRec, bar(kBarFull + s));
        else if (lane < kPagesPerBlock && w.k_begin + j * kKeys + lane * kPage < w.k_end)
          raise_status(a.status, kStatusBadInput);
        issued = j + 1;
        pages[s] = block_page(j + kStages);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- scores
    // The whole warp keeps the loop (uniform addresses), one lane issues.
    constexpr uint32_t idS = tc::idesc_f16(kRows, kKeys, 0), idSn = tc::idesc_f16(kRows, kMaxNew, 0);
    const uint64_t dK0 = tc::smem_desc_sw128(base + L::kOffKb, 16, 1024);
    auto score = [&](uint32_t tS, int tb, uint32_t idesc) {
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
        tc::mma_bf16_ts(tS, tmem + L::kColQ + kk * 8,
                        dK0 + ((uint32_t)(tb * L::kTile + (kk >> 2) * L::kHalf + (kk & 3) * 32) >> 4), idesc, kk > 0);
    };
    bool ok = mbar_wait_warp(bar(kBarQReady), 0, a.polls);
    for (int j = 0; ok && j < n_blocks; ++j) {
      const int tb = j & 1;
      ok = mbar_wait_warp(bar(kBarKbFull + tb), (j >> 1) & 1, a.polls) &&
           (j < 2 || mbar_wait_warp(bar(kBarPvDone + tb), ((j >> 1) - 1) & 1, a.polls));
      if (!ok) break;
      tc::fence_after_sync();
      if (tc::elect_one()) {
        if (j < fresh) score(tmem + kColS + tb * kKeys, tb, idSn);
        else score(tmem + kColS + tb * kKeys, tb, idS);
        tc::commit(bar(kBarSFull + tb));
      }
      __syncwarp();
    }
    if (!ok && lane == 0) give_up();
  } else if (warp == kPvWarp) {
    // ---------------------------------------------------------------- P V
    constexpr uint32_t idO = tc::idesc_f16(kRows, HD, 1);
    const uint64_t dV0 = tc::smem_desc_sw128(base + L::kOffVb, L::kHalf, 1024);
    bool ok = true;
    for (int j = 0; j < n_blocks; ++j) {
      const int tb = j & 1, jp = j - fresh;
      ok = mbar_wait_warp(bar(kBarVbFull + tb), (j >> 1) & 1, a.polls) && mbar_wait_warp(bar(kBarPFull + tb), (j >> 1) & 1, a.polls);
      if (!ok) break;
      tc::fence_after_sync();
      const int depth = jp < 0 ? n_pad : min(kKeys, (w.k_end - w.k_begin - jp * kKeys + 15) & ~15);
      const uint64_t dV = dV0 + ((uint32_t)(tb * L::kTile) >> 4);
      const uint32_t tP = tmem + kColS + tb * kKeys;
      if (tc::elect_one()) {
        if (depth == kKeys) {
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            tc::mma_bf16_ts(tmem + kColO, tP + weight_col(16 * kk), dV + kk * 128, idO, j > 0 || kk > 0);
        } else {
          for (int kk = 0; kk < depth / 16; ++kk)
            tc::mma_bf16_ts(tmem + kColO, tP + weight_col(16 * kk), dV + kk * 128, idO, j > 0 || kk > 0);
        }
        tc::commit(bar(kBarPvDone + tb));
      }
      __syncwarp();
    }
    if (!ok && lane == 0) give_up();
  } else if (warp >= kDecodeWarp) {
    // ------------------------------------------------------------- decode
    const bool values = warp >= kValueWarp;
    const int pg0 = (warp - (values ? kValueWarp : kDecodeWarp)) * kPagesPerWarp;   // this warp's pages of every block
    prepare();
    // (the tiles hold the angles and rows until the query is in TMEM)
    bool ok = mbar_wait_warp(bar(kBarQReady), 0, a.polls);
    if (ok && fresh && !values && lane == 0) mbar_arrive(bar(kBarKbFull));          // the new keys are the first key tile
    if (ok && fresh && values) {             // the new values, as f16, are the first value tile
      const __nv_bfloat16 *vs = reinterpret_cast<const __nv_bfloat16 *>(sb + L::kOffNew) + kMaxNew * HD;
#pragma unroll 1
      for (int e = threadIdx.x - 32 * kValueWarp; e < n_pad * CH; e += 32 * kDecoders) {
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
    // a tile is free when the product that read it is done: scores for keys, P V for values
    const int free_bar = values ? kBarPvDone : kBarSFull, full_bar = values ? kBarVbFull : kBarKbFull;
    for (int jp = 0; ok && jp < n_past; ++jp) {
      const int j = jp + fresh, tb = j & 1, s = jp & (kStages - 1);
      if (!mbar_wait_warp(bar(kBarFull + s), (jp / kStages) & 1, a.polls) ||
          (j >= 2 && !mbar_wait_warp(bar(free_bar + tb), ((j >> 1) - 1) & 1, a.polls))) { ok = false; break; }
      const uint8_t *rec = sb + L::kOffRing + s * L::kStage + pg0 * L::kRec;
      uint8_t *tile = sb + (values ? L::kOffVb : L::kOffKb) + tb * L::kTile;
      if (values) {
        const uint32_t gone = gone_s[jp & (kGone - 1)] >> pg0;
        const int valid = w.k_end - w.k_begin - jp * kKeys;
#pragma unroll
        for (int i = 0; i < kPagesPerWarp; ++i)
          decode_values<HD>(rec + i * L::kRec, tile, pg0 + i, (gone >> i) & 1u ? 0 : valid, lane);
      } else {
#pragma unroll
        for (int i = 0; i < kPagesPerWarp; ++i) decode_keys<HD>(rec + i * L::kRec, tile, pg0 + i, lane);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(full_bar + tb));
        mbar_arrive(bar(kBarEmpty + s));
      }
    }
    if (!ok && lane == 0) give_up();
  } else if (warp >= kSoftmaxWarp) {
    // ------------------------------------------------------------ softmax
    // With at most 64 real rows the tile's rows are replicated across the
    // four TMEM lane quadrants (R = 4 or 2 copies) and the copies split each
    // block's keys; every copy keeps its own reference, its weights of the
    // other copies' keys stay zero, and the epilogue merges the copies.
    const int half = (warp - kSoftmaxWarp) >> 2;
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
      const int r = 32 * g + lane;
#pragma unroll
      for (int k = 0; k < HD / 8; k += 2) {
        uint4 v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = *reinterpret_cast<const uint4 *>(sb + L::kOffQ + r * HD * 2 + (((k + i) ^ (r & 7)) << 4));
        tc::st8(trow + L::kColQ + k * 4, reinterpret_cast<const uint32_t *>(v));
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
    // (a factor and a ve for each key)
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
        // keys that count: all of a whole block's, else one bit each
        const int valid = is_new ? 0 : w.k_end - w.k_begin - jp * kKeys;
        ok = ok && mbar_wait_warp(bar(kBarSFull + tb), (j >> 1) & 1, a.polls);
        const uint32_t gone = is_new || !ok ? 0u : gone_s[jp & (kGone - 1)];
        const bool whole = !is_new && valid >= kKeys && gone == 0u;
        const float f = whole ? rscale : 1.f;      // t = f s
        uint64_t vis = 0;
        if (is_new) {
          vis = shift_right(newvis, k_lo);
        } else if (!whole) {
          vis = kvq_low_bits(valid - k_lo);
          for (int i = 0; i < KW / 16; ++i)
            if ((gone >> (k_lo / 16 + i)) & 1u) vis &= ~(0xffffull << (16 * i));
        }
        tc::fence_after_sync();
        // the scores of this warp's keys CW q ..; where some do not count, as t
        // with -inf for those.  (64 keys are read twice, 32 at a time: once for the
        // maximum, once for the weights.  That leaves registers for 20 warps.)
        constexpr int CW = KW < 32 ? KW : 32;
        uint32_t sr[CW];
        auto fetch = [&](int q) {
          if constexpr (CW == 16) tc::ld16(tS, sr);
          else tc::ld32(tS + CW * q, sr);
          tc::wait_ld();
          if (whole) return;
          if (is_new) {
#pragma unroll
            for (int i = 0; i < CW; i += 2) {
              const float4 x = load_shared4(base + L::kOffNewKv + (k_lo + CW * q + i) * 8);   // of two keys
              const uint32_t v = (uint32_t)(vis >> (CW * q + i));
              sr[i] = __float_as_uint(v & 1u ? fmaf(__uint_as_float(sr[i]), x.x * rscale, x.y) : -INFINITY);
              sr[i + 1] = __float_as_uint(v & 2u ? fmaf(__uint_as_float(sr[i + 1]), x.z * rscale, x.w) : -INFINITY);
            }
          } else {
            const uint32_t v = (uint32_t)(vis >> (CW * q));
#pragma unroll
            for (int i = 0; i < CW; ++i)
              sr[i] = __float_as_uint((v >> i) & 1u ? __uint_as_float(sr[i]) * rscale : -INFINITY);
          }
        };
        // the row's maximum over both warps' keys
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < KW / CW; ++q) {
          fetch(q);
#pragma unroll
          for (int i = 0; i < CW; i += 16) {
            float v[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] = __uint_as_float(sr[i + c]);
            const float m0 = max3(max3(v[0], v[1], v[2]), v[3], v[4]), m1 = max3(max3(v[5], v[6], v[7]), v[8], v[9]);
            const float m2 = max3(max3(v[10], v[11], v[12]), v[13], v[14]);
            mx = fmaxf(mx, max3(max3(m0, m1, m2), v[15], v[15]) * f);
          }
        }
        tc::fence_before_sync();
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
            const uint32_t at = tW + weight_col((kp + c) % RC * 2 * KW) + half * (KW / 2);
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
        const uint32_t tP = tW + weight_col(k_lo);
        const float2 f2 = make_float2(f, f), b2 = make_float2(-mu, -mu);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < KW / CW; ++q) {
          if (KW > CW) fetch(q);
          if (is_new) {                      // the new tokens' share of the sum, key by key
#pragma unroll
            for (int i = 0; i < CW; i += 4) {
              const float4 x = load_shared4(base + L::kOffNewInv + (k_lo + CW * q + i) * 4);
              l = fmaf(ex2(__uint_as_float(sr[i]) - mu), x.x, l);
              l = fmaf(ex2(__uint_as_float(sr[i + 1]) - mu), x.y, l);
              l = fmaf(ex2(__uint_as_float(sr[i + 2]) - mu), x.z, l);
              l = fmaf(ex2(__uint_as_float(sr[i + 3]) - mu), x.w, l);
            }
          }
          uint32_t pw[CW / 2];
#pragma unroll
          for (int e = 0; e < CW / 2; ++e) {
            const float2 x = fma_f32x2(make_float2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), f2, b2);
            const float2 p = make_float2(ex2(x.x), ex2(x.y));
            sum = add_f32x2(sum, p);
            pw[e] = pack_f16x2(p.x, p.y);
          }
          if constexpr (CW == 16) tc::st8(tP, pw);
          else tc::st16(tP + CW / 2 * q, pw);
        }
        if (!is_new) l += sum.x + sum.y;
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPFull + tb));   // (one for each parity: a warp may be a block ahead of another)
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
    for (int j = max(0, issued - kStages); j < issued; ++j)
      (void)mbar_wait_warp(bar(kBarFull + j % kStages), (j / kStages) & 1);
  if (warp == 1) {
    tc::fence_after_sync();
    tc::dealloc(tmem, L::kTmemCols);
  }
}

static_assert(Smem<128>::kAlloc <= 227 * 1024, "shared memory budget");

template <int HD>
cudaError_t launch_tc_hd(const KvqPlan &p, const KvqParams &a, cudaStream_t stream) {
  auto kern = kv4_tc_kernel<HD>;
  const int smem = Smem<HD>::kAlloc;
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

}  // namespace

cudaError_t launch_kv4_tc(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a, cudaStream_t stream) {
  return d->head_dim == 128 ? launch_tc_hd<128>(p, a, stream) : launch_tc_hd<64>(p, a, stream);
}

}  // namespace simsd
