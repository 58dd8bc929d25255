// kv4_attn_tc.cu -- simsd_kv4_verify for bf16 data, many query rows a KV head,
// on the tensor cores.
//
// S = Q K^T and O += P V in f16 with fp32 sums (kind::f16).  The cache's values
// are exact in f16 (an e2m1 code times a scale of four bits); a query row and a
// new key or value is held relative to a power of two of its own.  A row's
// weights are p = 2^(t - M), t its scores in log2 units (of new tokens: plus their
// values' exponent) and M a reference that starts 7 (15 in the new tokens' block)
// below the largest of them and moves before p passes 2^15, f16's range.  One CTA per (key split, KV head x 128-row
// tile, sequence); rows stack new tokens x heads of the group, so a byte of the
// cache is read and decoded once for all of them.
//   warps 0, 3   one bulk copy per page (18 hd bytes: keys, values, scales), a
//                block each in turns
//   warp 1       TMEM owner; issues the score MMAs; warp 2 the P V MMAs
//   warps 4-11   softmax, two warps per 32 rows: one thread of each per row,
//                half of the block's keys each.  Rows of tiles of at most 64
//                rows are replicated and the copies split the keys again
//   warps 12-15  codes times scales to f16 tiles, swizzled for the MMA: two pages
//                of a block's keys each; warps 16-19 of its values
// Warps 4-19 first rotate the query rows and the new keys; the new tokens are a
// block of their own ahead of the prompt.  A row's reference is not looked for in
// every block: the weights are made with the one there is, and their sum, needed
// anyhow, shows whether it holds (without the maxima 150 -> 137 us for 8 x 32768).
// Every wait is bounded (status bit, drain, return).
//
// What bounds it (2.07 GHz): at 128 rows the softmax's chain, 2100 cycles a block of
// 128 keys (scores from TMEM, 340 cycles of exponentials and packing twice, the
// pair's barrier, weights to TMEM), where the tensor cores need 1024; at 64 rows
// the decoding warps, 1600 to 1900 (700 to 1000 of it decoding, the rest the
// latencies of waits and arrivals); and 14000 cycles of set-up and 4300 of epilogue
// a CTA.  8 x 32768 keys, 16 + 16 new tokens, 32 / 8 heads of 128: 136 us, of 70
// on the tensor cores; 64 x 4096, 8 + 8: 139 us, of 48 by bytes; 256 x 256..8192,
// 4..8: 541 us, of 206 by bytes.
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
constexpr int kPvWarp = 2, kSecondProducer = 3, kSoftmaxWarp = 4, kDecodeWarp = 12, kValueWarp = 16, kWarps = 20;
constexpr int kDecoders = 4;          // warps for a tile
constexpr int kPagesPerWarp = kPagesPerBlock / kDecoders;
constexpr int kThreads = kWarps * 32;
constexpr int kPrep = 16 * 32;         // threads of the softmax and decoding warps
constexpr int kHalves = 2;            // softmax warps sharing 32 rows
constexpr int kGone = 16;             // blocks whose missing pages are kept (a producer is at most 7 ahead of a softmax)
constexpr float kLift = 7.f;         // log2 of a row's largest weight right after its reference moved
constexpr float kMostSum = 32768.f;  // sum of a thread's weights in a block that moves it
// TMEM: five units of 64 columns, then the output, then the query.  Block j's
// scores are in units j and j + 2 (mod 5; 64 keys each); its weights, f16, two
// keys a column, go over the first of them, so that the scores of block j + 2
// need wait only for block j's weights and for the P V of block j - 3: a cycle
// of score, softmax, P V and score again would be longer than the softmax.  A
// row's warp h has keys 32 h .. 32 h + 31 of both units and puts their weights
// into columns 32 h .. 32 h + 31, where nobody else reads.
constexpr int kUnits = 5;
constexpr uint32_t kUnitCols = 64;
constexpr uint32_t kColO = kUnits * kUnitCols;
__device__ __forceinline__ uint32_t unit_col(int j, int which) { return (uint32_t)((j + 2 * which) % kUnits) * kUnitCols; }
__host__ __device__ constexpr uint32_t weight_col(int key) { return (uint32_t)((key & 32) + (key >> 6) * 16 + (key & 31) / 2); }
// Barriers of the weights and of the P V, by block: the scores' warp looks three
// blocks back, and the softmax can be two blocks ahead of a P V whose values are
// late, so a pair of barriers would pass a phase that is still to be waited for.
constexpr int kPvBars = 4;

enum { kBarFull = 0, kBarEmpty = kBarFull + kStages, kBarKbFull = kBarEmpty + kStages, kBarVbFull = kBarKbFull + 2,
       kBarSFull = kBarVbFull + 2, kBarPFull = kBarSFull + 2, kBarPvDone = kBarPFull + kPvBars,
       kBarQReady = kBarPvDone + kPvBars, kBarNewRead = kBarQReady + 1, kBarRaw = kBarNewRead + 1, kNumBars = kBarRaw + 1 };

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
  static constexpr int kOffNewDown = kOffNewKv + kKeys * 8;                 // 2^-ve, and kShareLift - ve
  static constexpr int kOffNewShare = kOffNewDown + kMaxNew * 4;
  static constexpr int kOffGone = kOffNewShare + kMaxNew * 4;
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

__device__ __forceinline__ uint4 mul4(uint4 h, uint32_t s) {
  return make_uint4(mul_f16x2(h.x, s), mul_f16x2(h.y, s), mul_f16x2(h.z, s), mul_f16x2(h.w, s));
}

// One page's keys to a tile (rows of 64 elements of a key): a lane takes 32
// elements of a row.  Which 32 depends on the row, so that eight lanes' reads lie
// in all banks, and so do their writes (64 elements a head: only the writes).
template <int HD>
__device__ __forceinline__ void decode_keys(const uint8_t *rec, uint8_t *tile, int page, int lane) {
  constexpr int C = HD / 32;                         // lanes of a row
  constexpr int RPI = 32 / C;                        // rows in a step
#pragma unroll
  for (int i = 0; i < kPage / RPI; ++i) {
    const int r = i * RPI + lane % RPI, row = page * kPage + r;
    const int c = HD == 128 ? (lane / RPI) ^ ((r >> 1) & 3) : lane / RPI;
    const uint4 w = *reinterpret_cast<const uint4 *>(rec + r * (HD / 2) + c * 16);
    const uint32_t two = *reinterpret_cast<const uint16_t *>(rec + Record<HD>::kKs + r * (HD / 16) + 2 * c);
    const uint32_t s0 = scale4_twice(two, 0), s1 = scale4_twice(two, 1);
    uint8_t *dst = tile + (c >> 1) * Smem<HD>::kHalf;
    const int c0 = (c & 1) * 4;
    *reinterpret_cast<uint4 *>(dst + swz(row, c0)) = mul4(unpack_e2m1x8(w.x), s0);
    *reinterpret_cast<uint4 *>(dst + swz(row, c0 + 1)) = mul4(unpack_e2m1x8(w.y), s0);
    *reinterpret_cast<uint4 *>(dst + swz(row, c0 + 2)) = mul4(unpack_e2m1x8(w.z), s1);
    *reinterpret_cast<uint4 *>(dst + swz(row, c0 + 3)) = mul4(unpack_e2m1x8(w.w), s1);
  }
}

// A quarter of a block's values to a tile (rows of 64 keys of an element of the
// head, since a byte holds two keys of an element): warp `part` takes four pages
// and half of the elements, a lane eight keys of 16 elements (of 8 with 64 elements
// a head).  The four pairs of keys that make 16 bytes of a row stand there in
// the order 0..3 xor (chunk mod 4), which lets eight lanes read from all banks; the
// weights stand in that order too.  valid, gone: keys and pages that count.
__host__ __device__ constexpr int pair_slot(int chunk, int pair) { return pair ^ (chunk & 3); }
template <int HD>
__device__ __forceinline__ void decode_values(const uint8_t *stage, uint8_t *tile, int part, int valid, uint32_t gone, int lane) {
  using R = Record<HD>;
  constexpr int W = HD / 32;                         // words of a pair
  const int cc = lane & 7, chunk = 8 * (part >> 1) + cc, page = chunk >> 1;
  const int step = HD == 128 ? part & 1 : lane >> 4;
  const int g = 2 * (HD == 128 ? lane >> 3 : (lane >> 3) & 1) + (step ^ (cc >> 2));      // group of 16 elements
  const int w0 = HD == 128 ? 0 : 2 * (part & 1);     // first word of the group
  const uint8_t *rec = stage + page * R::kBytes;
  const bool whole = valid >= kKeys && gone == 0u;
  uint32_t k[4][W], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pr = 4 * (cc & 1) + pair_slot(cc, i);
    const uint8_t *src = rec + R::v_at(pr, g) + 4 * w0;
    if constexpr (W == 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(src);
      k[i][0] = v.x; k[i][1] = v.y; k[i][2] = v.z; k[i][3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2 *>(src);
      k[i][0] = v.x; k[i][1] = v.y;
    }
    s[i] = scale4_pair(*reinterpret_cast<const uint16_t *>(rec + R::vs_at(pr, g)));
    if (!whole) {                                    // no key, no value: not even a NaN
      const int key = page * kPage + 2 * pr, n = (gone >> page) & 1u ? 0 : valid;
      s[i] &= (key < n ? 0xffffu : 0u) | (key + 1 < n ? 0xffff0000u : 0u);
    }
  }
  uint8_t *dst = tile + (part >> 1) * (HD * 128);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    uint4 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = mul4(unpack_e2m1x8(k[i][w]), s[i]);
    const int row = 16 * g + 4 * (w0 + w);
    *reinterpret_cast<uint4 *>(dst + swz(row, cc)) = make_uint4(h[0].x, h[1].x, h[2].x, h[3].x);
    *reinterpret_cast<uint4 *>(dst + swz(row + 1, cc)) = make_uint4(h[0].y, h[1].y, h[2].y, h[3].y);
    *reinterpret_cast<uint4 *>(dst + swz(row + 2, cc)) = make_uint4(h[0].z, h[1].z, h[2].z, h[3].z);
    *reinterpret_cast<uint4 *>(dst + swz(row + 3, cc)) = make_uint4(h[0].w, h[1].w, h[2].w, h[3].w);
  }
}

// Whole warp: phases of two or three barriers.  All are tested before one is waited
// for: a wait takes some 200 cycles even when its phase is complete, as it mostly is.
struct Phase {
  uint32_t bar, parity;
};
__device__ __forceinline__ bool wait_all(uint32_t polls, Phase a, Phase b, Phase c) {
  const bool x = mbar_test(a.bar, a.parity), y = mbar_test(b.bar, b.parity), z = mbar_test(c.bar, c.parity);
  return __all_sync(0xffffffffu, x && y && z) ||
         (mbar_wait_warp(a.bar, a.parity, polls) && mbar_wait_warp(b.bar, b.parity, polls) && mbar_wait_warp(c.bar, c.parity, polls));
}
__device__ __forceinline__ bool wait_all(uint32_t polls, Phase a, Phase b) {
  const bool x = mbar_test(a.bar, a.parity), y = mbar_test(b.bar, b.parity);
  return __all_sync(0xffffffffu, x && y) || (mbar_wait_warp(a.bar, a.parity, polls) && mbar_wait_warp(b.bar, b.parity, polls));
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
  float *new_down_s = reinterpret_cast<float *>(sb + L::kOffNewDown), *new_share_s = new_down_s + kMaxNew;
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
  const bool producer = warp == 0 || warp == kSecondProducer;
  const int odd_blocks = warp == 0 ? 0 : 1;  // a producer's blocks: every other one
  int pages[kStages / 2];
  constexpr int CH = HD / 8;                 // 16-byte chunks of a bf16 row
  if (producer) {
#pragma unroll
    for (int d = 0; d < kStages / 2; ++d) pages[d] = block_page(2 * d + odd_blocks);
  } else if (prep_warp) {
    // the query rows (a token's heads lie together) and the new tokens' keys and
    // values come first of all, ahead of the stream of codes: one bulk copy each,
    // a few of them a warp (a warp issues its lanes' one after another)
    const int rows = min(kRows, w.M - w.row0), news = fresh ? w.n : 0;
    if (pt == 0) {
      mbar_init(bar(kBarRaw), 1);
      fence_barrier_init();
      mbar_arrive_expect_tx(bar(kBarRaw), (uint32_t)(rows + 2 * news) * HD * 2);
    }
    named_sync(1, kPrep);
    const int tok0 = div_by(w.row0, a.by_G), n_tok = div_by(w.row0 + rows - 1, a.by_G) - tok0 + 1;
    for (int e = (warp - kSoftmaxWarp) + 16 * lane; e < n_tok + 2 * news; e += 16 * 32) {
      const __nv_bfloat16 *src;
      uint32_t dst, bytes = HD * 2;
      if (e < n_tok) {
        const int t = tok0 + e, lo = max(w.row0, t * a.G), hi = min(w.row0 + rows, (t + 1) * a.G);
        src = (const __nv_bfloat16 *)a.q + (t0 + t) * a.q_row + w.kvh * a.G * HD + (lo - t * a.G) * HD;
        dst = L::kOffRaw + (lo - w.row0) * HD * 2;
        bytes *= hi - lo;
      } else {
        const int i = e - n_tok, j = i < news ? i : i - news;
        src = (i < news ? (const __nv_bfloat16 *)a.k_new + (t0 + j) * a.k_row : (const __nv_bfloat16 *)a.v_new + (t0 + j) * a.v_row) + w.kvh * HD;
        dst = L::kOffNew + (i < news ? j : kMaxNew + j) * HD * 2;
      }
      bulk_load(base + dst, src, bytes, bar(kBarRaw));
    }
    // angles of the new tokens' positions (identity past the rotated part)
    float2 *cs_s = reinterpret_cast<float2 *>(sb + L::kOffCs);            // [kMaxNew][HD / 2]
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
  }
  if (warp == kPvWarp) {
    for (int i = lane; i < kBarRaw; i += 32) {      // (that one is made)
      const bool rows = i >= kBarPFull && i < kBarPFull + kPvBars;
      const bool tiles = i >= kBarKbFull && i < kBarVbFull + 2;
      mbar_init(bar(i), rows ? n_valid : tiles ? kDecoders : i >= kBarEmpty && i < kBarEmpty + kStages ? 2 * kDecoders
                      : i == kBarQReady ? 4 : i == kBarNewRead ? kDecoders : 1);
    }
    if (lane == 0) {
      *flag_s = 0;
      odd_s[0] = odd_s[1] = 0u;
    }
    for (int i = lane; i < kKeys; i += 32) new_kv_s[i] = make_float2(0.f, 0.f);
    for (int i = lane; i < kMaxNew; i += 32) new_down_s[i] = new_share_s[i] = 0.f;
    fence_barrier_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  int issued = 0;                            // producers: blocks whose loads were started
  const float2 *cs_s = reinterpret_cast<const float2 *>(sb + L::kOffCs);
  auto pv_done = [&](int j) { return Phase{bar(kBarPvDone + (j & (kPvBars - 1))), (uint32_t)(j / kPvBars) & 1u}; };
  auto p_full = [&](int j) { return Phase{bar(kBarPFull + (j & (kPvBars - 1))), (uint32_t)(j / kPvBars) & 1u}; };
  auto two = [&](int first, int j) { return Phase{bar(first + (j & 1)), (uint32_t)(j >> 1) & 1u}; };   // of a pair of barriers
  auto give_up = [&]() { raise_status(a.status, kStatusTimeout); atomicOr(flag_s, 1); };
  // An issuing warp stays until its last product is done (default limit): after a
  // wait that gave up elsewhere nobody else waits for it, and the tiles and tensor
  // memory that it uses go with the CTA.
  auto drain = [&](int sent, auto phase) {
    if (sent > 0) (void)mbar_wait_warp(phase(sent - 1).bar, phase(sent - 1).parity);
  };
  // These warps together rotate the query rows and, in the CTA that owns the new
  // tokens, their keys, to f16 relative to a power of two of each row's; rolled
  // loops, since each CTA runs them once.
  auto prepare = [&]() {
    if (!mbar_wait_warp(bar(kBarRaw), 0, a.polls) && lane == 0) give_up();
    const __nv_bfloat16 *ks = reinterpret_cast<const __nv_bfloat16 *>(sb + L::kOffNew), *vs = ks + kMaxNew * HD;
    if (fresh) {                             // each token's ve: its largest finite value (CH lanes hold its row)
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
          const int ve = value_exponent(va);
          new_kv_s[e / CH].y = (float)ve;
          new_down_s[e / CH] = pow2i(-ve);
          new_share_s[e / CH] = kShareLift - (float)ve;
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
      if (query ? row >= w.M : r >= w.n) {
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

  if (producer) {
    // --------------------------------------------------------- producers
    bool ok = true;
    for (int j0 = odd_blocks; ok && j0 < n_past; j0 += kStages) {
#pragma unroll
      for (int d = 0; d < kStages / 2; ++d) {
        const int j = j0 + 2 * d, s = 2 * d + odd_blocks;                  // s: stage of block j
        if (j >= n_past) break;
        const int page = pages[d];
        const bool there = lane < kPagesPerBlock && in_cache(page);
        const uint32_t have = __ballot_sync(0xffffffffu, there);
        // (the last two stages hold the new tokens until they are converted)
        if ((j >= kStages && !mbar_wait_warp(bar(kBarEmpty + s), ((j / kStages) - 1) & 1, a.polls)) ||
            (j >= kStages - 2 && j < kStages && fresh && !mbar_wait_warp(bar(kBarNewRead), 0, a.polls))) {
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
        pages[d] = block_page(j + kStages);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- scores
    // The whole warp keeps the loop (uniform addresses), one lane issues.
    static_assert(kMaxNew <= (int)kUnitCols, "the new tokens are one unit");
    constexpr uint32_t idS = tc::idesc_f16(kRows, kUnitCols, 0);
    const uint64_t dK0 = tc::smem_desc_sw128(base + L::kOffKb, 16, 1024);
    auto score = [&](uint32_t tS, int at) {       // 64 keys, from byte `at` of the tiles on
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
        tc::mma_bf16_ts(tS, tmem + L::kColQ + kk * 8,
                        dK0 + ((uint32_t)(at + (kk >> 2) * L::kHalf + (kk & 3) * 32) >> 4), idS, kk > 0);
    };
    bool ok = mbar_wait_warp(bar(kBarQReady), 0, a.polls);
    int sent = 0;                            // blocks whose products were issued
    for (int j = 0; ok && j < n_blocks; ++j) {
      const int tb = j & 1;
      const Phase keys = two(kBarKbFull, j), weights = p_full(j - 2);
      ok = j < 3 ? mbar_wait_warp(keys.bar, keys.parity, a.polls) && (j < 2 || mbar_wait_warp(weights.bar, weights.parity, a.polls))
                 : wait_all(a.polls, pv_done(j - 3), keys, weights);
      if (!ok) break;
      tc::fence_after_sync();
      if (tc::elect_one()) {
        score(tmem + unit_col(j, 0), tb * L::kTile);
        if (j >= fresh) score(tmem + unit_col(j, 1), tb * L::kTile + 64 * 128);
        tc::commit(bar(kBarSFull + tb));
      }
      __syncwarp();
      sent = j + 1;
    }
    if (!ok && lane == 0) give_up();
    drain(sent, [&](int j) { return two(kBarSFull, j); });
  } else if (warp == kPvWarp) {
    // ---------------------------------------------------------------- P V
    constexpr uint32_t idO = tc::idesc_f16(kRows, HD, 0);
    auto value_at = [](int kk) { return (uint32_t)((kk >> 2) * (HD * 128) + (kk & 3) * 32) >> 4; };
    const uint64_t dV0 = tc::smem_desc_sw128(base + L::kOffVb, 16, 1024);
    bool ok = true;
    int sent = 0;
    for (int j = 0; j < n_blocks; ++j) {
      const int tb = j & 1, jp = j - fresh;
      ok = wait_all(a.polls, two(kBarVbFull, j), p_full(j));
      if (!ok) break;
      tc::fence_after_sync();
      const int depth = jp < 0 ? n_pad : min(kKeys, (w.k_end - w.k_begin - jp * kKeys + 15) & ~15);
      const uint64_t dV = dV0 + ((uint32_t)(tb * L::kTile) >> 4);
      const uint32_t tP = tmem + unit_col(j, 0);
      if (tc::elect_one()) {
        if (depth == kKeys) {
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            tc::mma_bf16_ts(tmem + kColO, tP + weight_col(16 * kk), dV + value_at(kk), idO, j > 0 || kk > 0);
        } else {
          for (int kk = 0; kk < depth / 16; ++kk)
            tc::mma_bf16_ts(tmem + kColO, tP + weight_col(16 * kk), dV + value_at(kk), idO, j > 0 || kk > 0);
        }
        tc::commit(bar(kBarPvDone + (j & (kPvBars - 1))));
      }
      __syncwarp();
      sent = j + 1;
    }
    if (!ok && lane == 0) give_up();
    drain(sent, pv_done);
  } else if (warp >= kDecodeWarp) {
    // ------------------------------------------------------------- decode
    const bool values = warp >= kValueWarp;
    const int part = warp - (values ? kValueWarp : kDecodeWarp);            // this warp's quarter of every block
    prepare();
    // (the tiles hold the angles and rows until the query is in TMEM)
    bool ok = mbar_wait_warp(bar(kBarQReady), 0, a.polls);
    if (ok && fresh && !values && lane == 0) mbar_arrive(bar(kBarKbFull));          // the new keys are the first key tile
    if (ok && fresh && values) {             // the new values, as f16, are the first value tile
      const __nv_bfloat16 *vs = reinterpret_cast<const __nv_bfloat16 *>(sb + L::kOffNew) + kMaxNew * HD;
#pragma unroll 1
      for (int e = threadIdx.x - 32 * kValueWarp; e < n_pad / 2 * CH; e += 32 * kDecoders) {
        const int c = e / (n_pad / 2), j = 2 * (e - c * (n_pad / 2));       // a pair of tokens
        float v[2][8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float vdown = new_down_s[j + t];
          load_vec<__nv_bfloat16, 8>(vs + (j + t) * HD + c * 8, v[t]);
#pragma unroll
          for (int i = 0; i < 8; ++i)        // (an odd one times a weight of 0 would reach every row)
            v[t][i] = j + t < w.n && fabsf(v[t][i]) < INFINITY ? v[t][i] * vdown : 0.f;
        }
        uint8_t *dst = sb + L::kOffVb + 4 * pair_slot(j >> 3, (j >> 1) & 3);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint32_t *>(dst + swz(8 * c + i, j >> 3)) = pack_f16x2(v[0][i], v[1][i]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kBarNewRead));
        mbar_arrive(bar(kBarVbFull));
      }
    }
    // a tile is free when the product that read it is done: scores for keys, P V for values
    const int full_bar = values ? kBarVbFull : kBarKbFull;
    for (int jp = 0; ok && jp < n_past; ++jp) {
      const int j = jp + fresh, tb = j & 1, s = jp & (kStages - 1);
      const Phase full = {bar(kBarFull + s), (uint32_t)(jp / kStages) & 1u};
      ok = j < 2 ? mbar_wait_warp(full.bar, full.parity, a.polls) : wait_all(a.polls, full, values ? pv_done(j - 2) : two(kBarSFull, j - 2));
      if (!ok) break;
      const uint8_t *stage = sb + L::kOffRing + s * L::kStage;
      uint8_t *tile = sb + (values ? L::kOffVb : L::kOffKb) + tb * L::kTile;
      if (values) {
        decode_values<HD>(stage, tile, part, w.k_end - w.k_begin - jp * kKeys, gone_s[jp & (kGone - 1)], lane);
      } else {
#pragma unroll
        for (int i = 0; i < kPagesPerWarp; ++i)
          decode_keys<HD>(stage + (part * kPagesPerWarp + i) * L::kRec, tile, part * kPagesPerWarp + i, lane);
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
    auto pair_any = [&](bool x) {            // of the two warps that share a row
      uint32_t r;
      asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                   : "=r"(r) : "r"((uint32_t)x), "r"(4 + q4) : "memory");
      return r != 0u;
    };
    auto pair_sync = [&]() { named_sync(4 + q4, 64); };
    const uint64_t newvis = fresh ? kvq_visible(a, w.B, tau_s, tok) : 0ull;
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
    const uint32_t tO = trow + kColO;
    // a row that sees a new token with an odd value is NaN
    const bool odd = (newvis & ((uint64_t)odd_s[1] << 32 | odd_s[0])) != 0ull;
    float m_ref = -INFINITY, l = odd ? __uint_as_float(0x7fc00000u) : 0.f;
    bool ok = true, next_ready = false;
    int j = 0;
    // the key loop, compiled once per copy count, the new tokens' block by itself
    // (a factor and a ve for each key)
    auto key_loop = [&](auto rc) {
      constexpr int RC = decltype(rc)::value;
      constexpr int KW = kKeys / (RC * kHalves);   // this warp's keys per block: 64, 32 or 16
      // keys k_lo .. (with 64 of them: 32 there, and 32 in the second unit)
      const int k_lo = RC == 4 ? 64 * (kp >> 1) + 32 * half + 16 * (kp & 1) : 64 * kp + 32 * half;
      // A warp whose wait gave up still meets its partner once, with a NaN in
      // the maximum's place (a maximum is never NaN), so both leave the loop.
      auto block = [&](auto newc) {            // block j; false: leave the loop
        constexpr bool is_new = decltype(newc)::value != 0;
        const int tb = is_new ? 0 : j & 1, jp = is_new ? -1 : j - fresh;
        const uint32_t tS[2] = {trow + unit_col(j, k_lo >> 6) + (k_lo & 63), trow + unit_col(j, 1) + (k_lo & 63)};
        // keys that count: all of a whole block's, else one bit each
        const int valid = is_new ? 0 : w.k_end - w.k_begin - jp * kKeys;
        ok = ok && (next_ready || mbar_wait_warp(bar(kBarSFull + tb), (j >> 1) & 1, a.polls));
        const uint32_t gone = is_new || !ok ? 0u : gone_s[jp & (kGone - 1)];
        const bool whole = !is_new && valid >= kKeys && gone == 0u;
        const float f = whole ? rscale : 1.f;      // t = f s
        tc::fence_after_sync();
        // the scores of this warp's keys, 32 at a time (q: those of the second
        // unit); where some do not count, as t with -inf for those
        constexpr int CW = KW < 32 ? KW : 32;
        uint32_t sr[CW];
        auto fetch = [&](int q) {
          if constexpr (CW == 16) tc::ld16(tS[q], sr);
          else tc::ld32(tS[q], sr);
          tc::wait_ld();
          if (whole) return;
          const int k0 = k_lo + 64 * q;
          if (is_new) {
            const uint32_t v = (uint32_t)shift_right(newvis, k0);
#pragma unroll
            for (int i = 0; i < CW; i += 8) {
              if (k0 + i >= w.n) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sr[i + e] = __float_as_uint(-INFINITY);
                continue;
              }
              float4 x[4];                   // of two keys each
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = load_shared4(base + L::kOffNewKv + (k0 + i + 2 * e) * 8);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t *t = sr + i + 2 * e;
                t[0] = __float_as_uint((v >> (i + 2 * e)) & 1u ? fmaf(__uint_as_float(t[0]), x[e].x * rscale, x[e].y) : -INFINITY);
                t[1] = __float_as_uint((v >> (i + 2 * e)) & 2u ? fmaf(__uint_as_float(t[1]), x[e].z * rscale, x[e].w) : -INFINITY);
              }
            }
          } else {
            uint32_t v = (uint32_t)kvq_low_bits(valid - k0);
            for (int i = 0; i < CW / 16; ++i)
              if ((gone >> (k0 / 16 + i)) & 1u) v &= ~(0xffffu << (16 * i));
#pragma unroll
            for (int i = 0; i < CW; ++i)
              sr[i] = __float_as_uint((v >> i) & 1u ? __uint_as_float(sr[i]) * rscale : -INFINITY);
          }
        };
        // weights 2^(t - mu) as f16 pairs, in the values' order, and their sum
        uint32_t pw[KW / 2];
        float2 sum;
        auto weigh = [&](float mu, bool held) {      // held: sr holds the (only) scores
          const float2 f2 = make_float2(f, f), b2 = make_float2(-mu, -mu);
          sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int q = 0; q < KW / CW; ++q) {
            if (is_new && k_lo + 64 * q >= w.n) {
#pragma unroll
              for (int e = 0; e < CW / 2; ++e) pw[CW / 2 * q + e] = 0u;
              continue;
            }
            if (!held) fetch(q);
            float4 sh;                       // the new tokens' share of the sum
#pragma unroll
            for (int e = 0; e < CW / 2; ++e) {
              const float2 x = fma_f32x2(make_float2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), f2, b2);
              const float2 p = make_float2(ex2(x.x), ex2(x.y));
              if (is_new) {
                if (e % 2 == 0) sh = load_shared4(base + L::kOffNewShare + (k_lo + 64 * q + 2 * e) * 4);
                const float2 y = add_f32x2(x, e % 2 == 0 ? make_float2(sh.x, sh.y) : make_float2(sh.z, sh.w));
                sum = add_f32x2(sum, make_float2(ex2(y.x), ex2(y.y)));
              } else {
                sum = add_f32x2(sum, p);
              }
              pw[CW / 2 * q + (e & ~3) + pair_slot(e >> 2, e & 3)] = pack_f16x2(p.x, p.y);
            }
          }
          if constexpr (CW == 16) {          // (chunks 2 and 3 of 32 keys)
            if (kp & 1) {
#pragma unroll
              for (int e = 0; e < 8; e += 4) {
                const uint32_t x = pw[e], y = pw[e + 1];
                pw[e] = pw[e + 2]; pw[e + 1] = pw[e + 3];
                pw[e + 2] = x; pw[e + 3] = y;
              }
            }
          }
        };
        // Mostly the reference holds, which a row's sum shows: no weight of a sum
        // of at most 2^15 is above that.
        bool moves = true;
        if (!is_new && j > fresh) {          // (the first of the prompt's moves it)
          if (ok) weigh(m_ref, false);
          moves = pair_any(!ok || (row_valid && !(m_ref > -INFINITY && sum.x + sum.y <= kMostSum)));
        }
        if (moves) {
          // the row's maximum over both warps' keys
          float mx = -INFINITY;
#pragma unroll
          for (int q = 0; q < KW / CW; ++q) {
            if (!ok || (is_new && k_lo + 64 * q >= w.n)) break;
            fetch(q);
#pragma unroll
            for (int i = 0; i < CW; ++i) mx = fmaxf(mx, __uint_as_float(sr[i]) * f);
          }
          both_s[(tb * kHalves + half) * kRows] = ok ? mx : __uint_as_float(0x7fc00000u);
          pair_sync();
          const float theirs = both_s[(tb * kHalves + (half ^ 1)) * kRows];
          if (!ok || theirs != theirs) { ok = false; return false; }
          mx = fmaxf(mx, theirs);
          constexpr float lift = is_new ? kNewLift : kLift;
          const bool move = row_valid && mx > m_ref + lift;
          const float m_new = move ? mx - lift : m_ref;
          const float alpha = move ? ex2(m_ref - m_new) : 1.f;     // m_ref = -inf -> 0
          l *= alpha;
          m_ref = m_new;
          // O's rows may be scaled once the previous block's P V is done
          if (!is_new && __any_sync(0xffffffffu, move) && j > 0) {
            if (!mbar_wait_warp(bar(kBarPvDone + ((j - 1) & (kPvBars - 1))), ((j - 1) / kPvBars) & 1, a.polls)) { ok = false; return true; }
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
          weigh(m_ref == -INFINITY ? 0.f : m_ref, is_new || KW == CW);
        }
        // they go over the first unit's scores, zeros for the other copies' keys
        const uint32_t tW = trow + unit_col(j, 0) + 32 * half;
        if constexpr (RC > 1) {
          uint32_t z[KW / 2];
#pragma unroll
          for (int e = 0; e < KW / 2; ++e) z[e] = 0u;
#pragma unroll
          for (int c = 1; c < RC; ++c) {
            const uint32_t at = tW + (kp + c) % RC * (KW / 2);
            if constexpr (KW == 16) tc::st8(at, z);
            else tc::st16(at, z);
          }
        }
        if constexpr (KW == 16) tc::st8(tW + kp * 8, pw);
        else if constexpr (KW == 32) tc::st16(tW + kp * 16, pw);
        else tc::st32(tW, pw);
        l = is_new ? fmaf(sum.x + sum.y, kShareUnlift, l) : l + (sum.x + sum.y);
        const Phase after = two(kBarSFull, j + 1);                         // (a test's latency passes here)
        const bool there = mbar_test(after.bar, after.parity);
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        next_ready = __all_sync(0xffffffffu, there);
        if (lane == 0) mbar_arrive(p_full(j).bar);
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
    if (ok && j > 0 && !mbar_wait_warp(bar(kBarPvDone + ((j - 1) & (kPvBars - 1))), ((j - 1) / kPvBars) & 1, a.polls)) ok = false;
    if (!ok && lane == 0) give_up();
    tc::fence_after_sync();
    // -------------------------------------------------------- epilogue
    // Every row, and every copy of one, puts its output, reference and sums into
    // the idle ring; then a warp takes four rows at a time, so that it writes whole lines.
    constexpr int LD = HD + 4;
    float *part = reinterpret_cast<float *>(sb + L::kOffRing);   // [R][groups * 32][LD]
    if (warp_valid) {
      float *mine = part + ((kp * groups + g) * 32 + lane) * LD;
#pragma unroll 1
      for (int c0 = half * (HD / 2); c0 < (half + 1) * (HD / 2); c0 += 32) {
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
      else mine[HD + 2] = l;
    }
    named_sync(3, 8 * 32);
    const int n_rows = *(volatile int *)flag_s != 0 ? 0 : min(32 * groups, w.M - w.row0);
    const int ln = lane & 7;                 // eight lanes a row, four columns of every 32 each
    for (int r0 = 4 * (warp - kSoftmaxWarp); r0 < n_rows; r0 += 4 * 8) {
      const int r = r0 + (lane >> 3);
      if (r >= n_rows) continue;
      const float *row = part + r * LD;      // copy 0; the others follow
      const int next = groups * 32 * LD;
      float4 ml[4], v[HD / 32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        ml[c] = c < R ? *reinterpret_cast<const float4 *>(row + c * next + HD) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      const float mt = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
      float lt = 0.f;
#pragma unroll
      for (int k = 0; k < HD / 32; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c >= R) break;
        const float wc = ex2_low(ml[c].x - (mt == -INFINITY ? 0.f : mt));   // -inf reference -> 0; below the normal range too
        lt = fmaf(wc, ml[c].y + ml[c].z, lt);
#pragma unroll
        for (int k = 0; k < HD / 32; ++k) {
          const float4 x = *reinterpret_cast<const float4 *>(row + c * next + 32 * k + 4 * ln);
          v[k] = make_float4(fmaf(wc, x.x, v[k].x), fmaf(wc, x.y, v[k].y), fmaf(wc, x.z, v[k].z), fmaf(wc, x.w, v[k].w));
        }
      }
      const int at = w.row0 + r, token = div_by(at, a.by_G);
      const int64_t orow = (t0 + token) * a.Hq + w.kvh * a.G + at - token * a.G;
      if (w.n_splits == 1) {
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        uint2 *dst = reinterpret_cast<uint2 *>((__nv_bfloat16 *)a.out + orow * HD) + ln;
#pragma unroll
        for (int k = 0; k < HD / 32; ++k)
          dst[8 * k] = make_uint2(pack_bf16x2(v[k].x * inv, v[k].y * inv), pack_bf16x2(v[k].z * inv, v[k].w * inv));
      } else {
        const int64_t prow = (int64_t)w.split * a.T * a.Hq + orow;
        float4 *dst = reinterpret_cast<float4 *>(a.o_part + prow * HD) + ln;
#pragma unroll
        for (int k = 0; k < HD / 32; ++k) dst[8 * k] = v[k];
        if (ln == 0) a.ml_part[prow] = make_float2(mt, lt);
      }
    }
  }
  // -------------------------------------------------------------- teardown
  tc::fence_before_sync();
  __syncthreads();
  // after a wait that gave up, the copies still in flight land before the CTA
  // can exit (default limit)
  if (producer && *(volatile int *)flag_s) {
    (void)mbar_wait_warp(bar(kBarRaw), 0);
    for (int j = issued - 3; j < issued; j += 2)         // (issued: the last one's number and 1)
      if (j >= 0) (void)mbar_wait_warp(bar(kBarFull + j % kStages), (j / kStages) & 1);
  }
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
