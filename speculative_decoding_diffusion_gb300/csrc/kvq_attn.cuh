// kvq_attn.cuh -- what the two kernels of simsd_kvq_verify (tensor cores for
// bf16, CUDA cores for fp32) and their merge share.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "rope_spec.cuh"

namespace simsd {

constexpr int kMaxNew = 64;              // new tokens of a sequence

// Units (sequence, KV head, row tile) run whole or in key splits, as in
// VerifyPlan: the first tail_from whole, each later one in s_tail splits of
// chunk_tail prompt keys.
struct KvqPlan {
  int T, per, G, rows_per_tile, row_tiles;
  int n_splits, tail_from, s_tail, chunk_tail, tail_first, grid;
  bool four;                             // the 4-bit cache
  bool few;                              // of it: the kernel for few rows (launch_kv4_mma)
  int warps;                             // of a CTA (4-bit cache, few rows)
  bool ranked;                           // units by the sequences' lengths (kvq_order_kernel)
  int merge_seqs;                        // sequences (the last in the units' order) with split units
  size_t esize, off_order, off_opart, off_ml, total;
};

struct KvqParams {
  RopePlan plan;
  const void *q, *k_new, *v_new;
  void *out;
  const uint8_t *k_cache, *v_cache, *k_scale, *v_scale;
  const int32_t *block_table, *tau, *lens, *cu_B;
  float *o_part;                         // [n_splits][T][Hq][hd], unnormalised
  int4 *order_ws;                         // [batch] (sequence, first section, sections, prompt), or null
  float2 *ml_part;                       // [n_splits][T][Hq] (log2 reference, sum)
  uint32_t *status;
  int64_t q_row, k_row, v_row;
  int batch, Hq, Hkv, G, T, total_B, B_max, order, node_size, per;
  int max_pages, num_pages;
  int rows_per_tile, row_tiles, tail_from, s_tail, chunk_tail, tail_first, merge_seqs;
  int n_tail, n_whole;                   // CTAs of split units; of them those of whole chunks, which come first
  FastDiv by_seq, by_kv, by_split, by_G, by_node;   // units of a sequence, KV heads, whole chunks of a unit, ..
  uint32_t polls;
  float scale;                           // sm_scale * log2(e)
};

// The sequence, KV head, row tile and split of a CTA, and the keys it owns.
struct KvqWork {
  int b, kvh, rtile, split;
  int c0, B, n, P, M, row0;              // first section entry, sections, new tokens, prompt, rows
  int k_begin, k_end, n_splits;
  bool first;                            // owns the new tokens' keys
  bool ok;                               // there is something to do
};

__device__ __forceinline__ bool kvq_bad(const KvqParams &a, int c0, int B, int P) {
  return B < 1 || B > a.B_max || c0 < 0 || c0 > a.total_B - B || P < 0 ||
         (int64_t)P > (int64_t)a.max_pages * kPage ||
         (a.order == SIMSD_ORDER_NODES && B != div_by(max(B, 0), a.by_node) * a.node_size);
}

// Sequence `rank` of the units' order; its first section, sections and prompt.
__device__ __forceinline__ int4 kvq_sequence(const KvqParams &a, int rank) {
  if (a.order_ws != nullptr) return __ldcg(a.order_ws + rank);
  const int c0 = __ldg(a.cu_B + rank);
  return make_int4(rank, c0, __ldg(a.cu_B + rank + 1) - c0, __ldg(a.lens + rank));
}

__device__ __forceinline__ KvqWork kvq_work(const KvqParams &a) {
  KvqWork w;
  const int ci = blockIdx.x;
  const bool tail = a.tail_first ? ci < a.n_tail : ci >= a.tail_from;
  const int ti = a.tail_first ? ci : ci - a.tail_from;
  // split units: the whole chunks of all of them, then their last ones
  const bool whole = ti < a.n_whole;
  const int of = whole ? div_by(max(ti, 0), a.by_split) : ti - a.n_whole;
  const int unit = !tail ? (a.tail_first ? ci - a.n_tail : ci) : a.tail_from + of;
  const int chunk = tail ? a.chunk_tail : a.max_pages * kPage;
  const int rank = div_by(unit, a.by_seq), in_seq = unit - rank * a.by_seq.d;
  w.split = !tail ? 0 : whole ? ti - of * a.by_split.d : a.by_split.d;
  const int4 seq = kvq_sequence(a, rank);
  w.b = seq.x;
  w.c0 = seq.y;
  w.B = seq.z;
  w.P = seq.w;
  w.rtile = div_by(in_seq, a.by_kv);
  w.kvh = in_seq - w.rtile * a.Hkv;
  w.ok = false;
  if (kvq_bad(a, w.c0, w.B, w.P)) {
    if (threadIdx.x == 0 && w.split == 0 && in_seq == 0) raise_status(a.status, kStatusBadInput);
    return w;
  }
  w.n = a.per * w.B;
  w.M = w.n * a.G;
  w.row0 = w.rtile * a.rows_per_tile;
  w.k_begin = w.split * chunk;
  w.first = w.split == 0;
  w.ok = w.row0 < w.M && (w.first || w.k_begin < w.P);
  w.k_end = min(w.P, w.k_begin + chunk);
  w.n_splits = tail ? max(1, (w.P + chunk - 1) / chunk) : 1;
  return w;
}

// Position of new token `tok` past the prompt.
__device__ __forceinline__ int kvq_offset(const KvqParams &a, int B, int tok) {
  return a.order == SIMSD_ORDER_PAIRED ? (tok < B ? tok : tok - B)
         : a.order == SIMSD_ORDER_NODES ? tok - div_by(tok, a.by_node) * a.node_size : tok;
}

// bits [0, n) set (n clamped to 0..64)
__device__ __forceinline__ uint64_t kvq_low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// The new tokens that row `tok` sees, one bit each; tau_s: labels of the
// sections (paired order).
__device__ __forceinline__ uint64_t kvq_visible(const KvqParams &a, int B, const int *tau_s, int tok) {
  if (a.order == SIMSD_ORDER_CAUSAL) return kvq_low_bits(tok + 1);
  if (a.order == SIMSD_ORDER_NODES)
    return kvq_low_bits(a.node_size) << (div_by(tok, a.by_node) * a.node_size);
  const bool slot = tok >= B;
  const int t = tau_s[slot ? tok - B : tok];
  uint64_t bits = 0;
  for (int j = 0; j < B; ++j) {
    const int tj = tau_s[j];
    if (slot ? tj < t : tj <= t) bits |= 1ull << j;
    if (slot && tj >= t) bits |= 1ull << (B + j);
  }
  return bits;
}

cudaError_t launch_kvq_simt(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a,
                            cudaStream_t stream);
cudaError_t launch_kvq_tc(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a,
                          cudaStream_t stream);
// The 4-bit cache, bf16: rows of a tile for units of up to max_rows rows; up to
// kFewRows of them are launch_kv4_mma's, 128 launch_kv4_tc's.
constexpr int kFewRows = 16;
int kv4_rows_per_tile(int64_t max_rows);
cudaError_t launch_kv4_mma(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a,
                           cudaStream_t stream);
cudaError_t launch_kv4_tc(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a,
                          cudaStream_t stream);
cudaError_t launch_kvq_merge(const simsd_kvq_verify_desc *d, const KvqPlan &p, const KvqParams &a,
                             cudaStream_t stream);

}  // namespace simsd
