// What the two kernels of mmdit_cache_attn share: the problem as the device
// sees it, the lengths and the visible keys of a row, and page look-ups.
//
// Rows.  The query heads that share a K/V head are rows of one problem: row r
// of (item, K/V head hk) is token r / g of query head hk g + r % g, so K and V
// are read once for all g.
//
// Scales.  K's scale multiplies the scores.  V's scale is folded into the
// exponent: with t = s log2(e) + log2(vs) and its running maximum m, the
// kernels form p' = 2^(t - m) <= 1, accumulate p' x code, and the sum of
// weights as p' / vs.  p' is fit for fp16 whatever the scales are, and the
// result needs no pass over V's values.
#pragma once

#include "internal.h"

namespace mmdit {

struct CacheAttnArgs {
  const void* q;
  void* o;
  float* lse;
  long long q_st, q_sb, o_st, o_sb;  // strides in elements
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  const int32_t *table, *kv_len, *q_len;
  int n_pages, page, max_pages;
  int B, N, H, Hk, G;  // G = H / Hk
  int causal;
  int splits;          // key ranges per row tile; > 1: partial results
  float scale_log2;
  float* part_o;       // [splits][B][Hk][rows][D], unnormalised
  float* part_ml;      // [splits][B][Hk][rows][2]: maximum (log2) and sum
  int rows;            // N * G rounded up to whole row tiles
  int* err;
};

__device__ __forceinline__ int held_tokens(const CacheAttnArgs& A, int b) {
  return min(max(A.kv_len[b], 0), A.max_pages * A.page);
}
__device__ __forceinline__ int query_tokens(const CacheAttnArgs& A, int b) {
  return A.q_len ? min(max(A.q_len[b], 0), A.N) : A.N;
}
// Keys that query token i of an item with kv tokens and ql queries sees.
__device__ __forceinline__ int visible_keys(const CacheAttnArgs& A, int kv, int ql, int i) {
  if (A.causal == 0) return kv;
  const int p = kv - ql + i;
  if (p < 0) return 0;
  const long long end = ((long long)(p / A.causal) + 1) * A.causal;
  return end < kv ? (int)end : kv;
}
// Page of token n of item b, or -1 (nothing to see there).
__device__ __forceinline__ int page_of(const CacheAttnArgs& A, int b, int n) {
  const int id = __ldg(A.table + (long long)b * A.max_pages + n / A.page);
  MMDIT_DCHECK(id >= 0 && id < A.n_pages, A.err);
  return (id >= 0 && id < A.n_pages) ? id : -1;
}

// few query rows (cache_attn.cu); many bf16 rows on tcgen05 (cache_attn_tc.cu)
constexpr int kFewTile = 16;
cudaError_t launch_cache_attn_few(const CacheAttnArgs& A, int D, int dtype, cudaStream_t s);

}  // namespace mmdit
