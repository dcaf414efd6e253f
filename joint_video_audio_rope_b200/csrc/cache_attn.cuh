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
// weights as p' / vs.  So p' is measured against what the row's largest term adds to
// the output, and the result needs no pass over V's values.  A V scale of 0 (zeros, whatever
// the codes) is taken as the smallest one, 2^-60, over codes of zero: it counts in the
// sum of weights and must not raise m, which would push the other terms out of fp16.
#pragma once

#include "cache.cuh"

namespace mmdit {

struct CacheAttnArgs {
  const void* q;
  void* o;
  float* lse;
  long long q_st, q_sb, o_st, o_sb;  // strides in elements
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  const int32_t *table, *kv_len, *q_len;
  int n_pages, page, page_log2, max_pages;
  int B, N, H, Hk, G;   // G = H / Hk
  uint32_t g_mul;       // r / G = (mulhi(r, g_mul) + r) >> g_shift for r < 2^31
  int g_shift;
  int causal;
  float scale_log2;
  // Items: one tile of rows of one (item, K/V head).  The first `whole` of them
  // are one CTA each; each of the others is split into `splits` key ranges.
  int tiles;           // row tiles per (item, K/V head)
  int whole, splits;
  float* part_o;       // [item - whole][split][tile rows][D], unnormalised
  float* part_ml;      // [item - whole][split][tile rows][2]: maximum (log2) and sum
  int* err;
};

// Rows per CTA: 8 or 16 (few rows, and every fp32 call: cache_attn.cu), or this (many
// bf16 rows, on tcgen05: cache_attn_tc.cu).
constexpr int kManyTile = 256;
constexpr int kUnit = 128;      // tokens: granularity of the split key ranges
constexpr float kNoScaleLog2 = -60.f;                  // of a V scale of 0
constexpr float kNoScaleInverse = 1152921504606846976.f;  // 2^60

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
// Token of row r; its query head is hk G + r - token G.  (A division costs as much as the
// row's load; a tile has 256 rows to address.)
__device__ __forceinline__ int row_token(const CacheAttnArgs& A, int r) {
  return (int)((__umulhi((uint32_t)r, A.g_mul) + (uint32_t)r) >> A.g_shift);
}
// Page of token n of item b, or -1 (nothing to see there): ids outside the cache stand for
// pages that are not there, so the device-checked build does not report them either.
__device__ __forceinline__ int page_of(const CacheAttnArgs& A, int b, int n) {
  const int id = __ldg(A.table + (long long)b * A.max_pages + (n >> A.page_log2));
  return (id >= 0 && id < A.n_pages) ? id : -1;
}

// What one CTA works on.
struct CacheItem {
  int b, hk, r0, live;  // rows r0 .. r0 + live - 1
  int kv, ql;
  int lo, hi;           // key range
  long long part;       // partial result, or -1: the item is whole
};
// Row tiles from the last to the first: with causal_block the last ones see the
// most keys, and the longest items are best started first.
__device__ __forceinline__ void item_rows(const CacheAttnArgs& A, int i, int tile, int& b, int& hk,
                                          int& r0) {
  r0 = (A.tiles - 1 - i % A.tiles) * tile;
  i /= A.tiles;
  hk = i % A.Hk;
  b = i / A.Hk;
}
__device__ __forceinline__ CacheItem item_of(const CacheAttnArgs& A, int i, int tile) {
  CacheItem w;
  int split = 0, splits = 1;
  w.part = -1;
  if (i >= A.whole) {
    w.part = i - A.whole;
    splits = A.splits;
    split = (i - A.whole) % splits;
    i = A.whole + (i - A.whole) / splits;
  }
  item_rows(A, i, tile, w.b, w.hk, w.r0);
  w.kv = held_tokens(A, w.b);
  w.ql = query_tokens(A, w.b);
  w.live = min(tile, w.ql * A.G - w.r0);
  w.lo = w.hi = 0;
  if (w.live > 0) {
    const int keys = visible_keys(A, w.kv, w.ql, row_token(A, w.r0 + w.live - 1));
    const int units = (keys + kUnit - 1) / kUnit, per = (units + splits - 1) / splits;
    w.lo = min(keys, split * per * kUnit);
    w.hi = min(keys, w.lo + per * kUnit);
  }
  return w;
}

// 2^k that brings |x| <= amax to at most 2^15 (1 where amax is 0, infinite or NaN).
__device__ __forceinline__ float fit_half(float amax) {
  if (!(amax > 0.f && amax <= 3.402823466e38f)) return 1.f;
  const int e = (__float_as_int(amax) >> 23) - 127;  // amax < 2^(e+1)
  return __int_as_float((min(max(14 - e, -126), 126) + 127) << 23);
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Natural logarithm of a row's sum of exponentials from its reference (log2) and its sum, in
// which V's scale left up to 60 octaves each, of opposite sign: the sum's exponent joins
// the reference first, so that only the result is rounded.
__device__ __forceinline__ float row_lse(float m, float l) {
  if (l == 0.f) return -INFINITY;
  const int bits = __float_as_int(l);
  if ((bits & 0x7f800000) == 0x7f800000) return l + m;  // no number
  const float whole = m + (float)((bits >> 23) - 127);
  return (whole + log2f(__int_as_float((bits & 0x7fffff) | 0x3f800000))) * 0.69314718055994531f;
}

// cp_async16, or zeros if not there.
__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

// bf16 q; `grid` CTAs (cache_attn_tc.cu)
cudaError_t launch_cache_attn_many(const CacheAttnArgs& A, int D, unsigned grid, cudaStream_t s);

}  // namespace mmdit
