// mmdit_cache_attn: the entry point, the kernel for few query rows, and the
// merge of split key ranges.
//
// Few rows (single tokens, a frame's audio tokens; every fp32 call).  The codes
// are read once and barely used, so the call is bound by HBM: the kernel
// keeps K and V in registers on their way from memory to the tensor cores.  A
// warp owns slabs of S tokens; a thread's 16-byte loads of codes are turned into
// fp16 pairs that are mma.m16n8k16 operands as they stand, because the order of
// channels inside a contraction (K) and of output channels (V) is free:
//   scores  A = Q (16 rows x 16 channels), B = K^T: thread (g, t) of a warp (g =
//           lane / 4, t = lane % 4) holds channels 16 t .. 16 t + 15 of token g;
//           step kk contracts channels 16 t + 4 kk .. + 3 of every t
//   output  A = P (the score fragment as it is), B = V: thread (g, t) holds
//           channels g D/8 .. of tokens 2t, 2t + 1, 2t + 8, 2t + 9; output tile j
//           holds channel g D/8 + j of every g
// e4m3 is exact in fp16.  Q is multiplied by a power of two per row that puts
// its largest value at 2^14..2^15, so bf16 values are exact in fp16 too down
// to 2^-29 of that; fp32 values are split into two fp16 parts (22 bits), and so
// are the probabilities of an fp32 call.  The next slab's loads are in flight
// while the current one is computed.  Each warp runs its own softmax; the CTA's
// warps, then the key ranges, are merged at the end in a fixed order.
#include <math.h>

#include <algorithm>

#include "cache_attn.cuh"

namespace mmdit {

namespace {

constexpr int kFewWarps = 4;
// bf16 rows per (item, K/V head) up to which 16-row tiles are taken
constexpr int kFewRows = 64;
// The largest probability of a row is held as 2^14: fp16 keeps its relative
// precision down to 2^-14, so what is 2^-28 of the largest is still whole.
constexpr float kShift = 14.f;

__device__ __forceinline__ float2 unpack_half2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&x)[4]) {
  if constexpr (sizeof(T) == 2) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  } else {
    const float4 r = *reinterpret_cast<const float4*>(p);
    x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kFewWarps * 32, 2)
    cache_attn_few_kernel(const __grid_constant__ CacheAttnArgs A) {
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int S = kF32 ? 16 : 32;   // tokens per slab
  constexpr int KK = D / 16;          // contraction steps over the channels
  constexpr int KV = D / 64;          // 16-byte code vectors per thread and token of K
  constexpr int NT = D / 8;           // output tiles
  constexpr int VW = D / 32;          // words of codes per thread and token of V
  constexpr int QP = kF32 ? 2 : 1;    // fp16 parts of Q and P
  __shared__ float sm_o[kFewWarps][16][D + 4];
  __shared__ float sm_ml[kFewWarps][16][2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const CacheItem w = item_of(A, blockIdx.x, kFewTile);
  const int b = w.b, hk = w.hk, r0 = w.r0, kv = w.kv, ql = w.ql, live = w.live;
  const int lo = w.lo, hi = w.hi;
  if (live <= 0) return;

  // ---- Q fragments of rows g and g + 8, and the rows' visible keys
  uint32_t qa[QP][KK][4];
  float mul[2];
  int limit[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + g + 8 * i, tok = r / A.G, head = hk * A.G + r % A.G;
    const bool row = g + 8 * i < live;
    limit[i] = row ? visible_keys(A, kv, ql, tok) : 0;
    const T* src = (const T*)A.q + b * A.q_sb + (long long)tok * A.q_st + (long long)head * D;
    float x[KK][4], am = 0.f;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      x[kk][0] = x[kk][1] = x[kk][2] = x[kk][3] = 0.f;
      if (row) load4(src + (kk >> 2) * 64 + t * 16 + (kk & 3) * 4, x[kk]);
#pragma unroll
      for (int j = 0; j < 4; ++j) am = fmaxf(am, fabsf(x[kk][j]));
    }
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
    const float f = fit_half(am);
    mul[i] = A.scale_log2 / f;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x0 = x[kk][2 * j] * f, x1 = x[kk][2 * j + 1] * f;
#pragma unroll
        for (int p = 0; p < QP; ++p) {
          const uint32_t h = pack_half2(x0, x1);
          qa[p][kk][i + 2 * j] = h;
          const float2 y = unpack_half2(h);
          x0 -= y.x;
          x1 -= y.y;
        }
      }
  }

  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  constexpr int HF = S / 16;  // 16-token halves of a slab: one page each at most
  const long long head_bytes = (long long)A.page * D;
  auto find = [&](int n, int (&id)[HF]) {
#pragma unroll
    for (int f = 0; f < HF; ++f) id[f] = n + 16 * f < hi ? page_of(A, b, n + 16 * f) : -1;
  };
  uint4 kr[S / 8][KV];
  uint32_t vr[S / 16][4][VW];
  float ks[HF], vs[HF];
  auto load_k = [&](int n, const int (&id)[HF]) {
#pragma unroll
    for (int nt = 0; nt < S / 8; ++nt) {
      const int tok = n + nt * 8 + g, pg = id[nt >> 1];
      const uint8_t* p = A.k + ((long long)pg * A.Hk + hk) * head_bytes + (tok & (A.page - 1)) * D;
#pragma unroll
      for (int c = 0; c < KV; ++c)
        kr[nt][c] = (pg >= 0 && tok < hi)
                        ? __ldg(reinterpret_cast<const uint4*>(p + c * 64 + t * 16))
                        : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int f = 0; f < HF; ++f)
      ks[f] = id[f] >= 0 ? __ldg(A.k_scale + (long long)id[f] * A.Hk + hk) : 0.f;
  };
  auto load_v = [&](int n, const int (&id)[HF]) {
#pragma unroll
    for (int f = 0; f < HF; ++f) {
      vs[f] = id[f] >= 0 ? __ldg(A.v_scale + (long long)id[f] * A.Hk + hk) : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = n + f * 16 + 2 * t + (i & 1) + (i >> 1) * 8;
        const uint8_t* p = A.v + ((long long)id[f] * A.Hk + hk) * head_bytes +
                           (tok & (A.page - 1)) * D + g * (D / 8);
        const bool in = id[f] >= 0 && tok < hi;
        if constexpr (D == 128) {
          const uint4 w = in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
          vr[f][i][0] = w.x, vr[f][i][1] = w.y, vr[f][i][2] = w.z, vr[f][i][3] = w.w;
        } else {
          const uint2 w = in ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0u, 0u);
          vr[f][i][0] = w.x, vr[f][i][1] = w.y;
        }
      }
    }
  };

  int n = lo + warp * S, id[HF], id2[HF];
  if (n < hi) {
    find(n, id);
    load_k(n, id);
    load_v(n, id);
    find(n + kFewWarps * S, id2);
  }
  for (; n < hi; n += kFewWarps * S) {
    const int n2 = n + kFewWarps * S;
    // ---- scores
    float sc[S / 8][4];
#pragma unroll
    for (int nt = 0; nt < S / 8; ++nt) {
      sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        const uint4& r = kr[nt][kk >> 2];
        const uint32_t w = (kk & 3) == 0 ? r.x : (kk & 3) == 1 ? r.y : (kk & 3) == 2 ? r.z : r.w;
        const uint32_t b0 = half2_of(w & 0xffffu), b1 = half2_of(w >> 16);
#pragma unroll
        for (int p = QP - 1; p >= 0; --p) mma16816(sc[nt], qa[p][kk], b0, b1);
      }
    }
    float kf[HF], lv[HF], iv[HF];
#pragma unroll
    for (int f = 0; f < HF; ++f) {
      kf[f] = ks[f];
      // a page that is not there is not seen; a V scale of 0 stands for zeros
      lv[f] = id[f] < 0 ? -INFINITY : (vs[f] > 0.f ? log2f(vs[f]) : 0.f);
      iv[f] = vs[f] > 0.f ? 1.f / vs[f] : 1.f;
      if (!(vs[f] > 0.f)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int w = 0; w < VW; ++w) vr[f][i][w] = 0u;
      }
    }
    int id3[HF];
    if (n2 < hi) {
      load_k(n2, id2);
      find(n2 + kFewWarps * S, id3);
    }
    // ---- softmax of rows g (i = 0) and g + 8 (i = 1)
    bool grew = false;
    float alpha[2], mref[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < S / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = sc[nt][2 * i + e];
          x = fmaf(x, mul[i] * kf[nt >> 1], lv[nt >> 1]);
          if (n + nt * 8 + 2 * t + e >= limit[i]) x = -INFINITY;
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[i], mx);
      mref[i] = mn == -INFINITY ? 0.f : mn - kShift;
      alpha[i] = mn == -INFINITY ? 1.f : ex2_approx(m[i] - mn);
      grew = grew || mn > m[i];
      m[i] = mn;
    }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        acc[j][0] *= alpha[0];
        acc[j][1] *= alpha[0];
        acc[j][2] *= alpha[1];
        acc[j][3] *= alpha[1];
      }
      l[0] *= alpha[0];
      l[1] *= alpha[1];
    }
    // ---- P and the output
#pragma unroll
    for (int f = 0; f < HF; ++f) {
      uint32_t pa[QP][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // rows g, g + 8 of tokens 2t.., then of 8 + 2t..
        const int i = q & 1, nt = 2 * f + (q >> 1);
        float p0 = ex2_approx(sc[nt][2 * i] - mref[i]);
        float p1 = ex2_approx(sc[nt][2 * i + 1] - mref[i]);
        l[i] = fmaf(p0 + p1, iv[f], l[i]);
#pragma unroll
        for (int p = 0; p < QP; ++p) {
          const uint32_t h = pack_half2(p0, p1);
          pa[p][q] = h;
          const float2 y = unpack_half2(h);
          p0 -= y.x;
          p1 -= y.y;
        }
      }
#pragma unroll
      for (int j = 0; j < NT; j += 4) {
        // four channels of tokens (2t, 2t + 1) and (2t + 8, 2t + 9), as pairs
        const uint32_t a0 = __byte_perm(vr[f][0][j >> 2], vr[f][1][j >> 2], 0x5140);
        const uint32_t a1 = __byte_perm(vr[f][0][j >> 2], vr[f][1][j >> 2], 0x7362);
        const uint32_t c0 = __byte_perm(vr[f][2][j >> 2], vr[f][3][j >> 2], 0x5140);
        const uint32_t c1 = __byte_perm(vr[f][2][j >> 2], vr[f][3][j >> 2], 0x7362);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x = e < 2 ? a0 : a1, y = e < 2 ? c0 : c1;
          const uint32_t b0 = half2_of((e & 1) ? x >> 16 : x & 0xffffu);
          const uint32_t b1 = half2_of((e & 1) ? y >> 16 : y & 0xffffu);
          if constexpr (kF32) {
            // a sum of its own per slab: the long sum is then a rounded fp32 one
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = QP - 1; p >= 0; --p) mma16816(d, pa[p], b0, b1);
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[j + e][c] += d[c];
          } else {
            mma16816(acc[j + e], pa[0], b0, b1);
          }
        }
      }
    }
    if (n2 < hi) load_v(n2, id2);
#pragma unroll
    for (int f = 0; f < HF; ++f) {
      id[f] = id2[f];
      id2[f] = n2 < hi ? id3[f] : -1;
    }
  }

  // ---- the CTA's warps, merged in their order
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (t == 0) {
      sm_ml[warp][g + 8 * i][0] = m[i] - kShift;
      sm_ml[warp][g + 8 * i][1] = l[i];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < NT; j += 4)
        *reinterpret_cast<float4*>(&sm_o[warp][g + 8 * i][(2 * t + e) * (D / 8) + j]) =
            make_float4(acc[j][2 * i + e], acc[j + 1][2 * i + e], acc[j + 2][2 * i + e],
                        acc[j + 3][2 * i + e]);
  }
  __syncthreads();
  constexpr int TPR = kFewWarps * 32 / 16;  // threads per row
  constexpr int W = D / TPR;                // channels per thread
  const int row = threadIdx.x / TPR, c0 = (threadIdx.x % TPR) * 4;
  if (row >= live) return;
  float M = -INFINITY, L = 0.f, out[W];
#pragma unroll
  for (int x = 0; x < kFewWarps; ++x) M = fmaxf(M, sm_ml[x][row][0]);
  const float Mr = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int c = 0; c < W; ++c) out[c] = 0.f;
#pragma unroll
  for (int x = 0; x < kFewWarps; ++x) {
    const float f = ex2_approx(sm_ml[x][row][0] - Mr);
    L = fmaf(f, sm_ml[x][row][1], L);
#pragma unroll
    for (int c = 0; c < W; c += 4) {
      const float4 y = *reinterpret_cast<const float4*>(&sm_o[x][row][c0 + c * TPR]);
      out[c] = fmaf(f, y.x, out[c]);
      out[c + 1] = fmaf(f, y.y, out[c + 1]);
      out[c + 2] = fmaf(f, y.z, out[c + 2]);
      out[c + 3] = fmaf(f, y.w, out[c + 3]);
    }
  }
  const int r = r0 + row;
  if (w.part >= 0) {
    const long long pr = w.part * kFewTile + row;
#pragma unroll
    for (int c = 0; c < W; c += 4)
      *reinterpret_cast<float4*>(A.part_o + pr * D + c0 + c * TPR) =
          make_float4(out[c], out[c + 1], out[c + 2], out[c + 3]);
    if (threadIdx.x % TPR == 0) {
      A.part_ml[2 * pr] = M;
      A.part_ml[2 * pr + 1] = L;
    }
    return;
  }
  const int tok = r / A.G, head = hk * A.G + r % A.G;
  const float inv = L == 0.f ? 0.f : 1.f / L;  // a NaN stays one
  T* dst = (T*)A.o + b * A.o_sb + (long long)tok * A.o_st + (long long)head * D;
#pragma unroll
  for (int c = 0; c < W; c += 4) {
    if constexpr (kF32)
      *reinterpret_cast<float4*>(dst + c0 + c * TPR) =
          make_float4(out[c] * inv, out[c + 1] * inv, out[c + 2] * inv, out[c + 3] * inv);
    else
      *reinterpret_cast<uint2*>(dst + c0 + c * TPR) =
          make_uint2(pack_bf16x2(out[c] * inv, out[c + 1] * inv),
                     pack_bf16x2(out[c + 2] * inv, out[c + 3] * inv));
  }
  if (A.lse && threadIdx.x % TPR == 0)
    A.lse[((long long)b * A.H + head) * A.N + tok] =
        L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

// Merges the key ranges of the split items in their order: a warp per row, a
// lane for D / 32 channels.
template <typename T, int D>
__global__ void __launch_bounds__(256)
    cache_attn_merge_kernel(const __grid_constant__ CacheAttnArgs A, int tile) {
  constexpr int W = D / 32;
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);  // over the split items' rows
  const int item = i / tile, row = i % tile;
  int b, hk, r0;
  item_rows(A, A.whole + item, tile, b, hk, r0);
  if (b >= A.B) return;
  const int r = r0 + row, tok = r / A.G, head = hk * A.G + r % A.G;
  if (tok >= query_tokens(A, b)) return;
  const long long step = tile;
  const long long p0 = (long long)item * A.splits * tile + row;
  float M = -INFINITY;
  for (int s = lane; s < A.splits; s += 32) M = fmaxf(M, A.part_ml[2 * (p0 + s * step)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float Mr = M == -INFINITY ? 0.f : M;
  float L = 0.f, out[W] = {};
#pragma unroll 4
  for (int s = 0; s < A.splits; ++s) {
    const long long pr = p0 + s * step;
    const float2 ml = *reinterpret_cast<const float2*>(A.part_ml + 2 * pr);
    if (ml.x == -INFINITY && ml.y == 0.f) continue;  // an empty range
    const float f = ex2_approx(ml.x - Mr);
    L = fmaf(f, ml.y, L);
    const float* src = A.part_o + pr * D + lane * W;
#pragma unroll
    for (int c = 0; c < W; c += 2) {
      const float2 x = *reinterpret_cast<const float2*>(src + c);
      out[c] = fmaf(f, x.x, out[c]);
      out[c + 1] = fmaf(f, x.y, out[c + 1]);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  T* dst = (T*)A.o + b * A.o_sb + (long long)tok * A.o_st + (long long)head * D + lane * W;
#pragma unroll
  for (int c = 0; c < W; c += 2) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2*>(dst + c) = make_float2(out[c] * inv, out[c + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(dst + c) = pack_bf16x2(out[c] * inv, out[c + 1] * inv);
  }
  if (A.lse && lane == 0)
    A.lse[((long long)b * A.H + head) * A.N + tok] =
        L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

// Kernel, items, key ranges and workspace of a call, from what the host knows
// (the lengths are on the device: a range of an item is cut there, from its
// own length).
struct CachePlan {
  int tile, tiles;  // rows per item, row tiles per (item, K/V head)
  long long items, whole;
  int splits;
  size_t part_o_bytes, bytes;
  long long grid() const { return whole + (items - whole) * splits; }
};

CachePlan plan_cache_attn(const mmdit_tensor_desc& q, const mmdit_cache& c) {
  CachePlan p{};
  const long long rows = (long long)q.n_tokens * (q.heads / c.heads);
  const long long cap = (long long)c.max_pages * c.page_tokens;
  p.tile = q.dtype == MMDIT_BF16 && rows > kFewRows ? kManyTile : kFewTile;
  p.tiles = (int)((rows + p.tile - 1) / p.tile);
  p.items = (long long)p.tiles * c.heads * q.batch;
  if (p.tile == kFewTile) {
    // Two CTAs of four warps per SM keep enough loads in flight; a range is at
    // least 512 tokens (16 slabs for the CTA), or its merge costs more than it saves.
    p.splits = (int)std::max(1LL, std::min(2 * 148 / p.items, (cap + 511) / 512));
    p.whole = p.splits > 1 ? 0 : p.items;
  } else {
    // One CTA per SM.  What is left behind the whole waves is split so that its
    // waves are short: ceil(left s / 148) waves of the key tiles of a range and about
    // four more for its set-up and its merge.
    p.whole = p.items / 148 * 148;
    p.splits = 1;
    const long long left = p.items - p.whole, units = (cap + kUnit - 1) / kUnit;
    long long best = 0;
    for (int s = 1; s <= std::min(148LL, std::max(1LL, units / 4)); ++s) {
      const long long cost = (left * s + 147) / 148 * ((units + s - 1) / s + (s > 1 ? 4 : 0));
      if (s == 1 || cost < best) best = cost, p.splits = s;
    }
    if (p.splits == 1) p.whole = p.items;
  }
  const size_t n = (size_t)(p.items - p.whole) * p.splits * p.tile;
  if (n > 0) {
    p.part_o_bytes = align256(n * q.head_dim * sizeof(float));
    p.bytes = p.part_o_bytes + align256(n * 2 * sizeof(float));
  }
  return p;
}

template <typename T, int D>
cudaError_t launch_few(const CacheAttnArgs& A, const CachePlan& p, cudaStream_t s) {
  cache_attn_few_kernel<T, D><<<(unsigned)p.grid(), kFewWarps * 32, 0, s>>>(A);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t launch_merge(const CacheAttnArgs& A, const CachePlan& p, cudaStream_t s) {
  const long long rows = (p.items - p.whole) * p.tile;
  cache_attn_merge_kernel<T, D><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(A, p.tile);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t launch_cache_attn(const CacheAttnArgs& A, const CachePlan& p, cudaStream_t s) {
  cudaError_t e = p.tile == kManyTile ? launch_cache_attn_many(A, D, (unsigned)p.grid(), s)
                                      : launch_few<T, D>(A, p, s);
  if (e == cudaSuccess && p.whole < p.items) e = launch_merge<T, D>(A, p, s);
  return e;
}

int check_cache_attn(const mmdit_tensor_desc* q, const mmdit_cache* c) {
  int rc;
  if ((rc = check_cache_desc(q, "cache_attn q")) || (rc = check_cache(c, "cache_attn", true)))
    return rc;
  if (q->batch != c->batch || q->head_dim != c->head_dim)
    return fail(MMDIT_EINVAL, "cache_attn: q and cache disagree on batch or head_dim");
  if (q->heads % c->heads != 0)
    return fail(MMDIT_EINVAL, "cache_attn: %d query heads over %d K/V heads", q->heads, c->heads);
  const long long rows = (long long)q->n_tokens * (q->heads / c->heads) + kManyTile;
  if (rows > 0x7fffffffLL || (rows / kFewTile + 1) * c->heads * q->batch > 0x7fffffffLL)
    return fail(MMDIT_EINVAL, "cache_attn: too many query rows");
  return MMDIT_OK;
}

}  // namespace

}  // namespace mmdit

using namespace mmdit;

extern "C" {

size_t mmdit_cache_attn_workspace_size(const mmdit_tensor_desc* q_desc, const mmdit_cache* cache) {
  if (check_cache_attn(q_desc, cache) || q_desc->n_tokens == 0) return 0;
  return plan_cache_attn(*q_desc, *cache).bytes;
}

int mmdit_cache_attn(const void* q, void* o, const mmdit_tensor_desc* q_desc,
                     const mmdit_tensor_desc* o_desc, const mmdit_cache* cache,
                     const int32_t* kv_len, const int32_t* q_len, int causal_block, float scale,
                     float* lse, void* workspace, size_t ws_bytes, mmdit_stream_t stream) {
  MMDIT_NVTX("mmdit_cache_attn");
  int rc;
  if ((rc = check_cache_attn(q_desc, cache)) || (rc = check_cache_desc(o_desc, "cache_attn o")))
    return rc;
  if (q_desc->batch != o_desc->batch || q_desc->n_tokens != o_desc->n_tokens ||
      q_desc->heads != o_desc->heads || q_desc->head_dim != o_desc->head_dim ||
      q_desc->dtype != o_desc->dtype)
    return fail(MMDIT_EINVAL, "cache_attn: q and o descriptors disagree");
  if (!q || !o || !kv_len) return fail(MMDIT_EINVAL, "cache_attn: q, o and kv_len must be non-NULL");
  if (!aligned16(q) || !aligned16(o))
    return fail(MMDIT_EINVAL, "cache_attn: tensors must be 16-byte aligned");
  if (o == q) return fail(MMDIT_EINVAL, "cache_attn: o aliases q");
  if (causal_block < 0) return fail(MMDIT_EINVAL, "cache_attn: causal_block %d", causal_block);
  if (!(scale > 0.f) || !isfinite(scale)) return fail(MMDIT_EINVAL, "cache_attn: scale must be > 0");
  if (q_desc->n_tokens == 0) return MMDIT_OK;
  const CachePlan plan = plan_cache_attn(*q_desc, *cache);
  if (plan.bytes > 0) {
    if (workspace == nullptr || ws_bytes < plan.bytes)
      return fail(MMDIT_EWORKSPACE, "cache_attn: workspace needs %zu bytes", plan.bytes);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
      return fail(MMDIT_EINVAL, "cache_attn: workspace must be 256-byte aligned");
  }
  if ((rc = check_sm100())) return rc;
  CacheAttnArgs A{};
  A.q = q;
  A.o = o;
  A.lse = lse;
  A.q_st = q_desc->stride_tok;
  A.q_sb = q_desc->stride_batch;
  A.o_st = o_desc->stride_tok;
  A.o_sb = o_desc->stride_batch;
  A.k = (const uint8_t*)cache->k;
  A.v = (const uint8_t*)cache->v;
  A.k_scale = cache->k_scale;
  A.v_scale = cache->v_scale;
  A.table = cache->page_table;
  A.kv_len = kv_len;
  A.q_len = q_len;
  A.n_pages = cache->n_pages;
  A.page = cache->page_tokens;
  while ((1 << A.page_log2) < A.page) ++A.page_log2;
  A.max_pages = cache->max_pages;
  A.B = q_desc->batch;
  A.N = q_desc->n_tokens;
  A.H = q_desc->heads;
  A.Hk = cache->heads;
  A.G = A.H / A.Hk;
  A.causal = causal_block;
  A.scale_log2 = scale * 1.4426950408889634f;
  A.tiles = plan.tiles;
  A.whole = (int)plan.whole;
  A.splits = plan.splits;
  A.part_o = (float*)workspace;
  A.part_ml = (float*)((char*)workspace + plan.part_o_bytes);
  if ((A.err = device_error_flag()) == nullptr)
    return fail(MMDIT_ECUDA, "device error flag unavailable");
  cudaStream_t s = (cudaStream_t)stream;
  const int D = q_desc->head_dim;
  cudaError_t e;
  if (q_desc->dtype == MMDIT_BF16)
    e = D == 128 ? launch_cache_attn<__nv_bfloat16, 128>(A, plan, s)
                 : launch_cache_attn<__nv_bfloat16, 64>(A, plan, s);
  else
    e = D == 128 ? launch_cache_attn<float, 128>(A, plan, s) : launch_cache_attn<float, 64>(A, plan, s);
  return e == cudaSuccess ? MMDIT_OK : cuda_fail(e, "cache_attn launch");
}

}  // extern "C"
