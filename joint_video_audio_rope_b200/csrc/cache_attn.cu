// mmdit_cache_attn: the entry point, the kernel for few query rows, and the
// merge of split key ranges.
//
// Few rows (single tokens, a frame's audio tokens; every fp32 call).  The codes
// are read once and barely used, so the call is bound by HBM: what counts is
// bytes in flight.  A warp owns slabs of 32 tokens and copies the codes of the next ones into
// its own ring in shared memory (cp.async, no barrier between warps) while it computes
// the current one.  16-byte vectors of codes are turned into fp16 pairs that are
// mma.m16n8k16 operands as they stand, because the order of channels inside a contraction (K) and of
// output channels (V) is free.  Scores and outputs are formed transposed, so that a tile of up to
// 8 query rows is one tile of 8 columns:
//   S^T  A = K (16 tokens x 16 channels), B = Q^T: thread (g, t) of a warp (g = lane
//        / 4, t = lane % 4) holds channels 16 t .. 16 t + 15 of tokens g and g + 8; step
//        kk contracts channels 16 t + 4 kk .. + 3 of every t
//   O^T  A = V^T (16 channels x 16 tokens), B = P^T: thread (g, t) holds channels
//        g D/8 .. of tokens 2t, 2t + 1, 2t + 8, 2t + 9; output tile j holds channels
//        g D/8 + 2j and + 2j + 1 of every g.  P^T is the score fragment with its
//        8 x 8 blocks transposed (movmatrix).
// The vectors of a slab's rows are permuted so that both reads meet every bank once.
// e4m3 is exact in fp16.  Q is multiplied by a power of two per row that puts
// its largest value at 2^14..2^15, so bf16 values are exact in fp16 too down
// to 2^-29 of that; fp32 values are split into two fp16 parts (22 bits), and so
// are the probabilities of an fp32 call.  Each warp runs its own softmax; the CTA's
// warps, then the key ranges, are merged at the end in a fixed order.
// One B200: 1 token of 24 heads over 75,600 tokens of 24 K/V heads (464 MB) 80 us = 5.8
// TB/s, 0.89 of the copy rate; of 8 K/V heads 34 us, 4 to 5 of them the merge; 24 heads
// over 32,760 tokens (201 MB, floor 31 us): 8 rows 41 us, 16 rows 49, 32 rows 77 (two tiles
// read the codes twice); 11 fp32 rows over 2 x 32,760 tokens of 12 heads of 64 41 us, bound
// by issue slots (16 rows and two fp16 parts make about 780 instructions per slab), 218
// fp32 rows over 32,760 tokens of 24 heads of 128 937 us: 14 tiles that read the codes one
// by one.
#include <math.h>

#include <algorithm>

#include "cache_attn.cuh"

namespace mmdit {

namespace {

constexpr int kFewWarps = 4;
// bf16 rows per (item, K/V head) up to which tiles of 8 or 16 rows are taken: 24 heads over
// 32,760 tokens, 32 rows: 77 us as two tiles, 80 on tcgen05 (33 rows); 48 rows: 105 as three and 81.
constexpr int kFewRows = 32;
constexpr long long kSummed = 1 << 17;  // most tokens in one running sum of a bf16 call
// The probability of a row's reference maximum is held as 2^14: fp16 keeps its relative
// precision down to 2^-14, so what is 2^-28 of it is still whole.  The reference may be
// behind the maximum by a factor of two (2^15 is still a number in fp16).
constexpr float kShift = 14.f;
constexpr float kGrow = 1.f;
// fp32 calls: the second part of a probability is held times 2^12, which makes it as large as the
// first one at most: held as it is, it was below fp16's numbers for what is 2^-27 of the
// maximum, and two parts were no better than one.
constexpr float kPartUp = 4096.f;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
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

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Shared memory of a warp's ring: per stage the slab's codes of K and V and, per
// 16 tokens, their scales and whether their page is there.
template <typename T, int D, int NQ>
struct Few {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int S = 32;  // tokens per slab
  static constexpr int kCtas = D * NQ * (kF32 ? 2 : 1) > 256 ? 2 : 3;  // per SM, by registers
  static constexpr int kCodes = S * D;
  static constexpr int kStage = 2 * kCodes + 32;
  static constexpr int kFit = 222 * 1024 / (kCtas * kFewWarps * kStage);
  static constexpr int kStages = kFit < 4 ? kFit : 4;
  static constexpr int kRing = kFewWarps * kStages * kStage;
  static constexpr int kMerge = kFewWarps * 8 * NQ * ((D + 4) + 2) * 4;
  static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
  static_assert(kStages >= 2, "a slab is copied while another is computed");
};

// Offset of 16-byte vector c of row r of a slab, permuted within 128 bytes: rows g,
// g + 1 (K, vectors t) and rows 2t (V, vectors g, g + 1) each cover all eight
// positions.
template <int D>
__device__ __forceinline__ int slab_at(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (r & 6) ^ ((r & 1) << 2)) << 4);
  else return (r >> 1) * 128 + ((((r & 1) << 2 | c) ^ (r & 6)) << 4);
}

// log2 of a normal x > 0: the exponent and the approximate logarithm of the mantissa,
// which is good to 2^-22 there (of a large x it would be to 2^-22 of the result).
__device__ __forceinline__ float log2_normal(float x) {
  const int bits = __float_as_int(x);
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__int_as_float((bits & 0x7fffff) | 0x3f800000)));
  return (float)((bits >> 23) - 127) + y;
}
// 8 x 8 block of 16-bit values held as a fragment (row g, columns 2t, 2t + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// NQ: tiles of 8 query rows.
template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kFewWarps * 32, Few<T, D, NQ>::kCtas)
    cache_attn_few_kernel(const __grid_constant__ CacheAttnArgs A) {
  using F = Few<T, D, NQ>;
  constexpr bool kF32 = F::kF32;
  constexpr int S = F::S;             // tokens per slab
  constexpr int ST = F::kStages;
  constexpr int HF = S / 16;          // 16-token parts of a slab: one page each
  constexpr int KK = D / 16;          // contraction steps over the channels
  constexpr int KV = D / 64;          // 16-byte code vectors per thread and token of K
  constexpr int NT = D / 16;          // output tiles
  constexpr int VW = D / 32;          // words of codes per thread and token of V
  constexpr int QP = kF32 ? 2 : 1;    // fp16 parts of Q and P
  constexpr int kTile = 8 * NQ;
  extern __shared__ __align__(128) uint8_t smem[];

  asm volatile("griddepcontrol.launch_dependents;");  // the merge may be launched
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const CacheItem w = item_of(A, blockIdx.x, kTile);
  const int b = w.b, hk = w.hk, r0 = w.r0, kv = w.kv, ql = w.ql, live = w.live;
  const int lo = w.lo, hi = w.hi;
  if (live <= 0) return;

  // ---- the ring: copies of the slab at token n into a stage
  uint8_t* ring = smem + warp * (ST * F::kStage);
  auto find = [&](int n, int (&id)[HF]) {
#pragma unroll
    for (int f = 0; f < HF; ++f) id[f] = n + 16 * f < hi ? page_of(A, b, n + 16 * f) : -1;
  };
  // This thread's vectors of a group of 16 tokens: lane + 32 i.  Their places differ
  // by 512 i, and for D = 128 by the permutation's bit of row 4.
  const uint32_t place = slab_at<D>(lane / (D / 16), lane % (D / 16));
  auto copy = [&](int n, const int (&id)[HF], int stage) {
    uint8_t* to = ring + stage * F::kStage;
    const uint32_t dst = smem_u32(to);
#pragma unroll
    for (int f = 0; f < HF; ++f) {
      const long long page = (long long)max(id[f], 0) * A.Hk + hk;
      const long long from = (page * A.page + ((n + 16 * f) & (A.page - 1))) * D + lane * 16;
      const uint8_t *kp = A.k + from, *vp = A.v + from;  // 16 D consecutive bytes
      const int rows = id[f] >= 0 ? hi - n - 16 * f : 0;
      const uint32_t at[2] = {dst + f * 16 * D + place,
                              dst + f * 16 * D + (D == 128 ? place ^ 64u : place)};
      if (rows >= 16) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          cp_async16(at[i & 1] + i * 512, kp + i * 512);
          cp_async16(at[i & 1] + i * 512 + F::kCodes, vp + i * 512);
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const bool there = (lane + 32 * i) / (D / 16) < rows;
          cp_async16_if(at[i & 1] + i * 512, there ? kp + i * 512 : A.k, there);
          cp_async16_if(at[i & 1] + i * 512 + F::kCodes, there ? vp + i * 512 : A.v, there);
        }
      }
      if (lane == f) {
        float* m = reinterpret_cast<float*>(to + 2 * F::kCodes) + 4 * f;
        m[2] = id[f] < 0 ? -INFINITY : 0.f;
        if (id[f] >= 0) {
          cp_async4(smem_u32(m), A.k_scale + page);
          cp_async4(smem_u32(m + 1), A.v_scale + page);
        } else {
          m[0] = m[1] = 0.f;
        }
      }
    }
  };
  constexpr int kStep = kFewWarps * S;
  const int n0 = lo + warp * S;
  int next[HF];  // pages of the slab that is copied next
  find(n0, next);
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) {
    const int n = n0 + i * kStep;
    if (n < hi) copy(n, next, i);
    cp_async_commit();
    find(n + kStep, next);
  }

  // ---- Q fragments of rows 8 q + g; factors and visible keys of rows 8 q + 2t + e
  uint32_t qb[QP][NQ][KK][2];
  float mul[NQ][2];
  int limit[NQ][2], full = hi;  // keys below `full` are seen by every row
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int rr = 8 * q + g, r = r0 + rr;
    const int rt = row_token(A, r);
    const T* src = (const T*)A.q + b * A.q_sb + (long long)rt * A.q_st +
                   (long long)(hk * A.G + r - rt * A.G) * D;
    float x[KK][4], am = 0.f;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      x[kk][0] = x[kk][1] = x[kk][2] = x[kk][3] = 0.f;
      if (rr < live) load4(src + (kk >> 2) * 64 + t * 16 + (kk & 3) * 4, x[kk]);
#pragma unroll
      for (int j = 0; j < 4; ++j) am = fmaxf(am, fabsf(x[kk][j]));
    }
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
    const float f = fit_half(am);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x0 = x[kk][2 * j] * f, x1 = x[kk][2 * j + 1] * f;
#pragma unroll
        for (int p = 0; p < QP; ++p) {
          const uint32_t h = pack_half2(x0, x1);
          qb[p][q][kk][j] = h;
          const float2 y = unpack_half2(h);
          x0 -= y.x;
          x1 -= y.y;
        }
      }
    const float m = A.scale_log2 * inverse_pow2(f);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mul[q][e] = __shfl_sync(0xffffffffu, m, (2 * t + e) * 4);
      // rows behind the last are computed with it and not stored
      const int row = min(8 * q + 2 * t + e, live - 1);
      limit[q][e] = visible_keys(A, kv, ql, row_token(A, r0 + row));
      full = min(full, limit[q][e]);
    }
  }
  full = min(full, __shfl_xor_sync(0xffffffffu, full, 1));
  full = min(full, __shfl_xor_sync(0xffffffffu, full, 2));

  float acc[NQ][NT][4];  // channels g D/8 + 2j (+ 1 from [2] on) of rows 2t + e
  float m[NQ][2], l[NQ][2], mref[NQ][2];  // reference maxima, sums; m - kShift (0: none yet)
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    m[q][0] = m[q][1] = -INFINITY;
    mref[q][0] = mref[q][1] = 0.f;
    l[q][0] = l[q][1] = 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[q][j][0] = acc[q][j][1] = acc[q][j][2] = acc[q][j][3] = 0.f;
  }

  int stage = 0;
  for (int n = n0; n < hi; n += kStep) {
    cp_async_wait<ST - 2>();
    __syncwarp();
    {  // the stage read last is free: the copies of the slab ST - 1 ahead
      const int ahead = n + (ST - 1) * kStep;
      if (ahead < hi) copy(ahead, next, stage == 0 ? ST - 1 : stage - 1);
      cp_async_commit();
      find(ahead + kStep, next);
    }
    const uint8_t* kc = ring + stage * F::kStage;
    const uint8_t* vc = kc + F::kCodes;
    const float4* meta = reinterpret_cast<const float4*>(vc + F::kCodes);
    stage = stage == ST - 1 ? 0 : stage + 1;
    // ---- scores of tokens 16 f + g (+ 8 from [2] on) and rows 2t + e
    float sc[NQ][HF][4];
#pragma unroll
    for (int f = 0; f < HF; ++f) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) sc[q][f][0] = sc[q][f][1] = sc[q][f][2] = sc[q][f][3] = 0.f;
#pragma unroll
      for (int c = 0; c < KV; ++c) {
        const uint4 r0v = *reinterpret_cast<const uint4*>(kc + slab_at<D>(f * 16 + g, c * 4 + t));
        const uint4 r8v =
            *reinterpret_cast<const uint4*>(kc + slab_at<D>(f * 16 + g + 8, c * 4 + t));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = k == 0 ? r0v.x : k == 1 ? r0v.y : k == 2 ? r0v.z : r0v.w;
          const uint32_t y = k == 0 ? r8v.x : k == 1 ? r8v.y : k == 2 ? r8v.z : r8v.w;
          uint32_t a[4];
          halves_of(x, a[0], a[2]);
          halves_of(y, a[1], a[3]);
#pragma unroll
          for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int p = QP - 1; p >= 0; --p)
              mma16816(sc[q][f], a, qb[p][q][c * 4 + k][0], qb[p][q][c * 4 + k][1]);
        }
      }
    }
    float kf[HF], lv[HF], iv[HF], wv[HF];
#pragma unroll
    for (int f = 0; f < HF; ++f) {
      const float4 m4 = meta[f];
      kf[f] = m4.x;
      // a page that is not there is not seen; a V scale of 0 stands for zeros
      lv[f] = m4.z + (m4.y > 0.f ? log2_normal(m4.y) : kNoScaleLog2);
      iv[f] = m4.y > 0.f ? __frcp_rn(m4.y) : 0.f;
      wv[f] = m4.y > 0.f ? iv[f] : kNoScaleInverse;
    }
    if (__any_sync(0xffffffffu, n + S > full)) {
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int f = 0; f < HF; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + f * 16 + g + 8 * (i >> 1) >= limit[q][i & 1]) sc[q][f][i] = -INFINITY;
    }
    // ---- softmax of rows 2t (e = 0) and 2t + 1: the reference moves once a score is beyond
    // twice it, which few slabs need, so lanes seldom have to agree on a maximum
    bool grew = false;
    float top[NQ][2], fac[NQ][HF][2];
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = -INFINITY;
#pragma unroll
        for (int f = 0; f < HF; ++f) {
          // at least the smallest normal number: -inf stays -inf
          fac[q][f][e] = fmaxf(mul[q][e] * kf[f], 1.1754944e-38f);
          mx = fmaxf(mx, fmaf(fmaxf(sc[q][f][e], sc[q][f][2 + e]), fac[q][f][e], lv[f]));
        }
        top[q][e] = mx;
        grew = grew || mx > m[q][e] + kGrow;
      }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = top[q][e];
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = fmaxf(m[q][e], mx);
          alpha[e] = mn == -INFINITY ? 1.f : ex2_approx(m[q][e] - mn);
          m[q][e] = mn;
          mref[q][e] = mn == -INFINITY ? 0.f : mn - kShift;
          l[q][e] *= alpha[e];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[q][j][0] *= alpha[0];
          acc[q][j][1] *= alpha[1];
          acc[q][j][2] *= alpha[0];
          acc[q][j][3] *= alpha[1];
        }
      }
    }
    // ---- P
    uint32_t pb[HF][QP][NQ][2];
#pragma unroll
    for (int f = 0; f < HF; ++f)
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // tokens g, then g + 8
          // one rounding, of what is left of the exponent beside the reference
          float p0 = ex2_approx(fmaf(sc[q][f][2 * i], fac[q][f][0], lv[f] - mref[q][0]));
          float p1 = ex2_approx(fmaf(sc[q][f][2 * i + 1], fac[q][f][1], lv[f] - mref[q][1]));
          l[q][0] = fmaf(p0, wv[f], l[q][0]);
          l[q][1] = fmaf(p1, wv[f], l[q][1]);
#pragma unroll
          for (int p = 0; p < QP; ++p) {
            const uint32_t h = pack_half2(p0, p1);
            pb[f][p][q][i] = transpose8(h);
            if (p + 1 < QP) {
              const float2 y = unpack_half2(h);
              p0 = (p0 - y.x) * kPartUp;
              p1 = (p1 - y.y) * kPartUp;
            }
          }
        }
    // ---- the output
    uint32_t vr[HF][4][VW];
#pragma unroll
    for (int f = 0; f < HF; ++f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = f * 16 + 2 * t + (i & 1) + (i >> 1) * 8;
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(vc + slab_at<D>(row, g));
          vr[f][i][0] = x.x, vr[f][i][1] = x.y, vr[f][i][2] = x.z, vr[f][i][3] = x.w;
        } else {
          const uint2 x =
              *reinterpret_cast<const uint2*>(vc + slab_at<D>(row, g >> 1) + (g & 1) * 8);
          vr[f][i][0] = x.x, vr[f][i][1] = x.y;
        }
      }
      if (!(iv[f] > 0.f)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < VW; ++k) vr[f][i][k] = 0u;
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      // fp32: a sum of its own per slab, so that the long sum is a rounded one (the
      // tensor cores truncate)
      float d[NQ][4];
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c) d[q][c] = kF32 ? 0.f : acc[q][j][c];
      uint32_t a[HF][4];
#pragma unroll
      for (int f = 0; f < HF; ++f) {
        // channels 2j and 2j + 1 of tokens (2t, 2t + 1) and (2t + 8, 2t + 9)
        const uint32_t pick = j & 1 ? 0x7362 : 0x5140;
        const uint32_t x = __byte_perm(vr[f][0][j >> 1], vr[f][1][j >> 1], pick);
        const uint32_t y = __byte_perm(vr[f][2][j >> 1], vr[f][3][j >> 1], pick);
        halves_of(x, a[f][0], a[f][1]);
        halves_of(y, a[f][2], a[f][3]);
      }
#pragma unroll
      for (int p = QP - 1; p >= 0; --p) {
#pragma unroll
        for (int f = 0; f < HF; ++f)
#pragma unroll
          for (int q = 0; q < NQ; ++q) mma16816(d[q], a[f], pb[f][p][q][0], pb[f][p][q][1]);
        if (p > 0) {  // the small parts, back to size before the large ones join them
#pragma unroll
          for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int c = 0; c < 4; ++c) d[q][c] *= 1.f / kPartUp;
        }
      }
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[q][j][c] = kF32 ? acc[q][j][c] + d[q][c] : d[q][c];
    }
  }

  // ---- the CTA's warps, merged in their order; the rings are done with
  // set: an earlier kernel timed out, and attention kernels leave their outputs alone
  const int skip = *(volatile int*)A.err;
  cp_async_wait<0>();
  __syncthreads();
  float(*sm_o)[kTile][D + 4] = reinterpret_cast<float(*)[kTile][D + 4]>(smem);
  float(*sm_ml)[kTile][2] =
      reinterpret_cast<float(*)[kTile][2]>(smem + kFewWarps * kTile * (D + 4) * 4);
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float& x = l[q][e];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      const int row = 8 * q + 2 * t + e;
      if (g == 0) {
        sm_ml[warp][row][0] = m[q][e] - kShift;
        sm_ml[warp][row][1] = x;
      }
#pragma unroll
      for (int j = 0; j < NT; j += 2)
        *reinterpret_cast<float4*>(&sm_o[warp][row][g * (D / 8) + 2 * j]) = make_float4(
            acc[q][j][e], acc[q][j][2 + e], acc[q][j + 1][e], acc[q][j + 1][2 + e]);
    }
  __syncthreads();
  constexpr int TPR = kFewWarps * 32 / kTile;  // threads per row
  constexpr int W = D / TPR;                   // channels per thread
  const int row = threadIdx.x / TPR, c0 = (threadIdx.x % TPR) * 4;
  if (row >= live || skip != 0) return;
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
    const long long pr = w.part * kTile + row;
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
  const int tok = row_token(A, r), head = hk * A.G + r - tok * A.G;
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
    A.lse[((long long)b * A.H + head) * A.N + tok] = row_lse(M, L);
}

// Merges the key ranges of the split items in a fixed order: WPR warps per row (warp
// w takes ranges w, w + WPR, ..), a lane for D / 32 channels.  Launched while the
// attention kernel still runs (its launch costs no time of its own) and waits for it here.
template <typename T, int D, int WPR>
__global__ void __launch_bounds__(256)
    cache_attn_merge_kernel(const __grid_constant__ CacheAttnArgs A, int tile) {
  constexpr int W = D / 32;
  __shared__ float part[WPR == 1 ? 1 : WPR][D + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * (8 / WPR) + warp / WPR;  // over the split items' rows
  const int item = i / tile, row = i % tile;
  int b, hk, r0;
  item_rows(A, A.whole + item, tile, b, hk, r0);
  const int r = r0 + row, tok = row_token(A, r), head = hk * A.G + r - tok * A.G;
  const bool live = b < A.B && tok < query_tokens(A, b);  // the same in all warps of a row
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!live) return;
  const int skip = *(volatile int*)A.err;  // set: the ranges have not been written
  const long long p0 = (long long)item * A.splits * tile + row;
  float M = -INFINITY, L = 0.f, out[W] = {};
  constexpr int kBatch = 8;  // ranges whose sums are under way at once, beside the maxima
  for (int s = lane; s < A.splits; s += 32)
    M = fmaxf(M, A.part_ml[2 * (p0 + (long long)s * tile)]);
  for (int s0 = warp % WPR; s0 < A.splits; s0 += WPR * kBatch) {
    float2 ml[kBatch], x[kBatch][W / 2];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const long long pr = p0 + (long long)min(s0 + u * WPR, A.splits - 1) * tile;
      ml[u] = *reinterpret_cast<const float2*>(A.part_ml + 2 * pr);
#pragma unroll
      for (int c = 0; c < W / 2; ++c)
        x[u][c] = *reinterpret_cast<const float2*>(A.part_o + pr * D + lane * W + 2 * c);
    }
    if (s0 < WPR) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    }
    const float Mr = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      // an empty range's sums are zeros: it adds nothing
      const bool none = s0 + u * WPR >= A.splits || (ml[u].x == -INFINITY && ml[u].y == 0.f);
      if (none) continue;
      const float f = ex2_approx(ml[u].x - Mr);
      L = fmaf(f, ml[u].y, L);
#pragma unroll
      for (int c = 0; c < W / 2; ++c) {
        out[2 * c] = fmaf(f, x[u][c].x, out[2 * c]);
        out[2 * c + 1] = fmaf(f, x[u][c].y, out[2 * c + 1]);
      }
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int c = 0; c < W; ++c) part[warp][lane * W + c] = out[c];
    if (lane == 0) part[warp][D] = L;
    __syncthreads();
    if (warp > 0) return;
    L = 0.f;
#pragma unroll
    for (int c = 0; c < W; ++c) out[c] = 0.f;
#pragma unroll
    for (int x = 0; x < WPR; ++x) {
      L += part[x][D];
#pragma unroll
      for (int c = 0; c < W; ++c) out[c] += part[x][lane * W + c];
    }
  }
  if (skip != 0) return;
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
    A.lse[((long long)b * A.H + head) * A.N + tok] = row_lse(M, L);
}

// Kernel, items, key ranges and workspace of a call, from what the host knows
// (the lengths are on the device: a range of an item is cut there, from its
// own length).
struct CachePlan {
  int tile, tiles;  // rows per item, row tiles per (item, K/V head)
  long long items, whole;
  long long splits;
  size_t part_o_bytes, bytes;
  long long grid() const { return whole + (items - whole) * splits; }
};

CachePlan plan_cache_attn(const mmdit_tensor_desc& q, const mmdit_cache& c) {
  CachePlan p{};
  const long long rows = (long long)q.n_tokens * (q.heads / c.heads);
  const long long cap = (long long)c.max_pages * c.page_tokens;
  p.tile = q.dtype == MMDIT_BF16 && rows > kFewRows ? kManyTile : rows > 8 ? 16 : 8;
  p.tiles = (int)((rows + p.tile - 1) / p.tile);
  p.items = (long long)p.tiles * c.heads * q.batch;
  // Ranges that one accumulator of the tensor cores sums: they truncate each sum, which over
  // 2^20 tokens had lost 0.5 % of positive values.  (fp32 calls sum up slab by slab.)
  const long long range = p.tile == kManyTile ? kSummed : q.dtype == MMDIT_BF16 ? kFewWarps * kSummed : cap;
  const long long least = std::max(1LL, (cap + range - 1) / range);
  if (p.tile != kManyTile) {
    // A wave of as many CTAs as fit (Few::kCtas); a range is at least 256 tokens, two slabs per
    // warp, and a history of up to 512 is not split (3 rows x 8 heads over 20,000 tokens: 14.4 us
    // in ranges of 256, 16.1 of 512; over 1,000: 10.9 and 14.8).
    const int weight = q.head_dim * (p.tile / 8) * (q.dtype == MMDIT_F32 ? 2 : 1);
    p.splits = std::max(
        least, std::min((weight > 256 ? 2 : 3) * 148 / p.items, cap <= 512 ? 1 : (cap + 255) / 256));
    p.whole = p.splits > 1 ? 0 : p.items;
  } else {
    // One CTA per SM.  What is left behind the whole waves is split so that its
    // waves are short: ceil(left s / 148) waves of the key tiles of a range and about
    // three more for its set-up and its merge (100 rows x 24 heads over 1,024 tokens: 26 us
    // in one range when four took 19.5; they take 16.4 now).
    p.whole = least > 1 ? 0 : p.items / 148 * 148;
    p.splits = least;
    const long long left = p.items - p.whole, units = (cap + kUnit - 1) / kUnit;
    const long long most = std::max(least, std::min(148LL, units / 2));
    long long best = 0;
    for (long long s = least; s <= most; ++s) {
      const long long cost = (left * s + 147) / 148 * ((units + s - 1) / s + (s > 1 ? 3 : 0));
      if (s == least || cost < best) best = cost, p.splits = s;
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

template <typename T, int D, int NQ>
cudaError_t launch_few(const CacheAttnArgs& A, const CachePlan& p, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once_per_device(dev, [] {
    return cudaFuncSetAttribute(cache_attn_few_kernel<T, D, NQ>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Few<T, D, NQ>::kSmem);
  });
  if (e != cudaSuccess) return e;
  cache_attn_few_kernel<T, D, NQ>
      <<<(unsigned)p.grid(), kFewWarps * 32, Few<T, D, NQ>::kSmem, s>>>(A);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t launch_merge(const CacheAttnArgs& A, const CachePlan& p, cudaStream_t s) {
  const long long rows = (p.items - p.whole) * p.tile;
  const bool few = p.splits <= 8;  // a warp reads that many ranges at once
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(few ? (rows + 7) / 8 : rows));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, cache_attn_merge_kernel<T, D, 1>, A, p.tile)
             : cudaLaunchKernelEx(&cfg, cache_attn_merge_kernel<T, D, 8>, A, p.tile);
}
template <typename T, int D>
cudaError_t launch_cache_attn(const CacheAttnArgs& A, const CachePlan& p, cudaStream_t s) {
  cudaError_t e = p.tile == kManyTile ? launch_cache_attn_many(A, D, (unsigned)p.grid(), s)
                  : p.tile == 16      ? launch_few<T, D, 2>(A, p, s)
                                      : launch_few<T, D, 1>(A, p, s);
  if (e == cudaSuccess && p.whole < p.items) e = launch_merge<T, D>(A, p, s);
  return e;
}

// checks q and the cache, and plans the call
int check_cache_attn(const mmdit_tensor_desc* q, const mmdit_cache* c, CachePlan& p) {
  int rc;
  if ((rc = check_cache_desc(q, "cache_attn q")) || (rc = check_cache(c, "cache_attn", true)))
    return rc;
  if (q->batch != c->batch || q->head_dim != c->head_dim)
    return fail(MMDIT_EINVAL, "cache_attn: q and cache disagree on batch or head_dim");
  if (q->heads % c->heads != 0)
    return fail(MMDIT_EINVAL, "cache_attn: %d query heads over %d K/V heads", q->heads, c->heads);
  const long long rows = (long long)q->n_tokens * (q->heads / c->heads) + kManyTile;
  if (rows > 0x7fffffffLL || (rows / 16 + 1) * c->heads * q->batch > 0x7fffffffLL)
    return fail(MMDIT_EINVAL, "cache_attn: too many query rows");
  p = CachePlan{};
  if (q->n_tokens == 0) return MMDIT_OK;
  p = plan_cache_attn(*q, *c);
  if (p.grid() > 0x7fffffffLL || (p.items - p.whole) * p.tile > 0x7ffffff0LL)  // CTAs, rows merged
    return fail(MMDIT_EINVAL, "cache_attn: too many query rows over %lld tokens",
                (long long)c->max_pages * c->page_tokens);
  return MMDIT_OK;
}

}  // namespace

}  // namespace mmdit

using namespace mmdit;

extern "C" {

size_t mmdit_cache_attn_workspace_size(const mmdit_tensor_desc* q_desc, const mmdit_cache* cache) {
  CachePlan plan;
  return check_cache_attn(q_desc, cache, plan) ? 0 : plan.bytes;
}

int mmdit_cache_attn(const void* q, void* o, const mmdit_tensor_desc* q_desc,
                     const mmdit_tensor_desc* o_desc, const mmdit_cache* cache,
                     const int32_t* kv_len, const int32_t* q_len, int causal_block, float scale,
                     float* lse, void* workspace, size_t ws_bytes, mmdit_stream_t stream) {
  MMDIT_NVTX("mmdit_cache_attn");
  int rc;
  CachePlan plan;
  if ((rc = check_cache_attn(q_desc, cache, plan)) || (rc = check_cache_desc(o_desc, "cache_attn o")))
    return rc;
  if (q_desc->batch != o_desc->batch || q_desc->n_tokens != o_desc->n_tokens ||
      q_desc->heads != o_desc->heads || q_desc->head_dim != o_desc->head_dim ||
      q_desc->dtype != o_desc->dtype)
    return fail(MMDIT_EINVAL, "cache_attn: q and o descriptors disagree");
  const bool some = q_desc->n_tokens > 0;  // tensors without tokens may have no address
  if (!kv_len || (some && (!q || !o)))
    return fail(MMDIT_EINVAL, "cache_attn: q, o and kv_len must be non-NULL");
  if (!aligned16(q) || !aligned16(o))
    return fail(MMDIT_EINVAL, "cache_attn: tensors must be 16-byte aligned");
  if (some && o == q) return fail(MMDIT_EINVAL, "cache_attn: o aliases q");
  if (causal_block < 0) return fail(MMDIT_EINVAL, "cache_attn: causal_block %d", causal_block);
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.f) || !isfinite(scale_log2))
    return fail(MMDIT_EINVAL, "cache_attn: scale must be > 0 and below 2^127");
  if (q_desc->n_tokens == 0) return MMDIT_OK;
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
  while ((1LL << A.g_shift) < A.G) ++A.g_shift;
  A.g_mul = (uint32_t)(((1ull << 32) * ((1ull << A.g_shift) - A.G)) / A.G + 1);
  A.causal = causal_block;
  A.scale_log2 = scale_log2;
  A.tiles = plan.tiles;
  A.whole = (int)plan.whole;
  A.splits = (int)plan.splits;
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
