// mmdit_cache_attn for many bf16 query rows: tcgen05 tiles over the paged cache.
//
// A CTA (512 threads, one per SM) takes 256 query rows of one K/V head (two
// tiles of 128) and a range of its keys:
//   warps 0-3, 4-7  softmax of row tile 0 and 1 (thread = row)
//   warps 8-11      converters: codes from global memory to registers, one
//                   tile ahead of use, and as fp16 (e4m3 is exact there) into
//                   the swizzled K and V tiles
//   warp 12         issues the MMAs
//   warp 13         looks up the pages and scales of the tiles to come
// Tensor memory: [0,128) S0 / P0, [128,256) S1 / P1, then O0 and O1 (D columns each).
//
// S = Q K^T with Q as fp16: each row is multiplied by the power of two that puts its
// largest value at 2^14..2^15 (bf16 is exact there down to 2^-29 of it). With f = Q's
// factor^-1 * scale * log2(e) * (K scale), constant over the 16 tokens of a page group, the
// exponent is t = S f + log2(V scale): its row maximum is found group by group from the
// maxima of S, so the scales cost eight multiply-adds per row and tile.  P = 2^(t - m + 12)
// is held as fp16: rounded by 2^-11 down to 2^-26 of the row's largest term and by 2^-37 of
// that below, so that the other tokens' terms stay whole beside a leading token whose V is
// small; m follows the maximum only once it has grown by 2^3 (P <= 2^15 then).  Three 480p
// frames: 2^7 and 2^8 took 0.2 to 1.1 % less time and kept terms whole down to 2^-21 only,
// 2^14 and 2^1 (2^-28) took 0.7 to 1.9 % more.  The sum of weights adds up 2^(t - m + 12) /
// (V scale) per group.
//
// One B200: 4,680 rows x 24 heads over 37,440 tokens 1.85 ms in a running program (power
// cap, 1,116 TFLOP/s; the first calls 1.61 ms), head_dim 64 1.68 ms; 218 rows x 24 heads
// over 32,760 tokens 111 us, head_dim 64 92; 100 rows over 1,024 tokens 16.4, over 128
// 10.3.  The tensor pipe is at 57 %, the exponentials at 58 % of their pipe, shared memory
// at 79 %.  What bounds it, by clock stamps (three frames, 3,840 cycles per 128 keys of two
// row tiles, 2,048 of them tensor work): a softmax warp computes for 2,600 and waits for
// its scores for 1,240; the issuing warp waits for P for 1,770 and is in its issue code for
// 1,700, so neither a row tile's chain (scores out, softmax, P in, product) nor the issue
// alone is all of it.
#include <math.h>

#include "cache_attn.cuh"

namespace mmdit {

namespace {

constexpr int kKeys = 128;                // keys per tile
constexpr int kHalf = 128 * 128;          // bytes of 64 channels of a 128-row fp16 tile
constexpr int kThreads = 512;
constexpr int kPageSlots = 8;             // tiles whose pages and scales are held
constexpr float kManyShift = 12.f;        // P of a row's reference maximum: 2^12
constexpr float kGrow = 3.f;              // the reference moves beyond 2^3 of it
// registers per thread: softmax, converters, MMA warpgroup; 128 (2 a + b + c) = 65,536
constexpr int kRegsSoftmax = 184, kRegsConvert = 104, kRegsMma = 40;
static_assert(2 * kRegsSoftmax + kRegsConvert + kRegsMma <= 512, "register split");

template <int D>
struct Many {
  static constexpr int kTile = 128 * D * 2;  // bytes of a 128-row fp16 tile
  static constexpr int kKOff = 2 * kTile;    // behind the two Q tiles
  static constexpr int kVOff = kKOff + 2 * kTile;
  static constexpr int kPageOff = kVOff + 2 * kTile;             // float4 [slots][8]
  static constexpr int kMulOff = kPageOff + kPageSlots * 8 * 16;  // float [256]
  static constexpr int kBarOff = kMulOff + 256 * 4;
  static constexpr int kSmem = kBarOff + 512 + 1024;  // and room to align
  static constexpr uint32_t kIdescQK = (1u << 4) | (kKeys / 8 << 17) | (128 / 16 << 24);
  static constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | (D / 8 << 17) | (128 / 16 << 24);
};

enum {
  M_QREADY = 0,  // 2: Q tile written (128 arrivals)
  M_KFULL = 2,   // 2: K tile converted (128)
  M_KEMPTY = 4,  // 2: its QKs done (commit)
  M_VFULL = 6,
  M_VEMPTY = 8,
  M_SFULL = 10,  // 2: S in tensor memory (commit)
  M_PHALF = 12,  // 2: P of keys 0..63 written (128)
  M_PFULL = 14,  // 2: P written (128)
  M_OFULL = 16,  // 2: last PV done (commit)
  M_DONE = 18,   // 1: every MMA done (commit)
  M_PAGES = 19,  // 8: pages and scales of a tile written (32)
  M_PFREE = 27,  // 8: every reader of them is done (one arrival)
  M_COUNT = 35
};

// mbar_wait with a short loop: the clock is read once in 32 tries, so that
// waiting warps leave the issue slots to the working ones.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  do {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) return true;
  } while (global_timer_ns() - t0 < kWaitLimitNs);
  atomicExch(err, (int)MMDIT_ETIMEOUT);
  return false;
}
// The same by a whole warp, which goes on or gives up together: where the lanes vote again
// later, one that left alone would keep the others waiting for good.
__device__ __forceinline__ bool all_wait(uint32_t bar, uint32_t parity, int* err) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, err));
}
// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// s[i] = -inf for i >= lim.  Few tiles need it; group by group, so that the
// compiler makes branches of it and not 128 selects that every tile runs.
__device__ __forceinline__ void mask_row(float (&s)[kKeys], int lim) {
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    if (lim < 16 * g + 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (16 * g + i >= lim) s[16 * g + i] = -INFINITY;
    }
  }
}

// GP: 16-token groups per page.
template <int D, int GP>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_many_kernel(const __grid_constant__ CacheAttnArgs A) {
  using C = Many<D>;
  asm volatile("griddepcontrol.launch_dependents;");  // the merge may be launched
  const CacheItem w = item_of(A, blockIdx.x, kManyTile);
  if (w.live <= 0) return;
  const int tiles = (w.hi - w.lo + kKeys - 1) / kKeys;  // 0: nothing to see
  const int nt = w.live > 128 ? 2 : 1;                  // row tiles in use

  extern __shared__ uint8_t smem_raw[];
  // an offset, not a cast address: the accesses below stay shared-memory ones
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::kBarOff + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 8 * M_COUNT);
  float4* pages = reinterpret_cast<float4*>(smem + C::kPageOff);  // K scale, log2 and inverse of V's, id
  float* muls = reinterpret_cast<float*>(smem + C::kMulOff);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  int* err = A.err;
  const bool skip = *(volatile int*)err != 0;  // an earlier kernel timed out

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(M_QREADY + t), 128);
      mbar_init(bar(M_KFULL + t), 128);
      mbar_init(bar(M_KEMPTY + t), 1);
      mbar_init(bar(M_VFULL + t), 128);
      mbar_init(bar(M_VEMPTY + t), 1);
      mbar_init(bar(M_SFULL + t), 1);
      mbar_init(bar(M_PHALF + t), 128);
      mbar_init(bar(M_PFULL + t), 128);
      mbar_init(bar(M_OFULL + t), 1);
    }
    for (int i = 0; i < kPageSlots; ++i) {
      mbar_init(bar(M_PAGES + i), 32);
      mbar_init(bar(M_PFREE + i), 1);
    }
    mbar_init(bar(M_DONE), 1);
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp >= 12) {
    // ------------------------------------------------------------ MMA issuer
    // As P_t lies over S_t, tile t's order is QK(0), PV(0), QK(1), PV(1), ...;
    // the two row tiles alternate, so one's softmax runs under the other's MMAs.
    // The whole warp runs the loop, so descriptors stay in uniform registers; one
    // elected lane issues.
    setmaxnreg_dec<kRegsMma>();
    if (warp == 12 && !skip) {
      bool ok = true;
      auto qk = [&](int t, int slot) {
        const uint64_t a = smem_desc_sw128(sbase + t * C::kTile, 16, 1024);
        const uint64_t b = smem_desc_sw128(sbase + C::kKOff + slot * C::kTile, 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t at = (uint64_t)((k >> 2) * (kHalf >> 4) + (k & 3) * 2);
            tc_mma_ss(tmem + t * 128, a + at, b + at, C::kIdescQK, k > 0);
          }
          tc_commit(bar(M_SFULL + t));
        }
        __syncwarp();
      };
      auto pv = [&](int t, int slot, int half, bool add) {
        const uint64_t b = smem_desc_sw128(sbase + C::kVOff + slot * C::kTile, kHalf, 1024);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_ts(tmem + 256 + t * D, tmem + t * 128 + (4 * half + k) * 8,
                      b + (uint64_t)((4 * half + k) * 128), C::kIdescPV, add || half + k > 0);
        }
        __syncwarp();
      };
      auto commit = [&](int i) {
        if (elect_one()) tc_commit(bar(i));
        __syncwarp();
      };
      if (tiles > 0) {
        for (int t = 0; t < nt && ok; ++t) ok = wait_for(bar(M_QREADY + t), 0, err);
        ok = __all_sync(0xffffffffu, ok && wait_for(bar(M_KFULL), 0, err));
        if (ok) {
          tc_fence_after();
          for (int t = 0; t < nt; ++t) qk(t, 0);
          commit(M_KEMPTY);
        }
        for (int j = 0; j < tiles && ok; ++j) {
          const int sv = j & 1, sk = sv ^ 1;
          const bool more = j + 1 < tiles;
          if (!(ok = all_wait(bar(M_VFULL + sv), (j >> 1) & 1, err))) break;
          for (int t = 0; t < nt; ++t) {
            if (!(ok = all_wait(bar(M_PHALF + t), j & 1, err))) break;
            tc_fence_after();
            pv(t, sv, 0, j > 0);
            if (!(ok = all_wait(bar(M_PFULL + t), j & 1, err))) break;
            tc_fence_after();
            pv(t, sv, 1, true);
            if (t == nt - 1) commit(M_VEMPTY + sv);
            if (more) {
              if (t == 0 && !(ok = all_wait(bar(M_KFULL + sk), ((j + 1) >> 1) & 1, err))) break;
              tc_fence_after();
              qk(t, sk);
              if (t == nt - 1) commit(M_KEMPTY + sk);
            }
          }
          // tile j is converted and both softmaxes have written their P
          if (lane == 0) mbar_arrive(bar(M_PFREE + j % kPageSlots));
        }
      }
      for (int t = 0; t < nt; ++t) commit(M_OFULL + t);
      commit(M_DONE);
      wait_for(bar(M_DONE), 0, err);
    } else if (warp == 13 && !skip) {
      // ---------------------------------------------------------- pages
      // Lane g < 8 looks up group g of every tile.  A page that is not there is not
      // seen; a V scale of 0 (its inverse held as a negative number) stands for zeros.
      bool ok = true;
      for (int j = 0; j < tiles && ok; ++j) {
        float4 x = make_float4(0.f, -INFINITY, 1.f, __int_as_float(-1));
        const int n = w.lo + j * kKeys + (lane & 7) * 16;
        const int page = n < w.hi ? page_of(A, w.b, n) : -1;
        if (page >= 0) {
          const long long at = (long long)page * A.Hk + w.hk;
          const float vs = __ldg(A.v_scale + at);
          x = make_float4(__ldg(A.k_scale + at), vs > 0.f ? log2f(vs) : kNoScaleLog2,
                          vs > 0.f ? 1.f / vs : -kNoScaleInverse, __int_as_float(page));
        }
        if (j >= kPageSlots)
          ok = all_wait(bar(M_PFREE + j % kPageSlots), (j / kPageSlots - 1) & 1, err);
        if (lane < 8) pages[(j % kPageSlots) * 8 + lane] = x;
        if (ok) mbar_arrive(bar(M_PAGES + j % kPageSlots));
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ converters
    // A warp converts 32 tokens of each tile.  Eight lanes hold four 16-code
    // vectors of two neighbouring tokens: their fp16 chunks fall on all eight
    // 16-byte columns of the swizzled tile, so the stores meet no bank twice.
    setmaxnreg_dec<kRegsConvert>();
    constexpr int NI = D / 16;                   // vectors per thread and tile
    constexpr int RS = 32 / NI;                  // tokens per load instruction
    const int cw = warp - 8;
    const int c4 = lane & 3, half = D == 128 ? (lane >> 3) & 1 : 0;
    const int row = ((lane >> 2) & 1) + 2 * (D == 128 ? lane >> 4 : lane >> 3);
    const int n0 = w.lo + cw * 32;
    int pg[2];  // pages of the warp's two groups; -1: nothing to load
    bool ok = !skip;
    // the pages of tile j; returns which of the groups have a V scale
    auto find = [&](int j) {
      const int slot = j % kPageSlots;
      ok = all_wait(bar(M_PAGES + slot), (j / kPageSlots) & 1, err);
      const float4 a = pages[slot * 8 + cw * 2], b = pages[slot * 8 + cw * 2 + 1];
      pg[0] = ok ? __float_as_int(a.w) : -1;
      pg[1] = ok ? __float_as_int(b.w) : -1;
      return (a.z > 0.f ? 1 : 0) | (b.z > 0.f ? 2 : 0);
    };
    auto load = [&](const uint8_t* codes, int j, uint4 (&r)[NI]) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int n = n0 + j * kKeys + f * 16;
        const uint8_t* src =
            codes + (((long long)pg[f] * A.Hk + w.hk) * GP + ((n >> 4) & (GP - 1))) * (16 * D) +
            row * D + half * 64 + c4 * 16;
        uint4* to = r + f * (NI / 2);
        if (pg[f] >= 0 && n + 16 <= w.hi) {  // the whole group is there
#pragma unroll
          for (int i = 0; i < NI / 2; ++i)
            to[i] = __ldg(reinterpret_cast<const uint4*>(src + i * RS * D));
        } else {
          const int rows = pg[f] >= 0 ? w.hi - n - row : 0;  // of this thread's tokens and later ones
#pragma unroll
          for (int i = 0; i < NI / 2; ++i) {
            to[i] = make_uint4(0u, 0u, 0u, 0u);
            if (i * RS < rows) to[i] = __ldg(reinterpret_cast<const uint4*>(src + i * RS * D));
          }
        }
      }
    };
    auto store = [&](uint8_t* tile, const uint4 (&r)[NI]) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int n = cw * 32 + i * RS + row;
        uint8_t* line = tile + half * kHalf + n * 128;
        uint4 a, b;
        halves_of(r[i].x, a.x, a.y);
        halves_of(r[i].y, a.z, a.w);
        halves_of(r[i].z, b.x, b.y);
        halves_of(r[i].w, b.z, b.w);
        *reinterpret_cast<uint4*>(line + (((2 * c4) ^ (n & 7)) << 4)) = a;
        *reinterpret_cast<uint4*>(line + (((2 * c4 + 1) ^ (n & 7)) << 4)) = b;
      }
    };
    uint4 kr[NI], vr[NI];
    int scaled = 0;  // groups of the V codes in flight that have a scale
    if (tiles > 0 && ok) {
      scaled = find(0);
      load(A.k, 0, kr);
      load(A.v, 0, vr);
    }
    for (int j = 0; j < tiles && ok; ++j) {
      const int slot = j & 1;
      const uint32_t free = ((j >> 1) & 1) ^ 1;
      const bool more = j + 1 < tiles;
      if (!(ok = all_wait(bar(M_KEMPTY + slot), free, err))) break;
      store(smem + C::kKOff + slot * C::kTile, kr);
      fence_proxy_async_smem();
      mbar_arrive(bar(M_KFULL + slot));
      int next = 0;
      if (more) {
        next = find(j + 1);
        load(A.k, j + 1, kr);
      }
      if (!ok || !(ok = all_wait(bar(M_VEMPTY + slot), free, err))) break;
      if (scaled != 3) {  // no scale: zeros
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (!(scaled >> (i >= NI / 2) & 1)) vr[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      store(smem + C::kVOff + slot * C::kTile, vr);
      fence_proxy_async_smem();
      mbar_arrive(bar(M_VFULL + slot));
      if (more) load(A.v, j + 1, vr);
      scaled = next;
    }
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<kRegsSoftmax>();
    const int t = warp >> 2;
    const int row = threadIdx.x;  // 0 .. 255
    const bool valid = row < w.live;
    if (t < nt) {
      if (tiles > 0) {
        // Q rows of this warp: fp16, largest value at 2^14..2^15
        // Copied to their places as they are, all at once, then turned into fp16 there by
        // the lane that copied them.  Short loops: code that runs once costs its fetch.
        constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes per row, rows per step
        const int c = lane % LPR, first = warp * 32 + lane / LPR;
        uint8_t* place = smem + t * C::kTile + (c >> 3) * kHalf;
        auto at = [&](int n) { return place + (n & 127) * 128 + (((c & 7) ^ (n & 7)) << 4); };
#pragma unroll 2
        for (int i = 0; i < 32; i += RPI) {
          const int n = first + i, r = w.r0 + n, tok = row_token(A, r);
          const bool there = n < w.live;
          const __nv_bfloat16* src = (const __nv_bfloat16*)A.q;
          if (there)
            src += w.b * A.q_sb + (long long)tok * A.q_st +
                   (long long)(w.hk * A.G + r - tok * A.G) * D + c * 8;
          cp_async16_if(smem_u32(at(n)), src, there);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        constexpr int U = 4;  // rows whose maxima are found side by side
#pragma unroll 1
        for (int i = 0; i < 32; i += U * RPI) {
          uint4 v[U];
          float am[U];
#pragma unroll
          for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const uint4*>(at(first + i + u * RPI));
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v[u]);
            am[u] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 x = __bfloat1622float2(p[k]);
              am[u] = max3f(am[u], fabsf(x.x), fabsf(x.y));
            }
          }
#pragma unroll
          for (int off = LPR / 2; off > 0; off >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u)
              am[u] = fmaxf(am[u], __shfl_xor_sync(0xffffffffu, am[u], off));
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int n = first + i + u * RPI;
            const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v[u]);
            const float f = fit_half(am[u]);
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 x = __bfloat1622float2(p[k]);
              h[k] = pack_half2(x.x * f, x.y * f);
            }
            *reinterpret_cast<uint4*>(at(n)) = make_uint4(h[0], h[1], h[2], h[3]);
            if (c == 0) muls[n] = A.scale_log2 * inverse_pow2(f);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(M_QREADY + t));
        __syncwarp();
      }
      const float mul = muls[row];
      // rows behind the last are computed with it and not stored
      const int limit = visible_keys(A, w.kv, w.ql, row_token(A, w.r0 + min(row, w.live - 1)));
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_addr = tmem + lane_off + t * 128;
      const uint32_t o_addr = tmem + lane_off + 256 + t * D;
      float m = -INFINITY, l = 0.f;  // reference maximum of t, sum of weights
      bool ok = !skip;
      for (int j = 0; j < tiles; ++j) {
        const int slot = j % kPageSlots;
        ok = ok && wait_for(bar(M_PAGES + slot), (j / kPageSlots) & 1, err) &&
             wait_for(bar(M_SFULL + t), j & 1, err);
        if (__any_sync(0xffffffffu, !ok)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        float s[128];
        {
          uint32_t v0[32], v1[32], v2[32], v3[32];
          tmem_ld32(s_addr, v0);
          tmem_ld32(s_addr + 32, v1);
          tmem_ld32(s_addr + 64, v2);
          tmem_ld32(s_addr + 96, v3);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            s[i] = __uint_as_float(v0[i]);
            s[32 + i] = __uint_as_float(v1[i]);
            s[64 + i] = __uint_as_float(v2[i]);
            s[96 + i] = __uint_as_float(v3[i]);
          }
        }
        const int lim = min(limit, w.hi) - (w.lo + j * kKeys);
        if (__any_sync(0xffffffffu, lim < kKeys)) mask_row(s, lim);
        float f[8 / GP], y[8 / GP], mt = -INFINITY;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          if (g % GP == 0) {
            const float2 sc = *reinterpret_cast<const float2*>(pages + slot * 8 + g);
            // at least the smallest normal number: -inf stays -inf
            f[g / GP] = fmaxf(mul * sc.x, 1.1754944e-38f);
            y[g / GP] = sc.y;
          }
          const float* x = s + 16 * g;
          const float a = max3f(max3f(x[0], x[1], x[2]), max3f(x[3], x[4], x[5]), x[6]);
          const float b = max3f(max3f(x[7], x[8], x[9]), max3f(x[10], x[11], x[12]), x[13]);
          mt = fmaxf(mt, fmaf(max3f(a, b, fmaxf(x[14], x[15])), f[g / GP], y[g / GP]));
        }
        const bool grow = mt > m + kGrow || (m == -INFINITY && mt > -INFINITY);
        if (__any_sync(0xffffffffu, grow)) {
          const float alpha = grow ? ex2_approx(m - mt) : 1.f;
          if (grow) m = mt;
          l *= alpha;
          // the PV before is complete: it was issued before this tile's QK
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(o_addr + c * 32, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
              tmem_st32(o_addr + c * 32, v);
            }
            tmem_wait_st();
          }
        }
        const float shift = m == -INFINITY ? 0.f : kManyShift - m;
        uint64_t acc[2] = {0ull, 0ull};  // sums of P of one page
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int g = 2 * c; g < 2 * c + 2; ++g) {
            const float d = y[g / GP] + shift;
            const uint64_t f2 = pack_f32x2(f[g / GP], f[g / GP]), d2 = pack_f32x2(d, d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float p0, p1;
              unpack_f32x2(ffma_f32x2(pack_f32x2(s[16 * g + 2 * i], s[16 * g + 2 * i + 1]), f2, d2),
                           p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              pk[(g & 1) * 8 + i] = pack_half2(p0, p1);
              acc[i & 1] = add_f32x2(acc[i & 1], pack_f32x2(p0, p1));
            }
            if (g % GP == GP - 1) {
              float a0, a1;
              unpack_f32x2(add_f32x2(acc[0], acc[1]), a0, a1);
              l = fmaf(a0 + a1, fabsf(pages[slot * 8 + g - (GP - 1)].z), l);
              acc[0] = acc[1] = 0ull;
            }
          }
          tmem_st16(s_addr + c * 16, pk);
          if (c == 1) {  // the first half of PV may start
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(M_PHALF + t));
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(M_PFULL + t));
      }

      // ---------------------------------------------------------- epilogue
      ok = ok && wait_for(bar(M_OFULL + t), 0, err);
      if (__all_sync(0xffffffffu, ok)) {
        __syncwarp();
        tc_fence_after();
        const float mref = m == -INFINITY ? -INFINITY : m - kManyShift;
        const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN stays one
        const int r = w.r0 + row, tok = row_token(A, r), head = w.hk * A.G + r - tok * A.G;
        const long long pr = w.part * kManyTile + row;
        uint8_t* stage = smem + t * C::kTile + (warp & 3) * (32 * D * 2);  // Q's place
        constexpr int CH = D / 8;  // 16-byte chunks per output row
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          if (tiles > 0) {
            tmem_ld32(o_addr + c * 32, v);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          }
          if (w.part >= 0) {
            // 32 rows x 32 channels through shared memory: whole 128-byte runs leave
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                  make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int n = i * 4 + (lane >> 3), rr = warp * 32 + n;
              if (rr < w.live)
                *reinterpret_cast<uint4*>(A.part_o + (w.part * kManyTile + rr) * D + c * 32 +
                                          (lane & 7) * 4) =
                    *reinterpret_cast<const uint4*>(stage + n * 128 +
                                                    (((lane & 7) ^ (n & 7)) << 4));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint4 o;
              o.x = pack_bf16x2(__uint_as_float(v[i]) * inv, __uint_as_float(v[i + 1]) * inv);
              o.y = pack_bf16x2(__uint_as_float(v[i + 2]) * inv, __uint_as_float(v[i + 3]) * inv);
              o.z = pack_bf16x2(__uint_as_float(v[i + 4]) * inv, __uint_as_float(v[i + 5]) * inv);
              o.w = pack_bf16x2(__uint_as_float(v[i + 6]) * inv, __uint_as_float(v[i + 7]) * inv);
              const int chunk = c * 4 + i / 8;
              *reinterpret_cast<uint4*>(stage + lane * (D * 2) + ((chunk ^ (lane & 7)) << 4)) = o;
            }
          }
        }
        if (w.part >= 0) {
          if (valid) *reinterpret_cast<float2*>(A.part_ml + 2 * pr) = make_float2(mref, l);
        } else {
          __syncwarp();
#pragma unroll 4
          for (int i = 0; i < 32; i += 32 / CH) {
            const int n = i + lane / CH, chunk = lane % CH, rr = warp * 32 + n;
            if (rr < w.live) {
              const int q = w.r0 + rr, qt = row_token(A, q);
              *reinterpret_cast<uint4*>((__nv_bfloat16*)A.o + w.b * A.o_sb +
                                        (long long)qt * A.o_st +
                                        (long long)(w.hk * A.G + q - qt * A.G) * D + chunk * 8) =
                  *reinterpret_cast<const uint4*>(stage + n * (D * 2) + ((chunk ^ (n & 7)) << 4));
            }
          }
          if (A.lse && valid)
            A.lse[((long long)w.b * A.H + head) * A.N + tok] = row_lse(mref, l);
        }
      }
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int GP>
cudaError_t launch_many(const CacheAttnArgs& A, unsigned grid, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once_per_device(dev, [] {
    return cudaFuncSetAttribute(cache_attn_many_kernel<D, GP>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Many<D>::kSmem);
  });
  if (e != cudaSuccess) return e;
  cache_attn_many_kernel<D, GP><<<grid, kThreads, Many<D>::kSmem, s>>>(A);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_many_pages(const CacheAttnArgs& A, unsigned grid, cudaStream_t s) {
  switch (A.page) {
    case 16: return launch_many<D, 1>(A, grid, s);
    case 32: return launch_many<D, 2>(A, grid, s);
    case 64: return launch_many<D, 4>(A, grid, s);
    default: return launch_many<D, 8>(A, grid, s);
  }
}

}  // namespace

cudaError_t launch_cache_attn_many(const CacheAttnArgs& A, int D, unsigned grid, cudaStream_t s) {
  return D == 128 ? launch_many_pages<128>(A, grid, s) : launch_many_pages<64>(A, grid, s);
}

}  // namespace mmdit
