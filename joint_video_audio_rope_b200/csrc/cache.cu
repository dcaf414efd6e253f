// The paged 8-bit K/V cache: storing new tokens (mmdit_cache_append) and
// copying pages (mmdit_cache_copy_pages).  Attention over it: cache_attn.cu.
//
// Append.  One CTA takes one page of one item and a slice of the heads, and
// finds the page's angles once, into shared memory.  The raw rows of K and V of the next
// head are copied into a two-stage ring (cp.async; the first head's while the angles are
// found) while the current head's maxima are found with one block reduction and its
// codes and scales written: each value is read once (2 or 4 bytes) and written once (1
// byte), so the call is HBM bound.  A scale is a power of two: e4m3 has its own
// exponent, so a finer scale would buy no precision, and dividing by it, or moving a page
// to a larger one, rounds nothing but the code itself.
//
// Copy.  The page lists travel in the kernel's parameters: no list has to be
// copied to the device first, and one launch moves up to kCopyPairs pages.
//
// One B200: 32,760 tokens x 24 heads of 128 in bf16 (604 MB, floor 92 us) 107 us as they are,
// 126 us with interleaved rotation, 163 us with half pairs (whose partners meet no
// alignment and cost single reads and writes of shared memory, and issue slots); 15,600 fp32
// tokens x 12 heads of 64 (120 MB, floor 18 us) 25, 31 and 36 us; 400 pages (315 MB, floor 48 us) 52 us.
#include <limits.h>

#include <algorithm>
#include <new>
#include <type_traits>
#include <vector>

#include "cache.cuh"
#include "rotary.cuh"

namespace mmdit {

int check_cache_desc(const mmdit_tensor_desc* d, const char* name) {
  if (d == nullptr) return fail(MMDIT_EINVAL, "%s: descriptor is NULL", name);
  if (d->batch < 1 || d->batch > 65535 || d->n_tokens < 0 || d->heads < 1 || d->heads > 65535)
    return fail(MMDIT_EINVAL, "%s: batch=%d n_tokens=%d heads=%d out of range", name, d->batch,
                d->n_tokens, d->heads);
  if (d->dtype != MMDIT_BF16 && d->dtype != MMDIT_F32)
    return fail(MMDIT_EUNSUPPORTED, "%s: dtype %d not supported", name, d->dtype);
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(MMDIT_EUNSUPPORTED, "%s: head_dim must be 64 or 128 (got %d)", name, d->head_dim);
  const long long row = (long long)d->heads * d->head_dim;
  if (d->stride_tok < row)
    return fail(MMDIT_EINVAL, "%s: stride_tok %lld < heads*head_dim %lld", name,
                (long long)d->stride_tok, row);
  // the last item needs no room behind its last token
  if (d->batch > 1 && d->n_tokens > 0 &&
      d->stride_batch < d->stride_tok * (long long)(d->n_tokens - 1) + row)
    return fail(MMDIT_EINVAL, "%s: stride_batch %lld overlaps batch items", name,
                (long long)d->stride_batch);
  const int es = d->dtype == MMDIT_BF16 ? 2 : 4;
  if ((d->stride_tok * es) % 16 != 0 || (d->batch > 1 && (d->stride_batch * es) % 16 != 0))
    return fail(MMDIT_EINVAL, "%s: strides must be multiples of 16 bytes", name);
  return MMDIT_OK;
}

int check_cache(const mmdit_cache* c, const char* name, bool table) {
  if (c == nullptr) return fail(MMDIT_EINVAL, "%s: cache is NULL", name);
  if (!c->k || !c->v || !c->k_scale || !c->v_scale)
    return fail(MMDIT_EINVAL, "%s: every array of the cache must be non-NULL", name);
  if (!aligned16(c->k) || !aligned16(c->v) || (reinterpret_cast<uintptr_t>(c->k_scale) & 3u) ||
      (reinterpret_cast<uintptr_t>(c->v_scale) & 3u))
    return fail(MMDIT_EINVAL, "%s: codes must be 16-byte and scales 4-byte aligned", name);
  if (c->k == c->v || c->k_scale == c->v_scale)
    return fail(MMDIT_EINVAL, "%s: K and V share an array", name);
  if (c->n_pages < 1 || c->heads < 1 || c->heads > 65535)
    return fail(MMDIT_EINVAL, "%s: n_pages=%d heads=%d out of range", name, c->n_pages, c->heads);
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
    return fail(MMDIT_EUNSUPPORTED, "%s: page_tokens must be 16, 32, 64 or 128 (got %d)", name,
                c->page_tokens);
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(MMDIT_EUNSUPPORTED, "%s: cache head_dim must be 64 or 128 (got %d)", name,
                c->head_dim);
  if (table) {
    if (c->page_table == nullptr || (reinterpret_cast<uintptr_t>(c->page_table) & 3u))
      return fail(MMDIT_EINVAL, "%s: page_table must be an aligned device int32 array", name);
    if (c->batch < 1 || c->batch > 65535 || c->max_pages < 1 ||
        (long long)c->max_pages * c->page_tokens > INT_MAX - (1 << 20))
      return fail(MMDIT_EINVAL, "%s: cache batch=%d max_pages=%d out of range", name, c->batch,
                  c->max_pages);
  }
  return MMDIT_OK;
}

namespace {

struct AppendArgs {
  const void *k, *v;
  long long st, sb;
  int N, slice, cluster, stages, mode;  // mode: 0 K as it is, 1 interleaved pairs, 2 half pairs
  const int32_t *start, *count;
  mmdit_cache c;
  DevLayout layout;
  RotaryTab tab;
};

// The power of two s with amax / s in (224, 448], 2^-60 at least (2^120 at most: amax < 2^128).
__device__ __forceinline__ float fit_scale(float amax) {
  const int bits = __float_as_int(amax);
  int e = (bits >> 23) - 127 - 8;         // amax = m 2^(e + 8), m in [1, 2)
  if ((bits & 0x7fffff) > 0x600000) ++e;  // m > 1.75: 448 = 1.75 * 2^8
  return __int_as_float((max(e, -60) + 127) << 23);
}
// The scale that older tokens of the page hold it to: theirs, rounded up to a
// power of two.
__device__ __forceinline__ float floor_scale(float old) {
  if (!(old > 0.f)) return 0.f;
  const int bits = __float_as_int(old);
  return __int_as_float((bits + 0x7fffff) & 0x7f800000);
}
__device__ __forceinline__ bool is_number(float x) { return fabsf(x) <= 3.402823466e38f; }

// Four values as e4m3 codes, to nearest, clipped to +-448; and the values of four codes.
// As 32-bit registers: the 16-bit halves of the type's C++ interface cost more than the
// conversions.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ void values4(uint32_t codes, float2& a, float2& b) {
  uint32_t lo, hi;
  halves_of(codes, lo, hi);
  a = unpack_half2(lo);
  b = unpack_half2(hi);
}

// the values of one 16-byte vector
__device__ __forceinline__ void values_of(const uint4& r, float (&x)[8], __nv_bfloat16*) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(p[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void values_of(const uint4& r, float (&x)[4], float*) {
  const float* p = reinterpret_cast<const float*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = p[i];
}

// the values of one 16-byte vector times a power of two (exact in bf16 too: what falls
// below its subnormals is far below the smallest code)
__device__ __forceinline__ void scaled_values(uint4 r, float f, float (&x)[8], __nv_bfloat16*) {
  __nv_bfloat162* p = reinterpret_cast<__nv_bfloat162*>(&r);
  const __nv_bfloat162 f2 = __float2bfloat162_rn(f);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = __hmul2(p[i], f2);
  values_of(r, x, (__nv_bfloat16*)nullptr);
}
__device__ __forceinline__ void scaled_values(const uint4& r, float f, float (&x)[4], float*) {
  values_of(r, x, (float*)nullptr);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] *= f;
}

// Maxima that a NaN wins.  Non-negative values order as their bits do, infinity and
// NaN above every number, so the rest of a reduction runs on integers.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t abs_bits(float a, float b, uint32_t m) {
  return __float_as_uint(max3_nan(fabsf(a), fabsf(b), __uint_as_float(m)));
}
// bits of the largest |x| of a raw vector and of `m`
__device__ __forceinline__ uint32_t vector_max(const uint4& r, uint32_t m, __nv_bfloat16*) {
  const uint32_t k = 0x7fff7fffu;
  const uint32_t p =
      __vmaxu2(__vmaxu2(r.x & k, r.y & k), __vmaxu2(r.z & k, r.w & k));
  return max(m, max(p & 0xffff0000u, p << 16));
}
__device__ __forceinline__ uint32_t vector_max(const uint4& r, uint32_t m, float*) {
  m = abs_bits(__uint_as_float(r.x), __uint_as_float(r.y), m);
  return abs_bits(__uint_as_float(r.z), __uint_as_float(r.w), m);
}
// Zeros in place of infinities and NaN; false if there were any.
__device__ __forceinline__ bool keep_numbers(uint4& r, __nv_bfloat16*) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u, ok = false;
    if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu, ok = false;
  }
  return ok;
}
__device__ __forceinline__ bool keep_numbers(uint4& r, float*) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] = 0u, ok = false;
  return ok;
}

// Moves the codes of a page's older rows to a scale that has grown.
__device__ __forceinline__ void rescale_codes(uint8_t* codes, int n, float f, int tid,
                                              int threads) {
  uint32_t* w = reinterpret_cast<uint32_t*>(codes);
  for (int i = tid; i < n / 4; i += threads) {
    float2 a, c;
    values4(w[i], a, c);
    w[i] = codes4(a.x * f, a.y * f, c.x * f, c.y * f);
  }
}

constexpr int kAppendCluster = 8;  // most CTAs that share a page's angles
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// x at the shared address `to` of the cluster's CTA `rank`
__device__ __forceinline__ void store_cluster(uint32_t to, int rank, float2 x) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.v2.f32 [a], {%2, %3};\n\t}" ::"r"(to),
      "r"(rank), "f"(x.x), "f"(x.y)
      : "memory");
}

// MODE: 0 K as it is, 1 interleaved pairs, 2 half pairs.  A thread has NV 16-byte vectors
// of K and of V of each head: vectors tid + i threads of the page's rows.
template <typename T, int MODE, int NV>
__global__ void __launch_bounds__(512, NV == 2 ? 2 : 1)
    append_kernel(const __grid_constant__ AppendArgs A) {
  constexpr int E = 16 / sizeof(T), P = E / 2;
  constexpr int NP = NV * P;  // half pairs: pairs per thread
  // the raw rows of K and V of `stages` heads; angles [page][D / 2] (cos, sin); half pairs:
  // K's codes
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint2 red[2][16];  // by head parity: maxima of V and K per warp
  __shared__ uint32_t lost[4];  // rows with an infinity or NaN in K or V
  __shared__ double place[MODE == 0 ? 1 : 128][3];  // positions of the page's new rows
  const mmdit_cache& C = A.c;
  const int page = C.page_tokens, D = C.head_dim;
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5;
  const int b = blockIdx.z;
  const long long start = A.start[b];
  const int cnt = A.count ? min(max(A.count[b], 0), A.N) : A.N;
  const long long lo = start > 0 ? start : 0;
  const long long cap = (long long)C.max_pages * page;
  const long long hi = start + cnt < cap ? start + cnt : cap;
  const long long p = lo / page + blockIdx.x;
  if (cnt <= 0 || p * page >= hi) return;
  const int id = C.page_table[(long long)b * C.max_pages + p];
  const int r_lo = (int)(max(lo, p * page) - p * page);  // new rows of the page
  const int r_hi = (int)(min(hi, (p + 1) * page) - p * page);
  const long long tok0 = p * page - start;               // input token of row 0

  const int cpr = D / E;  // vectors per row
  const int chunk = tid % cpr, row0 = tid / cpr, rstep = threads / cpr;
  const int half = page * D * (int)sizeof(T);  // bytes of K's (or V's) rows of a head
  float2* angles = reinterpret_cast<float2*>(smem + (size_t)A.stages * 2 * half);
  uint8_t* tile = reinterpret_cast<uint8_t*>(angles) + (size_t)page * D * 4;

  const int h0 = blockIdx.y * A.slice, h1 = min(C.heads, h0 + A.slice);
  const long long from0 = b * A.sb + (tok0 + row0) * A.st + chunk * E, step = rstep * A.st;
  const uint32_t ring = smem_u32(smem) + tid * 16;
  // copies a head's new rows into its stage; each thread reads its own vectors again
  auto load = [&](int h) {
    const T *kp = (const T*)A.k + from0 + (long long)h * D, *vp = (const T*)A.v + from0 + (long long)h * D;
    const uint32_t to = ring + (A.stages == 2 ? (h - h0) & 1 : 0) * 2 * half;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int row = row0 + i * rstep;
      if (row >= r_lo && row < r_hi) {
        cp_async16(to + i * threads * 16, kp + i * step);
        cp_async16(to + half + i * threads * 16, vp + i * step);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (h0 < h1) load(h0);  // under way while the angles are found

  // Interleaved bf16 pairs: a thread reads four angles as two 16-byte vectors.  The first
  // vectors of a row's chunks come first, then the second ones, so that
  // neighbouring threads read neighbouring vectors (no bank conflicts).
  const int m2 = tid % (D / 2), prow0 = tid / (D / 2), pstep = threads / (D / 2);
  const int angle_at =
      MODE == 1 && P == 4 ? (m2 & 1) | (m2 >> 2) << 1 | ((m2 >> 1) & 1) * (D / 4) : m2;
  int ch1 = 0, ch2 = 0;
  if constexpr (MODE == 2) rotary_channels(A.tab, m2, ch1, ch2);
  if constexpr (MODE != 0) {
    // The CTAs of a cluster share the page: each finds its part of the angles and
    // writes it to all of them.
    cluster_arrive();
    for (int r = tid; r < r_hi - r_lo; r += threads) {
      double* at = place[r_lo + r];
      token_position_f64(A.layout, p * page + r_lo + r, at[0], at[1], at[2]);
    }
    __syncthreads();
    const int size = A.cluster, rank = blockIdx.y % size;
    cluster_wait();  // every CTA of the cluster has started
    for (int row = r_lo + rank * pstep + prow0; row < r_hi; row += size * pstep) {
      float2 cs = make_float2(1.f, 0.f);
      if (m2 < A.tab.np) {
        const double* at = place[row];
        rotary_cos_sin(A.tab, m2, at[0], at[1], at[2], cs.x, cs.y);
      }
      const uint32_t to = smem_u32(angles + row * (D / 2) + angle_at);
      for (int r = 0; r < size; ++r) store_cluster(to, r, cs);
    }
    cluster_arrive();
    cluster_wait();
  }

  // the page's id is first needed here: its load ran under the work on the angles.  An id
  // outside the cache stands for a page that is not there (no error)
  if (id < 0 || id >= C.n_pages) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }

  constexpr uint32_t kInf = 0x7f800000u;
  // WHOLE: every row of the page is new, which spares the rows' checks.
  auto store_heads = [&](auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    auto live = [&](int row) { return WHOLE || (row >= r_lo && row < r_hi); };
    for (int h = h0; h < h1; ++h) {
      const int par = (h - h0) & 1;
      if (A.stages == 2 && h + 1 < h1) {
        load(h + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      const uint8_t* raw = smem + (A.stages == 2 ? par : 0) * 2 * half;
      auto k_vec = [&](int i) { return *reinterpret_cast<const uint4*>(raw + (tid + i * threads) * 16); };
      auto v_vec = [&](int i) {
        return *reinterpret_cast<const uint4*>(raw + half + (tid + i * threads) * 16);
      };
      const long long ph = (long long)id * C.heads + h;
      uint8_t* kc = (uint8_t*)C.k + ph * page * D;
      uint8_t* vc = (uint8_t*)C.v + ph * page * D;
      float old_k = 0.f, old_v = 0.f;
      if (!WHOLE && r_lo > 0) old_k = C.k_scale[ph], old_v = C.v_scale[ph];

      // ---- K turned, and the largest |x|
      [[maybe_unused]] float kx[MODE == 0 ? 1 : NV * E];
      uint32_t mv = 0u, mk = 0u;
      if constexpr (MODE == 2) {
        __syncthreads();  // the rows that other threads copied
        const T* rows = reinterpret_cast<const T*>(raw);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int row = prow0 + i * pstep;
          kx[2 * i] = kx[2 * i + 1] = 0.f;
          if (!live(row)) continue;
          const float x1 = (float)rows[row * D + ch1], x2 = (float)rows[row * D + ch2];
          const float2 cs = angles[row * (D / 2) + m2];
          kx[2 * i] = x1 * cs.x - x2 * cs.y;
          kx[2 * i + 1] = x1 * cs.y + x2 * cs.x;
          mk = abs_bits(kx[2 * i], kx[2 * i + 1], mk);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int row = row0 + i * rstep;
        if (!live(row)) continue;
        mv = vector_max(v_vec(i), mv, (T*)nullptr);
        if constexpr (MODE == 0) mk = vector_max(k_vec(i), mk, (T*)nullptr);
        if constexpr (MODE == 1) {
          float x[E];
          values_of(k_vec(i), x, (T*)nullptr);
          const float4* a = reinterpret_cast<const float4*>(angles + row * (D / 2)) + chunk;
          float4 two;
#pragma unroll
          for (int j = 0; j < P; ++j) {
            if (j % 2 == 0) two = a[j / 2 * (D / 8)];
            const float2 cs = j % 2 ? make_float2(two.z, two.w) : make_float2(two.x, two.y);
            const float t1 = x[2 * j] * cs.x - x[2 * j + 1] * cs.y;
            const float t2 = x[2 * j] * cs.y + x[2 * j + 1] * cs.x;
            kx[i * E + 2 * j] = t1;
            kx[i * E + 2 * j + 1] = t2;
            mk = abs_bits(t1, t2, mk);
          }
        }
      }
      auto block_max = [&](uint2* r) {
        mv = __reduce_max_sync(0xffffffffu, mv);
        mk = __reduce_max_sync(0xffffffffu, mk);
        if ((tid & 31) == 0) r[tid >> 5] = make_uint2(mv, mk);
        __syncthreads();
        for (int i = 0; i < warps; ++i) {
          const uint2 m = r[i];
          mv = max(mv, m.x);
          mk = max(mk, m.y);
        }
      };
      block_max(red[par]);
      const bool careful = max(mv, mk) >= kInf;  // the same in every thread
      if (careful) {
        // an infinity or NaN: mark its rows, leave it out of V and of the maxima
        __syncthreads();
        if (tid < 4) lost[tid] = 0u;
        __syncthreads();
        mv = mk = 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int row = row0 + i * rstep;
          if (!live(row)) continue;
          uint4 v = v_vec(i), k = k_vec(i);
          bool ok = keep_numbers(v, (T*)nullptr);
          mv = vector_max(v, mv, (T*)nullptr);
          ok = keep_numbers(k, (T*)nullptr) && ok;
          if constexpr (MODE == 0) mk = vector_max(k, mk, (T*)nullptr);
          if (!ok) atomicOr(&lost[row >> 5], 1u << (row & 31));
        }
        if constexpr (MODE != 0) {
#pragma unroll
          for (int j = 0; j < NV * E; ++j)
            if (WHOLE || MODE == 2 || live(row0 + j / E * rstep))
              if (is_number(kx[j])) mk = abs_bits(kx[j], 0.f, mk);
          // Turned values that overflowed mark their rows too.  Found from the raw rows again, pair
          // m2 of each: a few instructions that run almost never, while rows found from kx cost the
          // other path registers (480p clip, half pairs: 221 us instead of 166).
          const int c1 = MODE == 2 ? ch1 : 2 * m2, c2 = MODE == 2 ? ch2 : 2 * m2 + 1;
#pragma unroll 1
          for (int row = prow0; row < page; row += pstep) {
            if (!live(row)) continue;
            const T* at = reinterpret_cast<const T*>(raw) + row * D;
            const float x1 = (float)at[c1], x2 = (float)at[c2];
            const float2 cs = angles[row * (D / 2) + angle_at];
            if (!is_number(x1 * cs.x - x2 * cs.y) || !is_number(x1 * cs.y + x2 * cs.x))
              atomicOr(&lost[row >> 5], 1u << (row & 31));
          }
        }
        block_max(red[par]);
      }

      // ---- scales; every thread has read the old ones before that barrier
      float sv = fit_scale(__uint_as_float(mv)), sk = fit_scale(__uint_as_float(mk));
      if (!WHOLE && r_lo > 0) {
        sv = fmaxf(sv, floor_scale(old_v));
        sk = fmaxf(sk, floor_scale(old_k));
        if (sv > old_v) rescale_codes(vc, r_lo * D, old_v / sv, tid, threads);
        if (sk > old_k) rescale_codes(kc, r_lo * D, old_k / sk, tid, threads);
      }
      if (tid == 0) {
        C.v_scale[ph] = sv;
        C.k_scale[ph] = sk;
      }
      const float iv = inverse_pow2(sv), ik = inverse_pow2(sk);

      // ---- codes
      if constexpr (MODE == 2) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int row = prow0 + i * pstep;
          const uint32_t two = codes4(kx[2 * i] * ik, kx[2 * i + 1] * ik, 0.f, 0.f);
          tile[row * D + ch1] = (uint8_t)two;
          tile[row * D + ch2] = (uint8_t)(two >> 8);
        }
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int row = row0 + i * rstep;
        if (!live(row)) continue;
        const int to = row * D + chunk * E;
        uint32_t w[E / 4], v[E / 4];
        float x[E];
        uint4 r = v_vec(i);
        if (careful) keep_numbers(r, (T*)nullptr);
        scaled_values(r, iv, x, (T*)nullptr);
#pragma unroll
        for (int j = 0; j < E / 4; ++j)
          v[j] = codes4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        if constexpr (MODE == 2) {
#pragma unroll
          for (int j = 0; j < E / 4; ++j) w[j] = *reinterpret_cast<const uint32_t*>(tile + to + 4 * j);
        } else {
          if constexpr (MODE == 0) {
            scaled_values(k_vec(i), ik, x, (T*)nullptr);
          } else {
#pragma unroll
            for (int j = 0; j < E; ++j) x[j] = kx[i * E + j] * ik;
          }
#pragma unroll
          for (int j = 0; j < E / 4; ++j)
            w[j] = codes4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        }
        if (careful && ((lost[row >> 5] >> (row & 31)) & 1u)) {
#pragma unroll
          for (int j = 0; j < E / 4; ++j) w[j] = 0x7f7f7f7fu;
        }
        if constexpr (E == 8) {
          *reinterpret_cast<uint2*>(vc + to) = make_uint2(v[0], v[1]);
          *reinterpret_cast<uint2*>(kc + to) = make_uint2(w[0], w[1]);
        } else {
          *reinterpret_cast<uint32_t*>(vc + to) = v[0];
          *reinterpret_cast<uint32_t*>(kc + to) = w[0];
        }
      }
      if (A.stages == 1 && h + 1 < h1) {
        if (MODE == 2) __syncthreads();  // every thread is done with the rows
        load(h + 1);
      }
    }
  };
  if (r_lo == 0 && r_hi == page) store_heads(std::true_type{});
  else store_heads(std::false_type{});
}

template <typename T, int MODE, int NV>
cudaError_t launch_append_mode(AppendArgs& A, int batch, cudaStream_t s) {
  const int page = A.c.page_tokens, D = A.c.head_dim;
  const int rows = 2 * page * D * (int)sizeof(T);  // K's and V's rows of a head
  const int threads = rows / (32 * NV);
  const int rest = (MODE == 0 ? 0 : page * D * 4) + (MODE == 2 ? page * D : 0);
  constexpr int kMost = 227 * 1024 - 4096;  // static shared memory and the launch's own
  A.stages = 2 * rows + rest <= kMost ? 2 : 1;
  const int smem = A.stages * rows + rest;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once_per_device(dev, [] {
    return cudaFuncSetAttribute(append_kernel<T, MODE, NV>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  });
  if (e != cudaSuccess) return e;
  const int pages = (int)((A.N + page - 2LL) / page) + 1;  // most pages that N tokens touch
  // Slices of the heads, one CTA each: a CTA takes as long as its heads and about two
  // more for the page's look-ups and angles, and there are as many waves as the CTAs are of
  // what fits (480p clip, bf16, interleaved, side by side: 122 us with one or two slices, 126 with four, 160 with
  // eight; 1,560 tokens of it: 38, 23, 15 and 13).  Where K is turned, the CTAs of a page form
  // clusters of up to eight that share the work on its angles.
  const long long resident =
      148LL * std::max(1, std::min((NV == 2 ? 1024 : 512) / threads, 227 * 1024 / (smem + 4096)));
  int slices = 1, size = 1;
  long long best = 0;
  for (int n = 1; n <= std::min(A.c.heads, 256); n += n < 8 ? n : 8) {
    const long long cost = std::max(resident, (long long)pages * batch * n) *
                           ((A.c.heads + n - 1) / n + 2);
    if (n == 1 || cost < best) best = cost, slices = n;
  }
  A.slice = (A.c.heads + slices - 1) / slices;
  slices = (A.c.heads + A.slice - 1) / A.slice;
  if (MODE != 0) {
    while (size < kAppendCluster && 2 * size <= slices) size *= 2;
    slices = (slices + size - 1) / size * size;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(pages, slices, batch);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = attr.val.clusterDim.z = 1;
  attr.val.clusterDim.y = size;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  A.cluster = size;
  return cudaLaunchKernelEx(&cfg, append_kernel<T, MODE, NV>, A);
}

template <typename T, int NV>
cudaError_t launch_append_pairs(AppendArgs& A, int batch, cudaStream_t s) {
  if (A.mode == 0) return launch_append_mode<T, 0, NV>(A, batch, s);
  if (A.mode == 1) return launch_append_mode<T, 1, NV>(A, batch, s);
  return launch_append_mode<T, 2, NV>(A, batch, s);
}

template <typename T>
cudaError_t launch_append(AppendArgs& A, int batch, cudaStream_t s) {
  // Two vectors of K and of V per thread for pages up to 8 KB, four above (two CTAs of 256
  // threads: 123 us for the 480p clip in pages of 64; 512 threads with two: 144), eight where that
  // would take over 512 threads.
  const int vectors = A.c.page_tokens * A.c.head_dim * (int)sizeof(T) / 16;
  if (vectors <= 512) return launch_append_pairs<T, 2>(A, batch, s);
  if constexpr (sizeof(T) == 4)
    if (vectors > 2048) return launch_append_pairs<T, 8>(A, batch, s);
  return launch_append_pairs<T, 4>(A, batch, s);
}

// Every copy of a call runs at once: a page written twice, or read and written,
// would end in either state.  One bit per page, kept by the thread and cleared
// again: a list costs a few operations per entry, whatever the cache's size.
int check_page_lists(int n, const int32_t* src, const int32_t* dst, int n_pages) {
  thread_local std::vector<uint64_t> marks;
  const size_t words = (size_t)n_pages / 64 + 1;
  try {
    if (marks.size() < words) marks.resize(words);
  } catch (const std::bad_alloc&) {
    return fail(MMDIT_EINVAL, "cache_copy_pages: no host memory for marks of %d pages", n_pages);
  }
  auto marked = [&](int page) { return (marks[page >> 6] >> (page & 63)) & 1u; };
  int twice = -1, both = -1, seen = 0;
  for (; seen < n && twice < 0; ++seen) {
    if (marked(dst[seen])) twice = dst[seen];
    marks[dst[seen] >> 6] |= 1ull << (dst[seen] & 63);
  }
  for (int i = 0; i < n && twice < 0 && both < 0; ++i)
    if (marked(src[i])) both = src[i];
  while (seen-- > 0) marks[dst[seen] >> 6] = 0;
  if (twice >= 0) return fail(MMDIT_EINVAL, "cache_copy_pages: page %d is written twice", twice);
  if (both >= 0) return fail(MMDIT_EINVAL, "cache_copy_pages: page %d is read and written", both);
  return MMDIT_OK;
}

constexpr int kCopyPairs = 480;  // page pairs per launch: 3,840 bytes of parameters
struct CopyArgs {
  uint8_t *k, *v;
  float *ks, *vs;
  long long page_bytes;  // of K or V, a multiple of 1024
  int heads;
  int32_t src[kCopyPairs], dst[kCopyPairs];
};

__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ CopyArgs A) {
  const int src = A.src[blockIdx.y], dst = A.dst[blockIdx.y];
  const long long vecs = A.page_bytes / 16;
  const uint4* from = reinterpret_cast<const uint4*>((blockIdx.z ? A.v : A.k) + src * A.page_bytes);
  uint4* to = reinterpret_cast<uint4*>((blockIdx.z ? A.v : A.k) + dst * A.page_bytes);
  const long long step = (long long)gridDim.x * 1024;
  for (long long i = blockIdx.x * 1024LL + threadIdx.x; i < vecs; i += step) {
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * 256 < vecs) x[u] = from[i + u * 256];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * 256 < vecs) to[i + u * 256] = x[u];
  }
  if (blockIdx.x == 0) {
    float* sc = blockIdx.z ? A.vs : A.ks;
    for (int h = threadIdx.x; h < A.heads; h += 256)
      sc[(long long)dst * A.heads + h] = sc[(long long)src * A.heads + h];
  }
}

}  // namespace

}  // namespace mmdit

using namespace mmdit;

extern "C" {

int mmdit_cache_append(const void* k, const void* v, const mmdit_tensor_desc* desc,
                       const mmdit_cache* cache, const int32_t* start, const int32_t* count,
                       const mmdit_layout* layout, const mmdit_rotary_params* rotary,
                       mmdit_stream_t stream) {
  MMDIT_NVTX("mmdit_cache_append");
  int rc;
  if ((rc = check_cache_desc(desc, "cache_append")) ||
      (rc = check_cache(cache, "cache_append", true)))
    return rc;
  const bool some = desc->n_tokens > 0;  // tensors without tokens may have no address
  if (!start || (some && (!k || !v)))
    return fail(MMDIT_EINVAL, "cache_append: k, v and start must be non-NULL");
  if (!aligned16(k) || !aligned16(v))
    return fail(MMDIT_EINVAL, "cache_append: tensors must be 16-byte aligned");
  if (desc->batch != cache->batch || desc->heads != cache->heads ||
      desc->head_dim != cache->head_dim)
    return fail(MMDIT_EINVAL, "cache_append: tensor and cache disagree on batch, heads or head_dim");
  if ((layout == nullptr) != (rotary == nullptr))
    return fail(MMDIT_EINVAL, "cache_append: layout and rotary go together");
  AppendArgs A{};
  if (rotary != nullptr) {
    long long tokens;
    if ((rc = check_sequence(layout, "cache_append", tokens)) ||
        (rc = make_rotary_tab(rotary, desc->head_dim, A.tab)))
      return rc;
    A.layout = to_dev(layout);
    A.mode = A.tab.half ? 2 : 1;
  }
  if (desc->n_tokens == 0) return MMDIT_OK;
  A.k = k;
  A.v = v;
  A.st = desc->stride_tok;
  A.sb = desc->stride_batch;
  A.N = desc->n_tokens;
  A.start = start;
  A.count = count;
  A.c = *cache;
  if ((rc = check_sm100())) return rc;
  const cudaError_t e = desc->dtype == MMDIT_BF16
                            ? launch_append<__nv_bfloat16>(A, desc->batch, (cudaStream_t)stream)
                            : launch_append<float>(A, desc->batch, (cudaStream_t)stream);
  return e == cudaSuccess ? MMDIT_OK : cuda_fail(e, "cache_append launch");
}

int mmdit_cache_copy_pages(const mmdit_cache* cache, int n, const int32_t* src, const int32_t* dst,
                           mmdit_stream_t stream) {
  MMDIT_NVTX("mmdit_cache_copy_pages");
  int rc;
  if ((rc = check_cache(cache, "cache_copy_pages", false))) return rc;
  if (n < 0) return fail(MMDIT_EINVAL, "cache_copy_pages: n = %d", n);
  if (n == 0) return MMDIT_OK;
  if (!src || !dst) return fail(MMDIT_EINVAL, "cache_copy_pages: src and dst must be non-NULL");
  for (int i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= cache->n_pages || dst[i] < 0 || dst[i] >= cache->n_pages)
      return fail(MMDIT_EINVAL, "cache_copy_pages: pair %d (%d -> %d) outside %d pages", i, src[i],
                  dst[i], cache->n_pages);
  if ((rc = check_page_lists(n, src, dst, cache->n_pages))) return rc;
  if ((rc = check_sm100())) return rc;
  CopyArgs A;
  A.k = (uint8_t*)cache->k;
  A.v = (uint8_t*)cache->v;
  A.ks = cache->k_scale;
  A.vs = cache->v_scale;
  A.page_bytes = (long long)cache->heads * cache->page_tokens * cache->head_dim;
  A.heads = cache->heads;
  for (int at = 0; at < n; at += kCopyPairs) {
    const int m = std::min(kCopyPairs, n - at);
    std::copy(src + at, src + at + m, A.src);
    std::copy(dst + at, dst + at + m, A.dst);
    // 16 KB per CTA and step; many pages: a few longer walks per page instead
    const long long steps = (A.page_bytes + 16383) / 16384;
    const int x = (int)std::max(1LL, std::min(steps, 148LL * 16 / m));
    copy_pages_kernel<<<dim3(x, m, 2), 256, 0, (cudaStream_t)stream>>>(A);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "cache_copy_pages launch");
  }
  return MMDIT_OK;
}

}  // extern "C"
