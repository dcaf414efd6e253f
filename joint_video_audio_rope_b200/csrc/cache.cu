// The paged 8-bit K/V cache: storing new tokens (mmdit_cache_append) and
// copying pages (mmdit_cache_copy_pages).  Attention over it: cache_attn.cu.
//
// Append.  One CTA takes one page of one item and a slice of the heads.  Per
// head it holds the page's new rows of K and V in registers, finds max |x|
// of both with one block reduction, and writes codes and scales: each value
// is read once (2 or 4 bytes) and written once (1 byte), so the call is HBM
// bound.  A scale is a power of two: e4m3 has its own exponent, so a finer scale would
// buy no precision, and dividing by it, or moving a page to a larger one,
// rounds nothing but the code itself.
//
// Copy.  The page lists travel in the kernel's parameters: no list has to be
// copied to the device first, and one launch moves up to kCopyPairs pages.
#include <cuda_fp8.h>
#include <limits.h>

#include <algorithm>
#include <new>
#include <vector>

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
  int N, slice, mode;  // mode: 0 K as it is, 1 interleaved pairs, 2 half pairs
  const int32_t *start, *count;
  mmdit_cache c;
  int* err;
  DevLayout layout;
  RotaryTab tab;
};

// The power of two s with amax / s in (224, 448], 2^-60 at least.
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
__device__ __forceinline__ float inverse_pow2(float s) {  // s = 2^e, e in -60..120
  return __int_as_float((254 << 23) - __float_as_int(s));
}
__device__ __forceinline__ bool is_number(float x) { return fabsf(x) <= 3.402823466e38f; }

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ float2 value2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
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

// Maximum over the block; `red` is read until the next call with the other buffer.
__device__ __forceinline__ float block_max(float x, float* red, int tid, int warps) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  if ((tid & 31) == 0) red[tid >> 5] = x;
  __syncthreads();
  x = red[tid & 31 & (warps - 1)];  // a power of two of warps
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// The new scale of one half of a (page, head) that holds `older` rows already,
// whose codes move to it if it has grown.
__device__ __forceinline__ float settle_scale(float amax, float* scale, uint8_t* codes, int older,
                                              int D, int tid, int threads) {
  float s = fit_scale(amax);
  if (older > 0) {
    const float old = *scale;
    s = fmaxf(s, floor_scale(old));
    if (s > old) {
      const float f = old / s;
      uint32_t* w = reinterpret_cast<uint32_t*>(codes);
      for (int i = tid; i < older * D / 4; i += threads) {
        const float2 a = value2(w[i] & 0xffffu), c = value2(w[i] >> 16);
        w[i] = codes4(a.x * f, a.y * f, c.x * f, c.y * f);
      }
    }
    __syncthreads();  // every thread has read the old scale
  }
  if (tid == 0) *scale = s;
  return s;
}

// 16 values of K and of V per thread: page * D / 16 threads.
template <typename T, int MODE>
__global__ void __launch_bounds__(1024) append_kernel(const __grid_constant__ AppendArgs A) {
  constexpr int E = 16 / sizeof(T), NV = 16 / E, P = E / 2;
  extern __shared__ __align__(16) uint8_t smem[];  // half pairs: raw K rows, then their codes
  __shared__ float red[2][32];
  __shared__ uint32_t bad[2][4];  // rows with an infinity or NaN in K or V
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
  MMDIT_DCHECK(id >= 0 && id < C.n_pages, A.err);
  if (id < 0 || id >= C.n_pages) return;
  const int r_lo = (int)(max(lo, p * page) - p * page);  // new rows of the page
  const int r_hi = (int)(min(hi, (p + 1) * page) - p * page);
  const long long tok0 = p * page - start;               // input token of row 0

  const int cpr = D / E;  // vectors per row
  const int chunk = tid % cpr, row0 = tid / cpr, rstep = threads / cpr;
  // angles: interleaved, P pairs of each of NV rows; half, one pair of 8 rows
  constexpr int NA = MODE == 1 ? NV * P : (MODE == 2 ? 8 : 1);
  float cs[NA], sn[NA];
  const int m2 = tid % (D / 2), prow0 = tid / (D / 2), pstep = threads / (D / 2);
  int ch1 = 0, ch2 = 0;
  if constexpr (MODE == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      double pt, ph, pw;
      token_position_f64(A.layout, p * page + row0 + i * rstep, pt, ph, pw);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int m = chunk * P + j;
        if (m < A.tab.np) rotary_cos_sin(A.tab, m, pt, ph, pw, cs[i * P + j], sn[i * P + j]);
      }
    }
  }
  if constexpr (MODE == 2) {
    rotary_channels(A.tab, m2, ch1, ch2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      double pt, ph, pw;
      token_position_f64(A.layout, p * page + prow0 + i * pstep, pt, ph, pw);
      if (m2 < A.tab.np) rotary_cos_sin(A.tab, m2, pt, ph, pw, cs[i], sn[i]);
    }
  }
  if (tid < 8) bad[tid >> 2][tid & 3] = 0u;
  __syncthreads();

  const int h0 = blockIdx.y * A.slice, h1 = min(C.heads, h0 + A.slice);
  for (int h = h0; h < h1; ++h) {
    uint32_t* lost = bad[(h - h0) & 1];
    uint4 kr[NV], vr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int row = row0 + i * rstep;
      kr[i] = vr[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row >= r_lo && row < r_hi) {
        const long long at = b * A.sb + (tok0 + row) * A.st + (long long)h * D + chunk * E;
        vr[i] = *reinterpret_cast<const uint4*>((const T*)A.v + at);
        kr[i] = *reinterpret_cast<const uint4*>((const T*)A.k + at);
      }
    }
    const long long ph = (long long)id * C.heads + h;
    uint8_t* kc = (uint8_t*)C.k + ph * page * D;
    uint8_t* vc = (uint8_t*)C.v + ph * page * D;
    float x[E];

    // ---- V: what is not a number becomes 0, and its row is marked
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      values_of(vr[i], x, (T*)nullptr);
      bool ok = true;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        if (is_number(x[j])) am = fmaxf(am, fabsf(x[j]));
        else ok = false;
      }
      if (!ok) {
        const int row = row0 + i * rstep;
        atomicOr(&lost[row >> 5], 1u << (row & 31));
      }
      if constexpr (MODE == 2)
        *reinterpret_cast<uint4*>(smem + (size_t)(tid + i * threads) * 16) = kr[i];
    }
    am = block_max(am, red[0], tid, warps);
    // the next head's marks: the last ones there were read before that barrier
    if (tid < 4) bad[(h - h0 + 1) & 1][tid] = 0u;
    float s = settle_scale(am, C.v_scale + ph, vc, r_lo, D, tid, threads);
    float is = inverse_pow2(s);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int row = row0 + i * rstep;
      if (row < r_lo || row >= r_hi) continue;
      values_of(vr[i], x, (T*)nullptr);
      uint32_t w[E / 4];
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = is_number(x[j]) ? x[j] * is : 0.f;
#pragma unroll
      for (int j = 0; j < E / 4; ++j)
        w[j] = codes4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
      if constexpr (E == 8)
        *reinterpret_cast<uint2*>(vc + row * D + chunk * E) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(vc + row * D + chunk * E) = w[0];
    }

    // ---- K, turned
    float kx[16];
    am = 0.f;
    if constexpr (MODE == 2) {
      // the raw rows were complete at block_max's barrier
      const T* raw = reinterpret_cast<const T*>(smem);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = prow0 + i * pstep;
        const float x1 = (float)raw[row * D + ch1], x2 = (float)raw[row * D + ch2];
        if (!is_number(x1) || !is_number(x2)) atomicOr(&lost[row >> 5], 1u << (row & 31));
        const bool turned = m2 < A.tab.np;
        kx[2 * i] = turned ? x1 * cs[i] - x2 * sn[i] : x1;
        kx[2 * i + 1] = turned ? x1 * sn[i] + x2 * cs[i] : x2;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        values_of(kr[i], x, (T*)nullptr);
        bool ok = true;
#pragma unroll
        for (int j = 0; j < E; ++j) ok = ok && is_number(x[j]);
        if (!ok) {
          const int row = row0 + i * rstep;
          atomicOr(&lost[row >> 5], 1u << (row & 31));
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
          float x1 = x[2 * j], x2 = x[2 * j + 1];
          if (MODE == 1 && chunk * P + j < A.tab.np) {
            x1 = x[2 * j] * cs[(i * P + j) % NA] - x[2 * j + 1] * sn[(i * P + j) % NA];
            x2 = x[2 * j] * sn[(i * P + j) % NA] + x[2 * j + 1] * cs[(i * P + j) % NA];
          }
          kx[i * E + 2 * j] = x1;
          kx[i * E + 2 * j + 1] = x2;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (is_number(kx[j])) am = fmaxf(am, fabsf(kx[j]));
    am = block_max(am, red[1], tid, warps);
    s = settle_scale(am, C.k_scale + ph, kc, r_lo, D, tid, threads);
    is = inverse_pow2(s);
    if constexpr (MODE == 2) {
      uint8_t* tile = smem + (size_t)page * D * sizeof(T);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = prow0 + i * pstep;
        const uint32_t two = codes4(kx[2 * i] * is, kx[2 * i + 1] * is, 0.f, 0.f);
        tile[row * D + ch1] = (uint8_t)two;
        tile[row * D + ch2] = (uint8_t)(two >> 8);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int row = row0 + i * rstep;
      if (row < r_lo || row >= r_hi) continue;
      uint32_t w[E / 4];
#pragma unroll
      for (int j = 0; j < E / 4; ++j) {
        if constexpr (MODE == 2)
          w[j] = *reinterpret_cast<const uint32_t*>(smem + (size_t)page * D * sizeof(T) + row * D +
                                                    chunk * E + 4 * j);
        else
          w[j] = codes4(kx[i * E + 4 * j] * is, kx[i * E + 4 * j + 1] * is,
                        kx[i * E + 4 * j + 2] * is, kx[i * E + 4 * j + 3] * is);
        if ((lost[row >> 5] >> (row & 31)) & 1u) w[j] = 0x7f7f7f7fu;
      }
      if constexpr (E == 8)
        *reinterpret_cast<uint2*>(kc + row * D + chunk * E) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(kc + row * D + chunk * E) = w[0];
    }
  }
}

template <typename T, int MODE>
cudaError_t launch_append_mode(const AppendArgs& A, dim3 grid, int threads, size_t smem,
                               cudaStream_t s) {
  if (MODE == 2) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = once_per_device(dev, [] {
      return cudaFuncSetAttribute(append_kernel<T, MODE>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  128 * 128 * ((int)sizeof(T) + 1));
    });
    if (e != cudaSuccess) return e;
  }
  append_kernel<T, MODE><<<grid, threads, MODE == 2 ? smem : 0, s>>>(A);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_append(AppendArgs& A, int batch, cudaStream_t s) {
  const int page = A.c.page_tokens, D = A.c.head_dim;
  const int threads = page * D / 16;
  const int pages = (A.N + page - 2) / page + 1;  // most pages that N tokens touch
  // Heads per CTA: the angles of a page are found once for all of them, so as
  // many as leave two full waves of CTAs.
  const long long ctas = (long long)pages * batch * A.c.heads;
  const long long wave = 148LL * (1024 / threads);
  A.slice = (int)std::max(1LL, std::min<long long>(A.c.heads, ctas / (2 * wave)));
  const dim3 grid(pages, (A.c.heads + A.slice - 1) / A.slice, batch);
  const size_t smem = (size_t)page * D * (sizeof(T) + 1);
  if (A.mode == 0) return launch_append_mode<T, 0>(A, grid, threads, 0, s);
  if (A.mode == 1) return launch_append_mode<T, 1>(A, grid, threads, 0, s);
  return launch_append_mode<T, 2>(A, grid, threads, smem, s);
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
  if (!k || !v || !start) return fail(MMDIT_EINVAL, "cache_append: k, v and start must be non-NULL");
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
  if ((A.err = device_error_flag()) == nullptr)
    return fail(MMDIT_ECUDA, "device error flag unavailable");
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
