// mmdit_rotary: rotary positions with both pairings, bands that cover part of
// the head, frequencies scaled for longer sequences, any window of a sequence
// per batch item, and the transposed rotation (the gradient of the rotation).
//
// Pair i of band b turns by pos_b * w_i (SkyReels-V4 digest novelties 4 and 5 for the
// positions):   y1 = M (x1 cos - x2 sin),  y2 = M (x1 sin + x2 cos), with the sine's sign
// changed for the transpose.  One read and one write of every channel: HBM bound.  As in
// rope.cu the angles depend on the token and the pair only, so a thread finds its cosines
// and sines once and streams the heads of Q and K past them.  One B200: a 480p layer
// (33,490 tokens, 24 + 24 heads of 128, bf16, 823 MB) 139 us = 5.9 TB/s, 0.90 of the
// measured copy rate, fp32 259 us = 0.97; one token of eight sequences 4.3 us, of which the
// look-ups, one fp64 angle and the round trip are all.
//
// Interleaved pairs sit inside a thread's 16-byte chunk.  Half pairs are d_b/2
// channels apart, 22 and 21 channels for the bands of a 128-channel head, so
// they meet no alignment: a warp puts its rows in shared memory, turns them
// there pair by pair (consecutive lanes on consecutive channels: no bank
// conflicts), and writes them out in 16-byte chunks again.  The same layer: 180 us
// (0.70: single reads and writes of shared memory), fp32 276 us (0.91).
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "rotary.cuh"

namespace mmdit {

namespace {

struct RotaryJob {
  const void* x;
  void* y;
  int heads;
  long long x_st, x_sb, y_st, y_sb;  // strides in elements
};

struct RotaryArgs {
  RotaryJob job[2];  // Q, K; heads = 0: none
  int N, D, heads;   // heads of both
  int slice;         // heads that one thread streams
  float sign;        // -1: transposed
  const int32_t* first;
  DevLayout layout;
  RotaryTab tab;
};

template <typename T>
__device__ __forceinline__ const uint4* src_of(const RotaryArgs& A, int h, int b, int tok,
                                               int chunk) {
  const RotaryJob& j = A.job[h >= A.job[0].heads];
  const int hh = h >= A.job[0].heads ? h - A.job[0].heads : h;
  return reinterpret_cast<const uint4*>((const T*)j.x + b * j.x_sb + tok * j.x_st +
                                        (long long)hh * A.D) + chunk;
}
template <typename T>
__device__ __forceinline__ uint4* dst_of(const RotaryArgs& A, int h, int b, int tok, int chunk) {
  const RotaryJob& j = A.job[h >= A.job[0].heads];
  const int hh = h >= A.job[0].heads ? h - A.job[0].heads : h;
  return reinterpret_cast<uint4*>((T*)j.y + b * j.y_sb + tok * j.y_st + (long long)hh * A.D) +
         chunk;
}

__device__ __forceinline__ float2 get_pair(const uint4& v, int i, __nv_bfloat16*) {
  return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(&v)[i]);
}
__device__ __forceinline__ float2 get_pair(const uint4& v, int i, float*) {
  return reinterpret_cast<const float2*>(&v)[i];
}
__device__ __forceinline__ void set_pair(uint4& v, int i, float2 y, __nv_bfloat16*) {
  reinterpret_cast<__nv_bfloat162*>(&v)[i] = __float22bfloat162_rn(y);
}
__device__ __forceinline__ void set_pair(uint4& v, int i, float2 y, float*) {
  reinterpret_cast<float2*>(&v)[i] = y;
}

constexpr int kUnroll = 4;  // heads in flight per thread

template <typename T>
__global__ void __launch_bounds__(256) rotary_pairs_kernel(const __grid_constant__ RotaryArgs A) {
  constexpr int P = 8 / sizeof(T);  // pairs per 16-byte chunk
  const int cpr = A.D * (int)sizeof(T) / 16;
  const int tok = blockIdx.x * (256 / cpr) + threadIdx.x / cpr;
  const int chunk = threadIdx.x % cpr;
  const int b = blockIdx.z;
  if (tok >= A.N) return;
  double pt, ph, pw;
  token_position_f64(A.layout, (long long)tok + (A.first ? A.first[b] : 0), pt, ph, pw);
  float c[P], s[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int m = chunk * P + i;
    if (m < A.tab.np) rotary_cos_sin(A.tab, m, pt, ph, pw, c[i], s[i]);
    s[i] *= A.sign;
  }
  const int h0 = blockIdx.y * A.slice, h1 = min(A.heads, h0 + A.slice);
  for (int h = h0; h < h1; h += kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u < h1) v[u] = *src_of<T>(A, h + u, b, tok, chunk);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u >= h1) break;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (chunk * P + i < A.tab.np) {  // unturned channels keep their bits
          const float2 x = get_pair(v[u], i, (T*)nullptr);
          set_pair(v[u], i, make_float2(x.x * c[i] - x.y * s[i], x.x * s[i] + x.y * c[i]),
                   (T*)nullptr);
        }
      }
      *dst_of<T>(A, h + u, b, tok, chunk) = v[u];
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) rotary_halves_kernel(const __grid_constant__ RotaryArgs A) {
  // a warp's 32 chunks are 32 / cpr whole rows; their pairs go over the lanes
  constexpr int kItems = 8 / sizeof(T);  // most pairs a lane turns per step
  __shared__ uint4 buf[8][kUnroll][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cpr = A.D * (int)sizeof(T) / 16, rows = 32 / cpr;
  const int tok0 = (blockIdx.x * 8 + warp) * rows;
  const int tok = tok0 + lane / cpr, chunk = lane % cpr;
  const int b = blockIdx.z;
  if (tok0 >= A.N) return;
  const int items = rows * A.tab.np;
  float c[kItems], s[kItems];
  int i1[kItems], i2[kItems];  // channels of the pair, counted over the warp's rows
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int item = lane + 32 * i;
    if (item >= items) continue;
    const int row = item / A.tab.np, m = item - row * A.tab.np;
    double pt, ph, pw;
    token_position_f64(A.layout, (long long)tok0 + row + (A.first ? A.first[b] : 0), pt, ph, pw);
    rotary_cos_sin(A.tab, m, pt, ph, pw, c[i], s[i]);
    s[i] *= A.sign;
    rotary_channels(A.tab, m, i1[i], i2[i]);
    i1[i] += row * A.D;
    i2[i] += row * A.D;
  }
  const int h0 = blockIdx.y * A.slice, h1 = min(A.heads, h0 + A.slice);
  for (int h = h0; h < h1; h += kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u < h1 && tok < A.N) v[u] = *src_of<T>(A, h + u, b, tok, chunk);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) buf[warp][u][lane] = v[u];
    __syncwarp();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      T* row = reinterpret_cast<T*>(buf[warp][u]);
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        if (lane + 32 * i >= items) continue;
        const float x1 = (float)row[i1[i]], x2 = (float)row[i2[i]];
        row[i1[i]] = (T)(x1 * c[i] - x2 * s[i]);
        row[i2[i]] = (T)(x1 * s[i] + x2 * c[i]);
      }
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u < h1 && tok < A.N) *dst_of<T>(A, h + u, b, tok, chunk) = buf[warp][u][lane];
    __syncwarp();
  }
}

cudaError_t launch_rotary(RotaryArgs& A, int batch, int dtype, cudaStream_t s) {
  const int es = dtype == MMDIT_BF16 ? 2 : 4;
  const int cpr = A.D * es / 16, tpb = 256 / cpr;
  // Heads per thread: all of them share the angles, so as many as leave four
  // blocks for each SM (a single token of a few sequences gets one each).
  const long long blocks = ((long long)A.N + tpb - 1) / tpb * batch;
  const long long want = blocks * A.heads / (4 * 148);
  A.slice = (int)std::max(1LL, std::min<long long>(A.heads, want));
  A.slice = std::max(A.slice, (A.heads + 65534) / 65535);
  if (A.slice > kUnroll) A.slice = (A.slice + kUnroll - 1) / kUnroll * kUnroll;
  const dim3 grid((A.N + tpb - 1) / tpb, (A.heads + A.slice - 1) / A.slice, batch);
  if (dtype == MMDIT_BF16) {
    if (A.tab.half) rotary_halves_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(A);
    else rotary_pairs_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(A);
  } else {
    if (A.tab.half) rotary_halves_kernel<float><<<grid, 256, 0, s>>>(A);
    else rotary_pairs_kernel<float><<<grid, 256, 0, s>>>(A);
  }
  return cudaGetLastError();
}

}  // namespace

int make_rotary_tab(const mmdit_rotary_params* r, int head_dim, RotaryTab& tab) {
  if (r == nullptr) return fail(MMDIT_EINVAL, "rotary parameters are NULL");
  const int dims[3] = {r->dim_t, r->dim_h, r->dim_w};
  long long sum = 0;
  for (int d : dims) {
    if (d < 0 || (d & 1)) return fail(MMDIT_EINVAL, "rotary: band of %d channels", d);
    sum += d;
  }
  if (sum < 2 || sum > head_dim)
    return fail(MMDIT_EINVAL, "rotary: bands of %lld channels in a head of %d", sum, head_dim);
  if (!(r->theta > 0.0) || !isfinite(r->theta) || !(r->magnitude > 0.0) ||
      !isfinite((float)r->magnitude))
    return fail(MMDIT_EINVAL, "rotary: theta and magnitude must be positive and finite");
  if (r->pairing != MMDIT_PAIR_INTERLEAVED && r->pairing != MMDIT_PAIR_HALF)
    return fail(MMDIT_EINVAL, "rotary: bad pairing %d", r->pairing);
  if (r->scaling < MMDIT_SCALE_NONE || r->scaling > MMDIT_SCALE_PARTS)
    return fail(MMDIT_EINVAL, "rotary: bad scaling %d", r->scaling);
  tab = RotaryTab{};
  tab.pt = dims[0] / 2;
  tab.ph = (dims[0] + dims[1]) / 2;
  tab.np = (int)sum / 2;
  tab.half = r->pairing == MMDIT_PAIR_HALF;
  tab.magnitude = r->magnitude;
  const double pi = 3.14159265358979323846;
  int m = 0;
  for (int a = 0; a < 3; ++a) {
    if (dims[a] == 0) continue;
    const double f = r->factor[a];
    if (r->scaling != MMDIT_SCALE_NONE && !(f > 0.0 && isfinite(f)))
      return fail(MMDIT_EINVAL, "rotary: factor %g of band %d", f, a);
    if (r->scaling == MMDIT_SCALE_PARTS &&
        (!(r->trained[a] > 0.0) || !isfinite(r->trained[a]) || !(r->beta_slow >= 0.0) ||
         !(r->beta_fast > r->beta_slow) || !isfinite(r->beta_fast)))
      return fail(MMDIT_EINVAL, "rotary: scaling by parts needs trained > 0, beta_fast > beta_slow >= 0");
    const double d = dims[a];
    double theta = r->theta;
    if (r->scaling == MMDIT_SCALE_NTK && dims[a] > 2) theta *= pow(f, d / (d - 2.0));
    // theta^(-2i/d) from 8 fine and up to 8 coarse powers: one more rounding, 2^-53
    double fine[8], coarse[8];
    for (int i = 0; i < 8; ++i) {
      fine[i] = pow(theta, -2.0 * i / d);
      coarse[i] = 16 * i < dims[a] ? pow(theta, -16.0 * i / d) : 0.0;
    }
    for (int i = 0; i < dims[a] / 2; ++i, ++m) {
      double w = fine[i & 7] * coarse[i >> 3];
      if (r->scaling == MMDIT_SCALE_LINEAR) w /= f;
      if (r->scaling == MMDIT_SCALE_PARTS) {
        const double turns = r->trained[a] * w / (2.0 * pi);
        const double g =
            std::min(1.0, std::max(0.0, (turns - r->beta_slow) / (r->beta_fast - r->beta_slow)));
        w = g * w + (1.0 - g) * w / f;
      }
      tab.half_turns[m] = w / pi;
      // positions reach 2^63 (an audio token's numerator): their product is a number too
      if (!(tab.half_turns[m] < 9e288))  // 2^-64 of the largest double
        return fail(MMDIT_EINVAL, "rotary: frequency %g of pair %d of band %d is out of range", w, i, a);
    }
  }
  return MMDIT_OK;
}

int check_sequence(const mmdit_layout* L, const char* name, long long& tokens) {
  tokens = 0;
  if (L != nullptr && L->n_seg >= 1 && L->n_seg <= MMDIT_MAX_SEGMENTS)
    for (int i = 0; i < L->n_seg; ++i) tokens += L->seg[i].n_tokens;
  if (tokens > INT_MAX) return fail(MMDIT_EINVAL, "%s: layout of %lld tokens", name, tokens);
  return check_layout(L, (int)tokens);
}

}  // namespace mmdit

using namespace mmdit;

extern "C" int mmdit_rotary(const void* q, void* q_out, const mmdit_tensor_desc* q_desc,
                            const mmdit_tensor_desc* q_out_desc, const void* k, void* k_out,
                            const mmdit_tensor_desc* k_desc, const mmdit_tensor_desc* k_out_desc,
                            const mmdit_layout* layout, const mmdit_rotary_params* params,
                            const int32_t* first, int transpose, mmdit_stream_t stream) {
  MMDIT_NVTX("mmdit_rotary");
  if (q == nullptr && k == nullptr) {
    // tensors without tokens may have no address; their descriptors tell
    const mmdit_tensor_desc* d = q_desc != nullptr ? q_desc : k_desc;
    if (d == nullptr || d->n_tokens != 0 || q_out != nullptr || k_out != nullptr)
      return fail(MMDIT_EINVAL, "rotary: q and k are both NULL");
    RotaryTab tab;
    long long tokens;
    if (const int rc = check_cache_desc(d, "rotary")) return rc;
    if (const int rc = check_sequence(layout, "rotary", tokens)) return rc;
    return make_rotary_tab(params, d->head_dim, tab);
  }
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const mmdit_tensor_desc* ind[2] = {q_desc, k_desc};
  const mmdit_tensor_desc* outd[2] = {q_out_desc, k_out_desc};
  static const char* const names[4] = {"rotary q", "rotary k", "rotary q_out", "rotary k_out"};
  RotaryArgs A{};
  const mmdit_tensor_desc* ref = nullptr;
  int rc;
  for (int i = 0; i < 2; ++i) {
    if (in[i] == nullptr) {
      if (out[i] != nullptr) return fail(MMDIT_EINVAL, "%s: NULL input for an output", names[i]);
      continue;
    }
    if ((rc = check_cache_desc(ind[i], names[i])) || (rc = check_cache_desc(outd[i], names[2 + i])))
      return rc;
    if (out[i] == nullptr) return fail(MMDIT_EINVAL, "%s is NULL", names[2 + i]);
    if (!aligned16(in[i]) || !aligned16(out[i]))
      return fail(MMDIT_EINVAL, "%s: tensors must be 16-byte aligned", names[i]);
    const mmdit_tensor_desc &x = *ind[i], &y = *outd[i];
    if (x.batch != y.batch || x.n_tokens != y.n_tokens || x.heads != y.heads ||
        x.head_dim != y.head_dim || x.dtype != y.dtype)
      return fail(MMDIT_EINVAL, "%s: input and output descriptors disagree", names[i]);
    if (in[i] == out[i] &&
        (x.stride_tok != y.stride_tok || (x.batch > 1 && x.stride_batch != y.stride_batch)))
      return fail(MMDIT_EINVAL, "%s: in place with two sets of strides", names[i]);
    if (ref != nullptr && (x.batch != ref->batch || x.n_tokens != ref->n_tokens ||
                           x.head_dim != ref->head_dim || x.dtype != ref->dtype))
      return fail(MMDIT_EINVAL, "rotary: q and k disagree on batch, tokens, head_dim or dtype");
    ref = &x;
    A.job[i] = RotaryJob{in[i], out[i], x.heads, x.stride_tok, x.stride_batch,
                         y.stride_tok, y.stride_batch};
    A.heads += x.heads;
  }
  if (q != nullptr && k != nullptr && (q_out == k_out || q_out == k || k_out == q))
    return fail(MMDIT_EINVAL, "rotary: an output aliases the other tensor");
  long long tokens;
  if ((rc = check_sequence(layout, "rotary", tokens))) return rc;
  if (first == nullptr && tokens < ref->n_tokens)
    return fail(MMDIT_EINVAL, "rotary: layout holds %lld tokens, the tensor %d", tokens,
                ref->n_tokens);
  if ((rc = make_rotary_tab(params, ref->head_dim, A.tab))) return rc;
  if (transpose != 0 && transpose != 1)
    return fail(MMDIT_EINVAL, "rotary: transpose must be 0 or 1");
  if (ref->n_tokens == 0) return MMDIT_OK;
  A.N = ref->n_tokens;
  A.D = ref->head_dim;
  A.sign = transpose ? -1.f : 1.f;
  A.first = first;
  A.layout = to_dev(layout);
  if ((rc = check_sm100())) return rc;
  const cudaError_t e = launch_rotary(A, ref->batch, ref->dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? MMDIT_OK : cuda_fail(e, "rotary launch");
}
