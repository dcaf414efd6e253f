// Rotary positions with either pairing, partial bands and scaled frequencies:
// the device side shared by mmdit_rotary (rotary.cu) and by mmdit_cache_append
// (cache.cu), which turns K on its way into the cache.
#pragma once

#include "internal.h"

namespace mmdit {

// Per-pair frequencies in half turns per position (omega / pi, fp64), the
// band ends in pairs as in RopeTab, and how a pair's channels are found.
struct RotaryTab {
  double half_turns[64];
  double magnitude;
  int pt, ph, np;  // pairs [0, pt) turn by t, [pt, ph) by h, [ph, np) by w
  int half;        // pair i of a band: (i, i + d_b / 2) instead of (2i, 2i + 1)
};

// fills `tab`, or returns an mmdit_status with the message set (rotary.cu)
int make_rotary_tab(const mmdit_rotary_params* r, int head_dim, RotaryTab& tab);
// a layout whose segments may hold more tokens than the tensor (rotary.cu)
int check_sequence(const mmdit_layout* L, const char* name, long long& tokens);

// Position in fp64 of token n of the sequence (token_position's formulas);
// tokens behind the last segment sit at (0, 0, 0).
__device__ __forceinline__ void token_position_f64(const DevLayout& L, long long n, double& pt,
                                                   double& ph, double& pw) {
  pt = ph = pw = 0.0;
#pragma unroll 1
  for (int s = 0; s < L.n_seg; ++s) {
    const DevSeg& g = L.seg[s];
    if (n < g.start || n >= (long long)g.start + g.n) continue;
    const int j = (int)(n - g.start);
    if (g.kind == MMDIT_SEG_VIDEO) {
      int t, h, w;
      video_coords(g, j, t, h, w);
      pt = (double)g.t0 + t;
      ph = h;
      pw = w;
    } else if (g.kind == MMDIT_SEG_AUDIO) {
      pt = g.t0 + (double)((long long)j * g.t_num) / g.t_den;
    }
    return;
  }
}

// cos and sin (times the magnitude) of pair m at a position.  The angle of a
// far position loses its fraction of a turn in fp32 (at position 10^6 its
// rounding is 0.06 rad), so all of it is fp64, and cosine and sine are rounded once.
__device__ __forceinline__ void rotary_cos_sin(const RotaryTab& tab, int m, double pt, double ph,
                                               double pw, float& c, float& s) {
  const double pos = m < tab.pt ? pt : (m < tab.ph ? ph : pw);
  double cd, sd;
  sincospi(pos * tab.half_turns[m], &sd, &cd);
  c = (float)(cd * tab.magnitude);
  s = (float)(sd * tab.magnitude);
}

// The two channels of pair m (pairs from np on: the unturned channels).
__device__ __forceinline__ void rotary_channels(const RotaryTab& tab, int m, int& first,
                                                int& second) {
  first = 2 * m;
  second = 2 * m + 1;
  if (tab.half && m < tab.np) {
    const int lo = m < tab.pt ? 0 : (m < tab.ph ? tab.pt : tab.ph);
    const int hi = m < tab.pt ? tab.pt : (m < tab.ph ? tab.ph : tab.np);
    first = lo + m;  // 2 lo + (m - lo)
    second = first + (hi - lo);
  }
}

}  // namespace mmdit
