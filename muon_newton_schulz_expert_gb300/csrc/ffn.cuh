// What the feed-forward kernels share: the activations, and the check of the
// groups' offsets.
#pragma once

#include "tc.cuh"

namespace muon {
namespace {

// act(g) and act'(g): both activations are g * sigmoid(v), with v = g (silu)
// or v = 2 sqrt(2/pi) (g + 0.044715 g^3) (the tanh form of gelu, since
// (1 + tanh(z))/2 = sigmoid(2z)).
__device__ __forceinline__ float sigmoid_of(float g, int act, float *dv) {
  constexpr float c = 1.5957691216057308f, k = 0.044715f;
  float v = g;
  *dv = 1.f;
  if (act == MUON_ACT_GELU) {
    // rounded towards zero, so that a square past fp32's range is its largest value: dv stays
    // finite, and the derivative has it times 0 there
    const float g2 = __fmul_rz(g, g);
    v = c * g * fmaf(k, g2, 1.f);
    *dv = c * fmaf(3.f * k, g2, 1.f);
  }
  return __fdividef(1.f, 1.f + __expf(-v));
}

// dg, du and h of one place from dh, g and u.
__device__ __forceinline__ void gated_gradient(float dh, float g, float u, int act, float *dg, float *du, float *h) {
  float dv;
  const float s = sigmoid_of(g, act, &dv), a = g * s;
  *h = a * u;
  *du = dh * a;
  *dg = dh * u * fmaf(a * (1.f - s), dv, s);
}

// Offsets that do not cut 0..rows into consecutive groups are reported (by one
// warp of a launch; the kernels clamp what they read).
__device__ __forceinline__ void report_offsets(const int64_t *offsets, int experts, long long rows, unsigned *err) {
  if (!offsets) return;
  bool ok = true;
  for (int e = threadIdx.x & 31; e <= experts; e += 32) {
    const long long v = __ldg(offsets + e);
    ok = ok && (e == 0 ? v == 0 : v >= __ldg(offsets + e - 1)) && (e < experts || v == rows);
  }
  if (!__all_sync(0xffffffffu, ok) && (threadIdx.x & 31) == 0) atomicOr(err, kErrDevice);
}

// Walks the tiles of all experts in order, a warp together: every role of every
// CTA walks the same sequence, so the groups' sizes are read from the device
// and the host needs none.  An expert of n rows has ceil(n / row_tile) *
// col_tiles tiles (row_tile 0: col_tiles whatever n is).  32 experts at a time:
// lane i holds the rows of the i-th and the tiles up to and with it.
struct WarpCursor {
  const int64_t *offsets;
  long long rows;
  int experts, row_tile;
  long long col_tiles;
  int base = -32;                       // first expert of the 32
  long long first = 0, upto = 0, all = 0;   // tiles before them, this lane's inclusive sum, their sum
  int lane_lo = 0, lane_hi = 0;
  // the tile at hand
  int e = 0, lo = 0, hi = 0;
  long long index = 0;                  // within its expert

  __device__ WarpCursor(const int64_t *off, long long n, int ex, int rt, long long ct)
      : offsets(off), rows(n), experts(ex), row_tile(rt), col_tiles(ct) {}

  // all lanes of a warp together, with growing t
  __device__ bool seek(long long t) {
    const int lane = threadIdx.x & 31;
    while (t >= first + all) {
      base += 32;
      if (base >= experts) return false;
      first += all;
      const int mine = base + lane;
      long long count = 0;
      if (mine < experts) {
        long long a = 0, b = rows;
        if (offsets) {
          // clamped, so that no offsets can send an access outside the arrays
          a = __ldg(offsets + mine), b = __ldg(offsets + mine + 1);
          a = a < 0 ? 0 : a > rows ? rows : a;
          b = b < a ? a : b > rows ? rows : b;
        }
        lane_lo = (int)a, lane_hi = (int)b;
        // in 32 bits: rows are fewer than 2^31
        count = (row_tile ? ((unsigned)(b - a) + (unsigned)row_tile - 1u) / (unsigned)row_tile : 1u) * col_tiles;
      }
      upto = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      all = __shfl_sync(0xffffffffu, upto, 31);
    }
    const long long r = t - first;
    const int at = __ffs(__ballot_sync(0xffffffffu, r < upto)) - 1;
    const long long before = __shfl_sync(0xffffffffu, upto, at ? at - 1 : 0);
    e = base + at;
    lo = __shfl_sync(0xffffffffu, lane_lo, at);
    hi = __shfl_sync(0xffffffffu, lane_hi, at);
    index = at ? r - before : r;
    return true;
  }
};

}  // namespace
}  // namespace muon
