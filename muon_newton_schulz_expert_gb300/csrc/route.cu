// A router's choice of experts from its logits x [T][E], and the gradient of the
// weights in the logits.
//
//   s = softmax(x) or sigmoid(x); the k experts with the largest s + bias (of x
//   without a bias: both scores grow with x), ties to the lowest index; their
//   weights w_i = scale s_i, or scale s_i / sum of the chosen s
//
// A warp takes a row and keeps its keys in registers (lane l: experts l, l + 32, ..), so the
// logits are read once.  The k-th largest of the lanes' own maxima bounds the k-th largest key
// from below (redux.sync on fp32); the few keys that reach it are gathered in shared memory (k = 8
// of 384: about 10) and ranked by counting who is larger.  The kernel is bound by instructions,
// not by its bytes: 16384 rows of 384 with bias, top 8, took 34 us as k rounds of a warp-wide
// maximum in which the winning lane looked at its values again, 23 us with integer keys made
// of every value, 16.1 us so.  Where ties (a router before its first step, bf16 logits) or a long
// choice leave more candidates, the bound is found by bisection and equal keys are cut off by
// index: all 384 logits and biases equal 71 us, 357 with the choice made in 64 bits; top 32 of
// 1024 bf16 63 and 448 us.  An ordinary row's 10.3 us (no bias) become 10.9 by it.
//
// With a bias the keys are sums of two numbers, and fp32 may not tell two of them apart
// that 64 bits do.  Where two neighbours in the order are closer than the keys' error
// bound, and not equal logits with equal biases, the choice is made again from keys in
// 64 bits: of the candidates (a softmax with a sum that is only close), and where that does not
// settle it or the candidates are not known, of the whole row.  16384 rows of 384, softmax with bias, 17.4 us;
// 28.3 with the whole row in 64 bits for each (1 in a thousand or less).
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace muon {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kMaxTop = 32, kCandidates = 64;
constexpr int64_t kMaxExperts = 1024, kMaxRows = int64_t(1) << 27;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float *d, float v) { *d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16 *d, float v) { *d = __float2bfloat16_rn(v); }

// Whole numbers in the values' order; -0 is 0.  In 64 bits 0 for -inf (never chosen), the largest for NaN.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long order_of(double v) {
  if (v == -INFINITY) return 0ull;
  if (v != v) return ~0ull;
  const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
  return b >> 63 ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ double value_of(unsigned long long k) {
  return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k));
}

__device__ __forceinline__ float warp_max(float v) {   // a NaN counts for nothing
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {   // NaN if any is
  float r;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// 2^x, 1/x: within 2^-22 of themselves
__device__ __forceinline__ float fast_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float fast_inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }
__device__ __forceinline__ double sigmoid(double x) { return 1.0 / (1.0 + exp(-x)); }

struct Args {
  const void *logits;
  int64_t stride;
  const float *bias;
  int64_t rows;
  int experts, top;
  bool softmax, normalize;
  float scale;
  int64_t *ids;
  float *weights;
};

// The choice from keys in 64 bits over a whole row (without a bias a key is the logit): lane j leaves with the
// j-th expert's id.
template <typename T, int R>
__device__ __noinline__ int choose_in_64(const T *x, const float *bias, int experts, int top, bool softmax) {
  const int lane = threadIdx.x & 31;
  double v[R];
#pragma unroll
  for (int i = 0; i < R; ++i) v[i] = i * 32 + lane < experts ? (double)to_f(x[i * 32 + lane]) : -INFINITY;
  if (softmax && bias) {
    double most = v[0], sum = 0.0;
#pragma unroll
    for (int i = 1; i < R; ++i) most = fmax(most, v[i]);
    for (int o = 16; o; o >>= 1) most = fmax(most, __shfl_xor_sync(kAll, most, o));
#pragma unroll 1
    for (int i = 0; i < R; ++i) {
      const double e = v[0] == -INFINITY ? 0.0 : exp(v[0] - most);   // once around: each in turn is v[0]
      sum += e;
#pragma unroll
      for (int k = 0; k + 1 < R; ++k) v[k] = v[k + 1];
      v[R - 1] = e;
    }
    sum = 1.0 / warp_sum(sum);
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] *= sum;
  } else if (bias) {
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = sigmoid(v[i]);
  }
  unsigned long long key[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = i * 32 + lane;
    key[i] = e >= experts || (bias && to_f(x[e]) == -INFINITY) ? 0ull : order_of(bias ? v[i] + (double)bias[e] : v[i]);
  }
  int mine = -1;
  for (int j = 0; j < top; ++j) {
    unsigned long long best = 0ull;
    int at = 0;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (key[i] > best) best = key[i], at = i;
    int e = at * 32 + lane;
    for (int o = 16; o; o >>= 1) {
      const unsigned long long k = __shfl_xor_sync(kAll, best, o);
      const int f = __shfl_xor_sync(kAll, e, o);
      if (k > best || (k == best && f < e)) best = k, e = f;
    }
    if (best == 0ull) break;
    if (lane == j) mine = e;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i * 32 + lane == e) key[i] = 0ull;
  }
  return mine;
}

// A warp's candidates (key and complemented index in one number: the larger comes first), and the first of
// them in order.
typedef unsigned long long Candidate;
__device__ __forceinline__ Candidate candidate(float key, int e) {
  return (Candidate)order_of(key) << 32 | (0xffffffffu - (unsigned)e);
}
// as it is gathered, before its key is put in order
__device__ __forceinline__ Candidate gathered_as(float key, int e) {
  return (Candidate)__float_as_uint(key) << 32 | (unsigned)e;
}
__device__ __forceinline__ int expert_of(Candidate c) { return (int)(0xffffffffu - (unsigned)c); }
__device__ __forceinline__ float key_of(Candidate c) { return value_of((uint32_t)(c >> 32)); }
template <bool BIAS>
struct Gathered {
  Candidate c[kCandidates], sorted[kMaxTop + 1];
  unsigned long long key64[BIAS ? kCandidates : 1], sorted64[BIAS ? kMaxTop + 1 : 1];
};

// A row's softmax sum within 2^-21 of itself: fp32 exponentials (2^-22) of differences with what their rounding left,
// added in 64 bits.  64-bit exponentials of all the row's logits take 26 us for 1024 experts, for one row as for many.
template <typename T>
__device__ __noinline__ double close_sum(const T *x, int experts, float m) {
  double sum = 0.0;
#pragma unroll 4
  for (int e = threadIdx.x & 31; e < experts; e += 32) {
    const float v = to_f(x[e]), d = v - m, b = d - v, rest = (v - (d - b)) - (m + b), y = expf(d);
    sum += y > 0.f ? fmaf(y, rest, y) : 0.f;
  }
  return warp_sum(sum);
}

template <typename T, int R, bool BIAS>
__global__ void __launch_bounds__(kThreads, R <= 12 ? 5 : R <= 16 ? 4 : 3) route_kernel(const Args p) {
  __shared__ Gathered<BIAS> gathered[kWarps];
  const int lane = threadIdx.x & 31;
  Gathered<BIAS> &g = gathered[threadIdx.x >> 5];
  const int64_t row = blockIdx.x * (int64_t)kWarps + (threadIdx.x >> 5);
  if (row >= p.rows) return;   // a warp together
  const T *x = static_cast<const T *>(p.logits) + row * p.stride;
  float key[R], best = -INFINITY;
  float m = -INFINITY, sum = 1.f;
#pragma unroll
  for (int i = 0; i < R; ++i) key[i] = i * 32 + lane < p.experts ? to_f(x[i * 32 + lane]) : -INFINITY;
  // the softmax's sum, where keys or weights need it
  if (p.softmax && (BIAS || !p.normalize)) {
#pragma unroll
    for (int i = 0; i < R; ++i) m = fmaxf(m, key[i]);
    m = warp_max(m);
    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < R; ++i) part[i & 3] += key[i] == -INFINITY ? 0.f : fast_exp(key[i] - m);
    sum = warp_sum((part[0] + part[1]) + (part[2] + part[3]));
  }
  const float inv = 1.f / sum;
  if (BIAS) {
    float bias[R];
#pragma unroll
    for (int i = 0; i < R; ++i) bias[i] = i * 32 + lane < p.experts ? __ldg(p.bias + i * 32 + lane) : 0.f;
    if (p.softmax) {
#pragma unroll
      for (int i = 0; i < R; ++i) key[i] = key[i] == -INFINITY ? key[i] : fmaf(fast_exp(key[i] - m), inv, bias[i]);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        key[i] = key[i] == -INFINITY ? key[i] : fast_inverse(1.f + fast_exp(-key[i])) + bias[i];
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) best = max_nan(best, key[i]);
  // Keys are within eps and 2^-23 of themselves: a fast exponential is within 2^-22 + 2^-24 |its argument| of
  // itself, which a sigmoid turns into 2^-20 at most and a softmax, whose sum of up to 1024 terms takes 14
  // roundings on a path, into 2^-19 of its largest score (s |x - m| is at most 0.37 of that).
  const float eps = p.softmax ? 0x1p-19f * inv : 0x1p-20f;
  // at least `need` keys reach the bound: with a bias one more than the choice, to see how far the border is
  constexpr float kLowest = -3.402823466e38f;   // -inf is no candidate
  const int need = p.top + (BIAS ? 1 : 0);
  float bound = -INFINITY;
  for (int j = 0; j < need; ++j) {
    bound = warp_max_nan(best);
    if (!(bound > -INFINITY)) break;
    if (best == bound) best = -INFINITY;
  }
  bool whole = bound != bound || (BIAS && bound == INFINITY);   // a NaN among the keys; differences of infinities
  const float least = fmaxf(bound, kLowest);
  // what reaches v or may, with the keys' error
  auto below = [&](float v) { return BIAS ? fmaxf(v - (2.f * eps + fabsf(v) * 0x1p-21f), kLowest) : v; };
  // the number of keys that reach `bound`, which are gathered; of those that are `border` the first `room` alone
  auto gather = [&](int room, float border) {
    int count = 0, met = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      bool is = key[i] >= bound;
      if (room) {
        const unsigned on = __ballot_sync(kAll, key[i] == border);
        is = is && (key[i] != border || met + __popc(on & ((1u << lane) - 1u)) < room);
        met += __popc(on);
      }
      const unsigned who = __ballot_sync(kAll, is);
      if (who == 0u) continue;
      const int at = count + __popc(who & ((1u << lane) - 1u));
      if (is && at < kCandidates) g.c[at] = gathered_as(key[i], i * 32 + lane);
      count += __popc(who);
    }
    return count;
  };
  bound = below(least);
  int count = gather(0, 0.f);
  if (!whole && count > kCandidates) {
    // Ties, or a choice so long that the lanes' maxima say little.  The bound by bisection over the numbers in their
    // order, until few enough keys reach it or it is the border itself, with many keys on it or, with a bias, near it.
    auto reach = [&](float v) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) n += key[i] >= v;
      return __reduce_add_sync(kAll, n);
    };
    float most = key[0];
#pragma unroll
    for (int i = 1; i < R; ++i) most = fmaxf(most, key[i]);
    most = warp_max(most);
    uint32_t lo = order_of(least), hi = order_of(most) + 1u;   // `need` keys reach lo, fewer hi
    while (hi - lo > 1u && count > kCandidates) {
      const uint32_t mid = lo + (hi - lo) / 2u;
      if (reach(value_of(mid)) >= need) lo = mid, bound = below(value_of(mid)), count = reach(bound);
      else hi = mid;
    }
    const float border = value_of(lo);
    int room = 0;
    if (count > kCandidates) {   // hi is the next number
      if (BIAS) {
        // sure if none is just below, and those on the border are one logit with one bias
        int first = INT_MAX;
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (key[i] == border) first = min(first, i * 32 + lane);
        first = __reduce_min_sync(kAll, first);
        const float xf = to_f(x[first]), bf = __ldg(p.bias + first);
        bool differ = border == INFINITY || reach(border) != count;
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (key[i] == border) differ = differ || to_f(x[i * 32 + lane]) != xf || __ldg(p.bias + i * 32 + lane) != bf;
        whole = __any_sync(kAll, differ);
      }
      bound = border;
      room = need - reach(value_of(hi));
    }
    if (!whole) count = gather(room, border);
  }
  __syncwarp();
  int mine = -1;                                // lane j: the j-th expert
  if (!whole) {
    for (int c = lane; c < count; c += 32)
      g.c[c] = candidate(__uint_as_float((uint32_t)(g.c[c] >> 32)), (int)(uint32_t)g.c[c]);
    __syncwarp();
    for (int c = lane; c < count; c += 32) {
      const Candidate a = g.c[c];
      int before = 0;
#pragma unroll 4
      for (int j = 0; j < count; ++j) before += g.c[j] > a;
      if (before <= kMaxTop) g.sorted[before] = a;
    }
    __syncwarp();
    const bool has = lane < min(count, p.top);
    if (has) mine = expert_of(g.sorted[lane]);
    if (BIAS) {
      // two keys so close may be in the wrong order, unless they are one logit with one bias
      auto close = [&](float a, float b) { return a - b <= 2.f * eps + (fabsf(a) + fabsf(b)) * 0x1p-23f; };
      auto differ = [&](int a, int b) {
        return to_f(x[a]) != to_f(x[b]) || __ldg(p.bias + a) != __ldg(p.bias + b);
      };
      const Candidate next = g.sorted[min(lane + 1, kMaxTop)];
      bool unsure = has && lane + 1 < count && close(key_of(g.sorted[min(lane, kMaxTop)]), key_of(next));
      if (__any_sync(kAll, unsure)) {
        unsure = unsure && differ(mine, expert_of(next));
        // the first that was not chosen may be the same as the last that was, and hide another
        if (count > p.top) {
          const Candidate last = g.sorted[p.top - 1];
          for (int c = lane; c < count; c += 32)
            if (g.c[c] < last && close(key_of(last), key_of(g.c[c])))
              unsure = unsure || differ(expert_of(last), expert_of(g.c[c]));
        }
      }
      if (__any_sync(kAll, unsure)) {
        const double inv64 = p.softmax ? 1.0 / close_sum(x, p.experts, m) : 0.0;
        for (int c = lane; c < count; c += 32) {
          const int e = expert_of(g.c[c]);
          const double v = to_f(x[e]);
          g.key64[c] = order_of((p.softmax ? exp(v - (double)m) * inv64 : sigmoid(v)) + (double)__ldg(p.bias + e));
        }
        __syncwarp();
        for (int c = lane; c < count; c += 32) {
          int before = 0;
          for (int j = 0; j < count; ++j)
            before += g.key64[j] > g.key64[c] || (g.key64[j] == g.key64[c] && expert_of(g.c[j]) < expert_of(g.c[c]));
          if (before <= kMaxTop) g.sorted[before] = g.c[c], g.sorted64[before] = g.key64[c];
        }
        __syncwarp();
        if (has) mine = expert_of(g.sorted[lane]);
        if (p.softmax) {
          // The sum's error is in all scores alike: a difference of two keys is off by 2^-21 of the scores'
          // difference.  What that leaves open takes the whole row.
          auto unclear = [&](Candidate a, unsigned long long a64, Candidate b, unsigned long long b64) {
            const int ea = expert_of(a), eb = expert_of(b);
            const float ka = key_of(a), kb = key_of(b);
            const float apart = fabsf((ka - __ldg(p.bias + ea)) - (kb - __ldg(p.bias + eb))) + 2.f * eps +
                                (fabsf(ka) + fabsf(kb)) * 0x1p-22f;
            return !((float)(value_of(a64) - value_of(b64)) > apart * 0x1p-21f) && differ(ea, eb);
          };
          bool again = has && lane + 1 < count &&
                       unclear(g.sorted[lane], g.sorted64[lane], g.sorted[lane + 1], g.sorted64[lane + 1]);
          if (count > p.top) {
            const Candidate last = g.sorted[p.top - 1];
            const unsigned long long last64 = g.sorted64[p.top - 1];
            for (int c = lane; c < count; c += 32)
              if (g.key64[c] < last64 || (g.key64[c] == last64 && expert_of(g.c[c]) > expert_of(last)))
                again = again || unclear(last, last64, g.c[c], g.key64[c]);
          }
          whole = __any_sync(kAll, again);
        }
      }
    }
  }
  if (whole) mine = choose_in_64<T, R>(x, p.bias, p.experts, p.top, p.softmax);
  if (lane >= p.top) mine = -1;
  float s = 0.f;
  const float c = mine >= 0 ? to_f(x[mine]) : -INFINITY;
  if (p.softmax) {
    if (p.normalize) {
      m = warp_max(c);
      // a NaN or +inf that was not chosen is in the choice's sum all the same
      s = mine < 0 ? 0.f : BIAS && sum != sum ? sum : expf(c - m);
    } else {
      s = mine >= 0 ? expf(c - m) / sum : 0.f;
    }
  } else if (mine >= 0) {
    s = sigmoid(c);
  }
  if (p.normalize) {
    const float total = warp_sum(s);
    s = total == 0.f ? 0.f : s / total;   // sigmoids that are all 0 in fp32
  }
  if (lane < p.top) {
    p.ids[row * p.top + lane] = mine;
    p.weights[row * p.top + lane] = p.scale * s;
  }
}

// Few experts: a row for every L lanes of a warp, R values each, and k rounds of the L lanes' maximum, whose winner
// looks at its R values again.  65536 rows of 64 bf16, softmax, top 6: 14 us, 20 us with a warp a row; of 16 fp32, top
// 2, 7.5 and 16 us; of 128, top 8, in 16 lanes 34 and 27 us, so those take a warp.
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ int group_min(int v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v = min(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {   // a NaN counts for nothing
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
// 0 for -inf (never chosen), the largest for NaN
__device__ __forceinline__ uint32_t whole_order_of(float v) {
  return v == -INFINITY ? 0u : v != v ? 0xffffffffu : order_of(v);
}

template <typename T, int L, int R, bool BIAS>
__global__ void __launch_bounds__(kThreads) route_few_kernel(const Args p) {
  const int lane = threadIdx.x & 31, me = lane & (L - 1);
  const int64_t first = (blockIdx.x * (int64_t)kWarps + (threadIdx.x >> 5)) * (32 / L);   // the warp's first row
  if (first >= p.rows) return;   // a warp together
  const int64_t row = min(first + lane / L, p.rows - 1);   // groups behind the last row do it again
  const T *x = static_cast<const T *>(p.logits) + row * p.stride;
  uint32_t key[R];
  float m = -INFINITY, sum = 1.f;
  {
    float v[R];
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = i * L + me < p.experts ? to_f(x[i * L + me]) : -INFINITY;
    if (p.softmax && (BIAS || !p.normalize)) {
#pragma unroll
      for (int i = 0; i < R; ++i) m = fmaxf(m, v[i]);
      m = group_max<L>(m);
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) sum += v[i] == -INFINITY ? 0.f : fast_exp(v[i] - m);
      sum = group_sum<L>(sum);
    }
    const float inv = 1.f / sum;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (BIAS && v[i] != -INFINITY)
        v[i] = (p.softmax ? fast_exp(v[i] - m) * inv : fast_inverse(1.f + fast_exp(-v[i]))) +
               __ldg(p.bias + i * L + me);
      key[i] = whole_order_of(v[i]);
    }
  }
  const float eps = p.softmax ? 0x1p-19f / sum : 0x1p-20f;   // as above
  uint32_t best = 0u;
  int at = 0;
  auto look = [&] {
    best = 0u;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (key[i] > best) best = key[i], at = i;
  };
  look();
  int mine = -1, last_e = -1;   // the group's j-th lane: its j-th expert
  float last = 0.f;
  bool unsure = false;
  // two keys so close may be in the wrong order, unless they are one logit with one bias
  auto close = [&](float a, float b) { return a - b <= 2.f * eps + (fabsf(a) + fabsf(b)) * 0x1p-23f; };
  auto differ = [&](int a, int b) { return to_f(x[a]) != to_f(x[b]) || __ldg(p.bias + a) != __ldg(p.bias + b); };
  for (int j = 0; j < p.top; ++j) {
    const uint32_t k = group_max<L>(best);
    const int e = group_min<L>(best == k ? at * L + me : INT_MAX);
    if (BIAS && k) {
      const float v = value_of(k);
      if (j > 0 && close(last, v)) unsure = unsure || differ(last_e, e);
      last = v, last_e = e;
    }
    if (me == j && k) mine = e;
    if (best == k && at * L + me == e) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i == at) key[i] = 0u;
      look();
    }
  }
  if (BIAS && best && close(last, value_of(best))) {   // the last of the choice and all that were not chosen
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (key[i] && close(last, value_of(key[i]))) unsure = unsure || differ(last_e, i * L + me);
  }
  if (BIAS) {
    // the rows that are not sure of their order, one after the other by the whole warp
    unsigned rows = __ballot_sync(kAll, unsure);
    while (rows) {
      const int group = (__ffs(rows) - 1) / L;
      const T *xr = static_cast<const T *>(p.logits) + min(first + group, p.rows - 1) * p.stride;
      const int e = choose_in_64<T, (L * R + 31) / 32>(xr, p.bias, p.experts, p.top, p.softmax);
      const int of = __shfl_sync(kAll, e, me);
      if (lane / L == group) mine = me < p.top ? of : -1;
      rows &= ~(((1u << (L - 1) << 1) - 1u) << (group * L));
    }
  }
  float s = 0.f;
  const float c = mine >= 0 ? to_f(x[mine]) : -INFINITY;
  if (p.softmax) {
    if (p.normalize) {
      m = group_max<L>(c);
      // a NaN or +inf that was not chosen is in the choice's sum all the same
      s = mine < 0 ? 0.f : BIAS && sum != sum ? sum : expf(c - m);
    } else {
      s = mine >= 0 ? expf(c - m) / sum : 0.f;
    }
  } else if (mine >= 0) {
    s = sigmoid(c);
  }
  if (p.normalize) {
    const float total = group_sum<L>(s);
    s = total == 0.f ? 0.f : s / total;   // sigmoids that are all 0 in fp32
  }
  if (me < p.top && first + lane / L < p.rows) {
    p.ids[row * p.top + me] = mine;
    p.weights[row * p.top + me] = p.scale * s;
  }
}

// ---------------------------------------------------------------------------- gradient
//   with g_i = scale dw_i, and for a normalised call share_i = s_i / sum of the chosen s:
//   softmax, normalised:  dx_i = share_i h_i;         h_i = sum_j share_j (g_i - g_j)
//   sigmoid, normalised:  dx_i = share_i (1 - s_i) h_i
//   sigmoid:              dx_i = g_i s_i (1 - s_i)
//   softmax:              dx_e = p_e (sum of g at e - G), G = sum_j g_j p_j; for a chosen expert as
//                         p_e (g_e rest + sum over the chosen c of p_c (g_e - g_c)), rest = the p of the others
// Differences of the g and sums of what is left out, so that nothing cancels where one score is nearly all.  A slot's
// value is added at its expert; an id that comes twice counts twice.
struct BwdArgs {
  const float *dweights;
  const void *logits;
  int64_t stride;
  const int64_t *ids;
  int64_t rows;
  int experts, top;
  bool softmax, normalize;
  float scale;
  void *dlogits;
  int64_t out_stride;
  unsigned *err;
};

// A row for every L lanes, R values each (L below 32 for few experts: 30001 rows of 61, softmax, top 6, 7.4 us,
// 12.3 us with a warp a row).
template <typename T, int L, int R>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const BwdArgs p) {
  const int lane = threadIdx.x & 31, me = lane & (L - 1);
  const int64_t first_row = (blockIdx.x * (int64_t)kWarps + (threadIdx.x >> 5)) * (32 / L);
  if (first_row >= p.rows) return;   // a warp together
  const bool in = first_row + lane / L < p.rows;
  const int64_t row = in ? first_row + lane / L : p.rows - 1;
  const T *x = static_cast<const T *>(p.logits) + row * p.stride;
  int id = -1;
  float g = 0.f, c = -INFINITY;
  if (in && me < p.top) {
    const int64_t v = p.ids[row * p.top + me];
    if (v >= p.experts) atomicOr(p.err, kErrDevice);
    else if (v >= 0) id = (int)v;
    if (id >= 0) g = p.scale * p.dweights[row * p.top + me], c = to_f(x[id]);
  }
  // the warp's row of the gradient where slots meet it: first which experts are chosen, then what is added there
  __shared__ float slots[kThreads / L][R * L];
  float *at = slots[threadIdx.x / L];
#pragma unroll
  for (int i = 0; i < R; ++i) at[i * L + me] = 0.f;
  __syncwarp();
  float out[R];
#pragma unroll
  for (int i = 0; i < R; ++i) out[i] = 0.f;
  // the slots of this lane's expert; the first of them stands for it
  const unsigned same = __match_any_sync(kAll, id >= 0 ? lane / L << 16 | id : -1 - lane);
  const bool first = id >= 0 && (same & ((1u << lane) - 1u)) == 0u;
  const bool twice = __any_sync(kAll, (same & (same - 1u)) != 0u);
  auto added = [&](float v) {              // the sum of v over an expert's slots, for the first of them
    if (!twice) return v;
    float s = 0.f;
    for (int j = 0; j < p.top; ++j) {
      const float o = __shfl_sync(kAll, v, j, L);
      if (same >> (lane - me + j) & 1u) s += o;
    }
    return s;
  };
  float value = 0.f;                       // what this lane's slot adds at its expert
  const bool whole = p.softmax && !p.normalize;
  if (!p.softmax && !p.normalize) {
    if (id >= 0) value = g * sigmoid(c) * (1.f / (1.f + expf(c)));
  } else if (!whole) {
    const float m = p.softmax ? group_max<L>(c) : 0.f;
    const float s = id < 0 || c == -INFINITY ? 0.f : p.softmax ? expf(c - m) : sigmoid(c);
    const float total = group_sum<L>(s), share = total == 0.f ? 0.f : s / total;
    float h = 0.f;
    for (int j = 0; j < p.top; ++j) h = fmaf(__shfl_sync(kAll, share, j, L), g - __shfl_sync(kAll, g, j, L), h);
    if (id >= 0) value = share * h * (p.softmax ? 1.f : 1.f / (1.f + expf(c)));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      out[i] = i * L + me < p.experts ? to_f(x[i * L + me]) : -INFINITY;
      m = fmaxf(m, out[i]);
    }
    m = group_max<L>(m);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      out[i] = out[i] == -INFINITY ? 0.f : expf(out[i] - m);
      sum += out[i];
    }
    sum = group_sum<L>(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;   // a row with nothing but -inf
    const float d = added(g);              // slots of one expert count as one, with their g added
    if (first) at[id] = 1.f;
    __syncwarp();
    const float pr = id < 0 || c == -INFINITY ? 0.f : expf(c - m) * inv;
    const float pf = first ? pr : 0.f;
    float all = pr * g;                    // G, a slot's share
    all = group_sum<L>(all);
    float rest = 0.f;                      // the p of the experts that were not chosen
#pragma unroll
    for (int i = 0; i < R; ++i) {
      out[i] = at[i * L + me] == 0.f ? out[i] * inv : 0.f;
      rest += out[i];
      out[i] *= -all;
    }
    __syncwarp();
    rest = group_sum<L>(rest);
    float h = d * rest;
    for (int j = 0; j < p.top; ++j) h = fmaf(__shfl_sync(kAll, pf, j, L), d - __shfl_sync(kAll, d, j, L), h);
    if (first) value = pr * h;
  }
  if (!whole) value = added(value);
  if (first) at[id] = value;               // 0 elsewhere, but for `whole` where each chosen expert has its own
  __syncwarp();
#pragma unroll
  for (int i = 0; i < R; ++i) out[i] += at[i * L + me];
  T *o = static_cast<T *>(p.dlogits) + row * p.out_stride;
  __syncwarp();   // dlogits may be the logits: every lane has read its own
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (in && i * L + me < p.experts) from_f(o + i * L + me, out[i]);
}

// Calls f with the lanes of a row and the values of a lane.  8 lanes for few experts (figures above); each holds one of
// the row's choices, so 8 of those at most.
template <typename F>
void lanes_of_a_row(int experts, int top, F &&f) {
  constexpr std::integral_constant<int, 8> few{};
  constexpr std::integral_constant<int, 32> warp{};
  if (top <= 8 && experts <= 16) f(few, std::integral_constant<int, 2>());
  else if (top <= 8 && experts <= 32) f(few, std::integral_constant<int, 4>());
  else if (top <= 8 && experts <= 64) f(few, std::integral_constant<int, 8>());
  else if (experts <= 64) f(warp, std::integral_constant<int, 2>());
  else if (experts <= 128) f(warp, std::integral_constant<int, 4>());
  else if (experts <= 256) f(warp, std::integral_constant<int, 8>());
  else if (experts <= 384) f(warp, std::integral_constant<int, 12>());
  else if (experts <= 512) f(warp, std::integral_constant<int, 16>());
  else f(warp, std::integral_constant<int, 32>());
}

bool bad_type(int t) { return t != MUON_BF16 && t != MUON_F32; }
bool bad_score(int s) { return s != MUON_SCORE_SOFTMAX && s != MUON_SCORE_SIGMOID; }

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int muon_route(const void *logits, int64_t stride, const float *bias, int64_t rows, int64_t experts, int type,
               int top, int score, int normalize, float scale, int64_t *ids, float *weights, muon_stream_t stream) {
  if (rows < 0 || experts < 1 || bad_type(type) || bad_score(score) || top < 1 || top > experts || stride < experts ||
      !isfinite(scale))
    return MUON_ERR_INVALID_ARG;
  if (top > kMaxTop || experts > kMaxExperts || rows > kMaxRows) return MUON_ERR_UNSUPPORTED;
  if (rows == 0) return MUON_OK;
  if (!logits || !ids || !weights) return MUON_ERR_INVALID_ARG;
  if (!on_elements({logits}, type == MUON_BF16 ? 2 : 4) || !on_elements({bias, weights}, 4) || !on_elements({ids}, 8))
    return MUON_ERR_UNSUPPORTED;
  const Args a{logits, stride, bias, rows, (int)experts, top, score == MUON_SCORE_SOFTMAX, normalize != 0, scale, ids,
               weights};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  trace_before(kTraceRoute, s);
  lanes_of_a_row((int)experts, top, [&](auto l, auto r) {
    constexpr int L = decltype(l)::value, R = decltype(r)::value;
    const unsigned blocks = (unsigned)((rows + kThreads / L - 1) / (kThreads / L));
    auto run = [&](auto element, auto with_bias) {
      typedef decltype(element) T;
      constexpr bool BIAS = decltype(with_bias)::value;
      if constexpr (L == 32) route_kernel<T, R, BIAS><<<blocks, kThreads, 0, s>>>(a);
      else route_few_kernel<T, L, R, BIAS><<<blocks, kThreads, 0, s>>>(a);
    };
    auto with = [&](auto element) {
      if (bias) run(element, std::true_type());
      else run(element, std::false_type());
    };
    if (type == MUON_BF16) with(__nv_bfloat16());
    else with(float());
  });
  return trace_after(kTraceRoute, s);
}

int muon_route_backward(const float *dweights, const void *logits, int64_t stride, const int64_t *ids, int64_t rows,
                        int64_t experts, int type, int top, int score, int normalize, float scale, void *dlogits,
                        int64_t dlogits_stride, muon_stream_t stream) {
  if (rows < 0 || experts < 1 || bad_type(type) || bad_score(score) || top < 1 || top > experts || stride < experts ||
      dlogits_stride < experts || !isfinite(scale))
    return MUON_ERR_INVALID_ARG;
  if (top > kMaxTop || experts > kMaxExperts || rows > kMaxRows) return MUON_ERR_UNSUPPORTED;
  if (rows == 0) return MUON_OK;
  if (!dweights || !logits || !ids || !dlogits) return MUON_ERR_INVALID_ARG;
  if (!on_elements({logits, dlogits}, type == MUON_BF16 ? 2 : 4) || !on_elements({dweights}, 4) ||
      !on_elements({ids}, 8))
    return MUON_ERR_UNSUPPORTED;
  const BwdArgs a{dweights, logits, stride, ids, rows, (int)experts, top, score == MUON_SCORE_SOFTMAX, normalize != 0,
                  scale, dlogits, dlogits_stride, device_error_word()};
  if (!a.err) return MUON_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  trace_before(kTraceRouteBwd, s);
  lanes_of_a_row((int)experts, top, [&](auto l, auto r) {
    constexpr int L = decltype(l)::value, R = decltype(r)::value;
    const unsigned blocks = (unsigned)((rows + kThreads / L - 1) / (kThreads / L));
    if (type == MUON_BF16) route_backward_kernel<__nv_bfloat16, L, R><<<blocks, kThreads, 0, s>>>(a);
    else route_backward_kernel<float, L, R><<<blocks, kThreads, 0, s>>>(a);
  });
  return trace_after(kTraceRouteBwd, s);
}

}  // extern "C"
